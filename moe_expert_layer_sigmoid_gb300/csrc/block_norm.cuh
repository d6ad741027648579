// The norms between blocks: the launcher.
#pragma once

#include "common.cuh"

namespace moe {

cudaError_t launch_block_norm(const uint16_t* y, const void* residual, const void* gate, const float* w_post,
                              const float* w_pre, const moe_norm_dims_t& d, void* residual_out, uint16_t* x,
                              cudaStream_t st);

}  // namespace moe
