// Rotary positions: launchers and the frequencies behind the table.
#pragma once

#include "kv.cuh"

namespace moe {

struct RopeWriteArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv, ldo;
    const int32_t *pos, *slots;
    moe_rope_t rope;
    moe_kv_dims_t d;
    moe_kv_t cache;
    uint16_t* out;
    WsHeader* hdr;
};

// The angle of pair i from one position to the next, at most 1.
double rope_frequency(const moe_rope_config_t& g, int i);
cudaError_t launch_rope_table(const moe_rope_config_t& g, int32_t pos0, int32_t n_pos, float* table,
                              cudaStream_t st);
cudaError_t launch_rope_rows(const uint16_t* x, int64_t ldx, const int32_t* pos, int32_t T, int32_t H, int32_t D,
                             const moe_rope_t& rope, uint16_t* out, int64_t ldo, WsHeader* hdr, cudaStream_t st);
cudaError_t launch_rope_kv_write(const RopeWriteArgs& a, cudaStream_t st);

}  // namespace moe
