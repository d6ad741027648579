// The paged key/value cache as the kernels see it: row formats, addressing of
// a pool, and the launchers of the calls on it.
#pragma once

#include "common.cuh"

namespace moe {

enum KvFormat : int { kKvBf16 = 0, kKvE4m3 = 1, kKvInt4 = 2 };

constexpr int kv_row_bytes(int fmt, int D) {
    return fmt == kKvBf16 ? 2 * D : fmt == kKvE4m3 ? D : D / 2;
}

// One pool's rows (keys or values) and their scales.
struct KvRows {
    uint8_t* q;
    float* s;
    int64_t page_stride, head_stride, slot_stride;  // bytes
    __device__ __forceinline__ int64_t offset(int page, int h, int slot) const {
        return page * page_stride + h * head_stride + slot * slot_stride;
    }
};
__host__ __device__ inline KvRows kv_rows(const moe_kv_t& c, bool keys) {
    return KvRows{static_cast<uint8_t*>(keys ? c.k : c.v), keys ? c.ks : c.vs, c.page_stride,
                  c.head_stride, c.slot_stride};
}

struct AttnArgs {
    const uint16_t* q;
    int64_t ldq;
    const int32_t* q_off;
    const int32_t* kv_len;
    const int32_t* pages;
    moe_kv_dims_t d;
    moe_kv_t cache;
    float scale;
    uint16_t* out;
    float* lse;
    WsHeader* hdr;
};

cudaError_t launch_kv_write(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                            const int32_t* slots, const moe_kv_dims_t& d, const moe_kv_t& cache,
                            WsHeader* hdr, cudaStream_t st);
cudaError_t launch_kv_read(const int32_t* slots, const moe_kv_dims_t& d, const moe_kv_t& cache,
                           uint16_t* k, uint16_t* v, WsHeader* hdr, cudaStream_t st);
size_t attn_workspace_bytes(const moe_kv_dims_t& d);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st);

}  // namespace moe
