// Projections with both operands in microscaled 4-bit floats.
//
// out[t][n] = (sum over blocks bx bw (sum of 16 code products)) * s_x * s_w.  The plain form: tiles of 64
// tokens and 64 outputs, codes times block scales as fp32 in shared memory.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "fp4.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void block_values(const moe_fp4_t& w, int64_t r, int64_t rows, int j, int K, float* to) {
    if (r >= rows) {
#pragma unroll
        for (int i = 0; i < 16; ++i) to[i] = 0.0f;
        return;
    }
    const uint2 c = *reinterpret_cast<const uint2*>(w.q + r * (K / 2) + 8 * j);
    const __half_raw hb = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)w.b[fp4_scale_at(r, j, K)], __NV_E4M3);
    const float b = __half2float(*reinterpret_cast<const __half*>(&hb));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t two = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu;
        const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        to[2 * i] = v.x * b;
        to[2 * i + 1] = v.y * b;
    }
}

__global__ void __launch_bounds__(256) linear_kernel(moe_fp4_t x, moe_fp4_t w, int T, int N, int K,
                                                     uint16_t* __restrict__ out) {
    __shared__ float xs[64][65], ws[64][65];
    const int64_t t0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k = 0; k < K; k += 64) {
        const int r = threadIdx.x >> 2, j = threadIdx.x & 3;
        block_values(x, t0 + r, T, k / 16 + j, K, &xs[r][16 * j]);
        block_values(w, n0 + r, N, k / 16 + j, K, &ws[r][16 * j]);
        __syncthreads();
        for (int i = 0; i < 64; ++i)
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[a][c] += xs[ty + 16 * a][i] * ws[tx + 16 * c][i];
        __syncthreads();
    }
    for (int a = 0; a < 4; ++a)
        for (int c = 0; c < 4; ++c) {
            const int64_t t = t0 + ty + 16 * a, n = n0 + tx + 16 * c;
            if (t < T && n < N) out[t * N + n] = float_to_bf16_bits(acc[a][c] * x.s[t] * w.s[n]);
        }
}

}  // namespace

cudaError_t launch_linear_fp4(moe_fp4_t x, moe_fp4_t w, int T, int N, int K, uint16_t* out, void*,
                              cudaStream_t st) {
    linear_kernel<<<dim3((N + 63) / 64, (T + 63) / 64), 256, 0, st>>>(x, w, T, N, K, out);
    return cudaGetLastError();
}

}  // namespace moe
