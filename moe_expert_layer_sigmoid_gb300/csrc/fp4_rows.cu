// Rows to 4-bit floats with a scale for each 16 of them, and back.
//
//   s = absmax(row) / 2688,  b = e4m3(absmax(block) / (6 s)),  code = e2m1(x / (b s))
// A thread takes a block of 16 elements and keeps it in registers while the row's largest magnitude is
// found, so a row is read once; the bound is DRAM bandwidth, and for a few rows the launch.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "fp4.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void load16(const uint16_t* p, float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            f[8 * i + 2 * n] = bf16_lo(w[n]);
            f[8 * i + 2 * n + 1] = bf16_hi(w[n]);
        }
    }
}
__device__ __forceinline__ void load16(const float* p, float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 x = reinterpret_cast<const float4*>(p)[i];
        f[4 * i] = x.x; f[4 * i + 1] = x.y; f[4 * i + 2] = x.z; f[4 * i + 3] = x.w;
    }
}

// One block's scale and codes, the row's scale known.
__device__ __forceinline__ uint32_t quant_block(const float (&f)[16], float m, float s, uint2& codes) {
    const float six = 6.0f * s;
    const uint32_t b =
        six > 0.0f ? (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(m, six), __NV_SATFINITE, __NV_E4M3) : 0u;
    const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
    const float t = __half2float(*reinterpret_cast<const __half*>(&hr)) * s;
    uint32_t c[2] = {0, 0};
    if (t > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 y = make_float2(__fdiv_rn(f[2 * i], t), __fdiv_rn(f[2 * i + 1], t));
            c[i / 4] |= (uint32_t)__nv_cvt_float2_to_fp4x2(y, __NV_E2M1, cudaRoundNearest) << (8 * (i % 4));
        }
    }
    codes = make_uint2(c[0], c[1]);
    return b;
}

// threads.x (a multiple of 32) threads take a row, threads.y rows a CTA; a thread up to PER blocks.
template <typename Src, int PER>
__global__ void __launch_bounds__(1024) quant_kernel(const Src* __restrict__ src, int64_t ld, int64_t rows, int K,
                                                     Fp4Rows out) {
    __shared__ float part[32];
    pdl_trigger();  // the projection's kernel fetches weights meanwhile
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int blocks = K / 16, lane = threadIdx.x & 31;
    float f[PER][16], m[PER];
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int at = threadIdx.x + j * blockDim.x;
        m[j] = 0.0f;
        if (r < rows && at < blocks) {
            load16(src + r * ld + 16 * at, f[j]);
#pragma unroll
            for (int i = 0; i < 16; ++i) m[j] = fmaxf(m[j], fabsf(f[j][i]));
        }
        top = fmaxf(top, m[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (blockDim.x > 32) {
        const int warps = blockDim.x >> 5;  // of a row
        if (lane == 0) part[threadIdx.y * warps + (threadIdx.x >> 5)] = top;
        __syncthreads();
        top = lane < warps ? part[threadIdx.y * warps + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    if (r >= rows) return;
    const float s = __fdiv_rn(top, 2688.0f);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int at = threadIdx.x + j * blockDim.x;
        if (at >= blocks) break;
        uint2 c;
        const uint32_t b = quant_block(f[j], m[j], s, c);
        *reinterpret_cast<uint2*>(out.q + r * (K / 2) + 8 * at) = c;
        out.b[fp4_scale_at(r, at, K)] = (uint8_t)b;
    }
    if (threadIdx.x == 0) out.s[r] = s;
}

__device__ __forceinline__ float e4m3_value(uint32_t b) {
    const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&hr));
}

// The 16 values of a block's codes, without scales.
__device__ __forceinline__ void code_values(uint2 c, float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t two = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu;
        const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

__global__ void __launch_bounds__(256) unpack_kernel(moe_fp4_t w, int64_t rows, int K, uint16_t* __restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int blocks = K / 16;
    const int64_t r = i / blocks;
    if (r >= rows) return;
    const int j = (int)(i - r * blocks);
    float f[16];
    code_values(*reinterpret_cast<const uint2*>(w.q + r * (K / 2) + 8 * j), f);
    const float t = e4m3_value(w.b[fp4_scale_at(r, j, K)]) * w.s[r];
    uint32_t o[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * n] * t, f[2 * n + 1] * t);
        o[n] = *reinterpret_cast<const uint32_t*>(&v);
    }
    uint4* p = reinterpret_cast<uint4*>(out + r * K + 16 * j);
    p[0] = make_uint4(o[0], o[1], o[2], o[3]);
    p[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <typename Src>
cudaError_t launch_quant(const Src* src, int64_t ld, int64_t rows, int64_t K, const Fp4Rows& out, cudaStream_t st) {
    const int blocks = (int)(K / 16);
    const int per = blocks <= 1024 ? 1 : blocks <= 2048 ? 2 : 4;
    const int x = ((blocks + per - 1) / per + 31) / 32 * 32;
    const int y = per == 1 ? std::max(1, 256 / x) : 1;
    const unsigned grid = (unsigned)((rows + y - 1) / y);
    const dim3 threads(x, y);
    if (per == 1) quant_kernel<Src, 1><<<grid, threads, 0, st>>>(src, ld, rows, (int)K, out);
    else if (per == 2) quant_kernel<Src, 2><<<grid, threads, 0, st>>>(src, ld, rows, (int)K, out);
    else quant_kernel<Src, 4><<<grid, threads, 0, st>>>(src, ld, rows, (int)K, out);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_fp4(const void* src, bool bf16, int64_t ld, int64_t rows, int64_t K, Fp4Rows out,
                             cudaStream_t st) {
    return bf16 ? launch_quant(static_cast<const uint16_t*>(src), ld, rows, K, out, st)
                : launch_quant(static_cast<const float*>(src), ld, rows, K, out, st);
}

cudaError_t launch_unpack_fp4(moe_fp4_t w, int64_t rows, int64_t K, uint16_t* out, cudaStream_t st) {
    const int64_t threads = rows * (K / 16);
    unpack_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(w, rows, (int)K, out);
    return cudaGetLastError();
}

}  // namespace moe
