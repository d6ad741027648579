// Rows of the paged cache as codes: what every kernel that writes them shares.
#pragma once

#include <cuda_fp8.h>

#include "kv.cuh"

namespace moe {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The largest magnitude of a lane's two pieces of a row, in one of the two halves each.
__device__ __forceinline__ uint32_t absmax_pair(uint4 a, uint4 b) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    return max_bf16x2(max_bf16x2(max_bf16x2(a.x & kAbs, a.y & kAbs), max_bf16x2(a.z & kAbs, a.w & kAbs)),
                      max_bf16x2(max_bf16x2(b.x & kAbs, b.y & kAbs), max_bf16x2(b.z & kAbs, b.w & kAbs)));
}

// f / s rounded once, from the rounded reciprocal r of s: f * r corrected by its own remainder
// (P. Markstein, IBM J. Res. Dev. 34, 1990), which is exact while nothing is tiny or infinite.
// Written so that a zero keeps its sign.
__device__ __forceinline__ float quotient(float f, float s, float r) {
    const float y = f * r;
    return __fmaf_rn(-__fmaf_rn(y, s, -f), r, y);
}

// The codes of eight quotients.  int4: they round to -8 .. 7, which those of bf16 rows do without the recipe's clamp (a seventh
// of 2^-133 or more keeps 13 bits, so no quotient by it rounds to more than 7 in magnitude); fp32 rows are clamped by who
// calls.  Adding 1.5 * 2^23 leaves the rounded number in the low bits.
template <int FMT>
__device__ __forceinline__ uint2 codes_of(const float (&f)[8]) {
    if (FMT == kKvE4m3) {
        uint32_t d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        return make_uint2(d[0] | d[1] << 16, d[2] | d[3] << 16);
    }
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t low = (1u << (4 * i)) - 1;  // what is in place
        d = (d & low) | (__float_as_uint(f[i] + 12582912.0f) << (4 * i) & ~low);
    }
    return make_uint2(d, 0);
}

// The codes of eight values; `plain` for scales that the corrected product does not hold for.
template <int FMT>
__device__ __forceinline__ uint2 quantised(uint4 x, float s, float r, bool plain) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
    if (plain) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], s);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = quotient(f[i], s, r);
    }
    return codes_of<FMT>(f);
}

// Stores a lane's two pieces of a row whose largest magnitude is m, as bf16 or as codes with their scale.
template <int FMT, int D>
__device__ __forceinline__ void store_row(const uint4 (&x)[2], float m, uint8_t* row, float* scale, int sub) {
    constexpr int kLanes = D / 16;
    if (FMT == kKvBf16) {
#pragma unroll
        for (int j = 0; j < 2; ++j) reinterpret_cast<uint4*>(row)[sub + j * kLanes] = x[j];
        return;
    }
    constexpr float kTop = FMT == kKvE4m3 ? 448.0f : 7.0f;
    // The recipe's code is that of the fp32 quotient, and bf16 values over a bf16 maximum lie on
    // midpoints between codes so often that its last bit matters.  A division for each element
    // made the kernel issue-bound (115 us against 62 us of DRAM time at 65537 tokens of 8
    // E4M3 heads).
    const bool plain = m < 0x1p-70f || m == __int_as_float(0x7F800000);
    const float s = plain ? m / kTop : quotient(m, kTop, 1.0f / kTop);
    uint2 c[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    if (s > 0.0f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int j = 0; j < 2; ++j) c[j] = quantised<FMT>(x[j], s, r, plain);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (FMT == kKvE4m3) reinterpret_cast<uint2*>(row)[sub + j * kLanes] = c[j];
        else reinterpret_cast<uint32_t*>(row)[sub + j * kLanes] = c[j].x;
    }
    if (sub == 0) *scale = s;
}

}  // namespace moe
