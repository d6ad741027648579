// Blocks of 16 elements as 4-bit floats: what every kernel that makes them shares.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "fp4.cuh"

namespace moe {

__device__ __forceinline__ float e4m3_value(uint32_t b) {
    const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&hr));
}

__device__ __forceinline__ void load16(const uint4* p, float (&f)[16]) {  // (bf16)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 x = p[i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            f[8 * i + 2 * n] = bf16_lo(w[n]);
            f[8 * i + 2 * n + 1] = bf16_hi(w[n]);
        }
    }
}
__device__ __forceinline__ void load16(const uint16_t* p, float (&f)[16]) {
    load16(reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void load16(const float* p, float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 x = reinterpret_cast<const float4*>(p)[i];
        f[4 * i] = x.x; f[4 * i + 1] = x.y; f[4 * i + 2] = x.z; f[4 * i + 3] = x.w;
    }
}

// f / t from t's rounded reciprocal r: the product corrected by its own remainder (P. Markstein, IBM J. Res. Dev. 34,
// 1990).  Written so that a zero keeps its sign.
// The result is the rounded quotient unless the exact one lies within 2^-23 of a unit of where rounding changes.  For the
// codes that could matter beside a border M (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5) only, where f = t (M +- half a unit) but for
// that much: with T t's 24 bits, F f's 8 and M = a 2^e (a 1, 3, 5 or 7), |F 2^k - T (a 2^s +- 1)| < 8 units, k at least 40.  T's
// low bits then are e' or -e' for some e' < 8, and the middle of the product vanishes only if a e' is the number j (1 to 4)
// of quarters in T's first digits: a = 1, T = 2^24 - 1, F a power of 2, and there the steps below come out right.
__device__ __forceinline__ float quotient8(float f, float t, float r) {
    const float y = f * r;
    return __fmaf_rn(-__fmaf_rn(y, t, -f), r, y);
}

// f / s rounded once for any f and s: corrected twice, the first time to within a unit, which is what the theorem asks.
__device__ __forceinline__ float quotient24(float f, float s, float r) {
    const float y = quotient8(f, s, r);
    return __fmaf_rn(-__fmaf_rn(y, s, -f), r, y);
}

// A row's scale and what every block of it needs of that.  `usual`: nothing on the way is tiny or infinite.
struct RowScale {
    float s, six, r_six;
    bool usual;
};
__device__ __forceinline__ RowScale row_scale(float top) {
    RowScale q;
    q.s = __fdiv_rn(top, 2688.0f);
    q.six = 6.0f * q.s;
    q.r_six = __frcp_rn(q.six);
    q.usual = q.s > 0x1p-50f && q.s < 0x1p90f;
    return q;
}

// Eight quotients as codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes_of_8(const float* y) {
    uint32_t c;
    asm("{\n .reg .b8 p, q, r, s;\n"
        " cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n"
        " mov.b32 %0, {p, q, r, s};\n}"
        : "=r"(c)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return c;
}

// A block's codes and scale, m its largest magnitude.  The recipe's codes are those of the fp32 quotients: bf16 values
// lie between two codes so often that the last bit matters.  BF16: the elements are bf16 values.
template <bool BF16>
__device__ __forceinline__ uint32_t quant_block(const float (&f)[16], float m, const RowScale& q, uint2& codes) {
    // (a largest magnitude so small that something is lost on the way has the scale 0 either way)
    const float ratio = q.usual ? quotient24(m, q.six, q.r_six) : q.six > 0.0f ? __fdiv_rn(m, q.six) : 0.0f;
    const uint32_t b = (uint32_t)__nv_cvt_float_to_fp8(ratio, __NV_SATFINITE, __NV_E4M3);
    const float t = e4m3_value(b) * q.s;
    uint32_t c[2] = {0, 0};
    if (t > 0.0f) {
        float y[16];
        if (BF16 && q.usual) {
            // (elements so small that something on the way is lost are far below the first border)
            const float r = __frcp_rn(t);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = quotient8(f[i], t, r);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(f[i], t);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = codes_of_8(y + 8 * i);
    }
    codes = make_uint2(c[0], c[1]);
    return b;
}

}  // namespace moe
