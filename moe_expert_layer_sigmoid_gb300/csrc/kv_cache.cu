// Writing new keys and values into the paged cache, and reading slots back.
//
// Row x[D] of a token and head, with the recipes of the weight formats and one
// fp32 scale per row:
//   E4M3: s = absmax / 448, code = e4m3(x / s);  int4: s = absmax / 7,
//   q = clamp(rint(x / s), -8, 7);  s = 0 gives codes 0.
// Both kernels move each byte once: the bound is DRAM bandwidth, and for small
// calls the launch.  D / 16 lanes take a row, two pieces of 16 bytes of bf16 each, of the
// keys and of the values, so what is done once per row is spread over 32 values, and
// three (D = 128) or two exchanges make the absolute maxima of both.
//
// Measured (GB300, 65537 tokens of 8 heads of 128, us and TB/s; a copy's bandwidth is 6.8):
//   bf16 write 81.7, 6.6    read 82.0, 6.5
//   E4M3 write 73.4, 5.5    read 66.8, 6.1
//   int4 write 71.8, 4.7    read 61.8, 5.5
// The writes of codes are held up by their arithmetic (E4M3 46% ALU, 57% of issue slots).
#include <cuda_fp8.h>

#include "kv.cuh"

namespace moe {
namespace {

struct KvCopyParams {
    const uint16_t* k;   // write: new rows; read: unused
    const uint16_t* v;
    int64_t ldk, ldv;    // elements from token to token
    uint16_t* k_out;     // read: the rows, contiguous
    uint16_t* v_out;
    const int32_t* slots;
    KvRows kr, vr;
    WsHeader* hdr;
    int T, H_kv, page, page_log2, n_slots;
    // i / H_kv = i * h_mul >> h_shift for every i < 2^31: h_mul is 2^h_shift / H_kv rounded up, and the
    // rounding adds less than i / 2^h_shift <= 1 / H_kv
    uint32_t h_mul;
    int h_shift;
};

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

// The codes of eight quotients.  int4: no quotient by s rounds to more than 7 in magnitude, so the
// recipe's clamp has nothing to do; adding 1.5 * 2^23 leaves the rounded number in the low bits.
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

// A lane's two pieces of a row, as bf16.
template <int FMT, int D>
__device__ __forceinline__ void load_row(uint4 (&x)[2], const uint8_t* row, const float* scale, int sub) {
    constexpr int kLanes = D / 16;
    const float s = FMT == kKvBf16 ? 0.0f : *scale;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int at = sub + j * kLanes;
        uint32_t w[4];
        if (FMT == kKvBf16) {
            x[j] = reinterpret_cast<const uint4*>(row)[at];
            continue;
        } else if (FMT == kKvE4m3) {
            const uint2 c = reinterpret_cast<const uint2*>(row)[at];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c2 = ((i < 2 ? c.x : c.y) >> (16 * (i & 1))) & 0xFFFFu;
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c2, __NV_E4M3);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                w[i] = pack_bf16(f.x * s, f.y * s);
            }
        } else {
            const uint32_t c = reinterpret_cast<const uint32_t*>(row)[at];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int lo = (int)(c << (28 - 8 * i)) >> 28, hi = (int)(c << (24 - 8 * i)) >> 28;
                w[i] = pack_bf16((float)lo * s, (float)hi * s);
            }
        }
        x[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int FMT, int D, bool WRITE>
__global__ void __launch_bounds__(256, 5) kv_copy_kernel(const KvCopyParams p) {
    constexpr int kLanes = D / 16;  // lanes of a row
    const unsigned i = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;  // row: token and head (below 2^31)
    const int sub = threadIdx.x % kLanes;
    const bool live = i < (unsigned)p.T * (unsigned)p.H_kv;
    const int t = live ? (int)((uint64_t)i * p.h_mul >> p.h_shift) : 0, h = live ? (int)i - t * p.H_kv : 0;
    int slot = live ? p.slots[t] : -1;
    if (slot >= p.n_slots) {
        if (sub == 0) record_error(p.hdr, kErrBadSlot);
        slot = -1;
    }
    const bool put = slot >= 0;
    const int page = put ? slot >> p.page_log2 : 0, at = put ? slot & (p.page - 1) : 0;
    // (one offset for both pools and one for both scales)
    const int64_t row = p.kr.offset(page, h, at), scale = ((int64_t)page * p.H_kv + h) * p.page + at;
    uint4 k[2], v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) k[j] = v[j] = make_uint4(0, 0, 0, 0);
    if (WRITE) {
        if (put) {
            const uint4* pk = reinterpret_cast<const uint4*>(p.k + t * p.ldk + h * D) + sub;
            const uint4* pv = reinterpret_cast<const uint4*>(p.v + t * p.ldv + h * D) + sub;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                k[j] = pk[j * kLanes];
                v[j] = pv[j * kLanes];
            }
        }
        float mk = 0.0f, mv = 0.0f;
        if (FMT != kKvBf16) {
            // Magnitudes of bf16 are bf16: keys' in the low half and values' in the high one, one exchange for both.
            const uint32_t a = absmax_pair(k[0], k[1]), b = absmax_pair(v[0], v[1]);
            uint32_t m = max_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) m = max_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            mk = fmaxf(bf16_lo(m), 0.0f);  // (a row of NaN alone has none)
            mv = fmaxf(bf16_hi(m), 0.0f);
        }
        if (!put) return;
        store_row<FMT, D>(k, mk, p.kr.q + row, p.kr.s + scale, sub);
        store_row<FMT, D>(v, mv, p.vr.q + row, p.vr.s + scale, sub);
    } else if (live) {
        if (put) {
            load_row<FMT, D>(k, p.kr.q + row, p.kr.s + scale, sub);
            load_row<FMT, D>(v, p.vr.q + row, p.vr.s + scale, sub);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            reinterpret_cast<uint4*>(p.k_out)[(int64_t)i * (D / 8) + sub + j * kLanes] = k[j];
            reinterpret_cast<uint4*>(p.v_out)[(int64_t)i * (D / 8) + sub + j * kLanes] = v[j];
        }
    }
}

template <bool WRITE>
cudaError_t launch_copy(const KvCopyParams& p, const moe_kv_dims_t& d, cudaStream_t st) {
    const int rows = 256 / (d.D / 16);  // of a CTA
    const unsigned grid = (unsigned)(((int64_t)d.T * d.H_kv + rows - 1) / rows);
    const bool wide = d.D == 128;
    switch (d.format) {
        case kKvBf16:
            if (wide) kv_copy_kernel<kKvBf16, 128, WRITE><<<grid, 256, 0, st>>>(p);
            else kv_copy_kernel<kKvBf16, 64, WRITE><<<grid, 256, 0, st>>>(p);
            break;
        case kKvE4m3:
            if (wide) kv_copy_kernel<kKvE4m3, 128, WRITE><<<grid, 256, 0, st>>>(p);
            else kv_copy_kernel<kKvE4m3, 64, WRITE><<<grid, 256, 0, st>>>(p);
            break;
        case kKvInt4:
            if (wide) kv_copy_kernel<kKvInt4, 128, WRITE><<<grid, 256, 0, st>>>(p);
            else kv_copy_kernel<kKvInt4, 64, WRITE><<<grid, 256, 0, st>>>(p);
            break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

KvCopyParams copy_params(const int32_t* slots, const moe_kv_dims_t& d, const moe_kv_t& cache,
                         WsHeader* hdr) {
    KvCopyParams p{};
    p.slots = slots;
    p.kr = kv_rows(cache, true);
    p.vr = kv_rows(cache, false);
    p.hdr = hdr;
    p.T = d.T;
    p.H_kv = d.H_kv;
    p.h_shift = 31;
    while ((1ll << (p.h_shift - 31)) < p.H_kv) ++p.h_shift;
    p.h_mul = (uint32_t)(((1ull << p.h_shift) + p.H_kv - 1) / p.H_kv);
    p.page = d.page;
    p.page_log2 = __builtin_ctz(d.page);
    p.n_slots = d.n_pages * d.page;
    return p;
}

}  // namespace

cudaError_t launch_kv_write(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                            const int32_t* slots, const moe_kv_dims_t& d, const moe_kv_t& cache,
                            WsHeader* hdr, cudaStream_t st) {
    KvCopyParams p = copy_params(slots, d, cache, hdr);
    p.k = k;
    p.ldk = ldk;
    p.v = v;
    p.ldv = ldv;
    return launch_copy<true>(p, d, st);
}

cudaError_t launch_kv_read(const int32_t* slots, const moe_kv_dims_t& d, const moe_kv_t& cache,
                           uint16_t* k, uint16_t* v, WsHeader* hdr, cudaStream_t st) {
    KvCopyParams p = copy_params(slots, d, cache, hdr);
    p.k_out = k;
    p.v_out = v;
    return launch_copy<false>(p, d, st);
}

}  // namespace moe
