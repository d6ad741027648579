// Writing new keys and values into the paged cache, and reading slots back.
//
// Row x[D] of a token and head, with the recipes of the weight formats and one
// fp32 scale per row:
//   E4M3: s = absmax / 448, code = e4m3(x / s);  int4: s = absmax / 7,
//   q = clamp(rint(x / s), -8, 7);  s = 0 gives codes 0.
// Both kernels move each byte once: the bound is DRAM bandwidth, and for small
// calls the launch.  D / 8 lanes take a row, 16 bytes of bf16 each, so a warp
// has two (D = 128) or four rows' absolute maxima in a few shuffles; keys and
// values go in one launch, the lane holding its 16 bytes of both.
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
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
}

// The codes of two quotients: two E4M3 bytes, or two nibbles.
template <int FMT>
__device__ __forceinline__ uint32_t pair_code(float a, float b) {
    if (FMT == kKvE4m3) return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    return (__float2int_rn(fminf(fmaxf(a, -8.0f), 7.0f)) & 15) | (__float2int_rn(fminf(fmaxf(b, -8.0f), 7.0f)) & 15) << 4;
}

// Quantises the row that D / 8 neighbouring lanes hold (8 values each) and
// stores codes and scale where `put`; every lane of the warp takes part (the
// lanes of a row all put or all do not).
template <int FMT, int D>
__device__ __forceinline__ void store_row(uint4 x, const KvRows& r, int page, int h, int slot,
                                          int page_slots, int H_kv, int sub, bool put) {
    uint8_t* row = r.row(page, h, slot);
    if (FMT == kKvBf16) {
        if (put) *reinterpret_cast<uint4*>(row + 16 * sub) = x;
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8], m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
        m = fmaxf(m, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
    }
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float s = m / (FMT == kKvE4m3 ? 448.0f : 7.0f);
    if (!put) return;
    uint32_t code[2] = {0, 0};
    if (s > 0.0f) {
        // The recipe's code is that of the fp32 quotient f / s, and bf16 values over a bf16 maximum lie on
        // midpoints between codes so often that its last bit matters.  A division for each element
        // made the kernel issue-bound (115 us against 62 us of DRAM time at 65537 tokens of 8
        // E4M3 heads).  With the rounded reciprocal r of the row's scale, f * r corrected by
        // its own remainder is the rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990); the remainder
        // is exact while s is not tiny.
        const float r = 1.0f / s;
        if (s < 0x1p-80f) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                // (by pairs from the row's words: no indexing of registers)
                const uint32_t x2 = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
                const uint32_t d = pair_code<FMT>(bf16_lo(x2) / s, bf16_hi(x2) / s);
                if (FMT != kKvE4m3) code[0] |= d << (8 * i);
                else if (i < 2) code[0] |= d << (16 * i);
                else code[1] |= d << (16 * i - 32);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = f[i] * r, q = __fmaf_rn(__fmaf_rn(-y, s, f[i]), r, y);
                f[i] = copysignf(q, f[i]);  // (-0 stays -0)
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t d = pair_code<FMT>(f[2 * i], f[2 * i + 1]);
                if (FMT == kKvE4m3) code[i / 2] |= d << (16 * (i & 1));
                else code[0] |= d << (8 * i);
            }
        }
    }
    if (FMT == kKvE4m3) *reinterpret_cast<uint2*>(row + 8 * sub) = make_uint2(code[0], code[1]);
    else *reinterpret_cast<uint32_t*>(row + 4 * sub) = code[0];
    if (sub == 0) r.s[((int64_t)page * H_kv + h) * page_slots + slot] = s;
}

// The eight values that a lane's codes stand for, as bf16.
template <int FMT>
__device__ __forceinline__ uint4 load_row(const KvRows& r, int page, int h, int slot, int page_slots,
                                          int H_kv, int sub) {
    const uint8_t* row = r.row(page, h, slot);
    if (FMT == kKvBf16) return *reinterpret_cast<const uint4*>(row + 16 * sub);
    const float s = r.s[((int64_t)page * H_kv + h) * page_slots + slot];
    uint32_t w[4];
    if (FMT == kKvE4m3) {
        const uint2 c = *reinterpret_cast<const uint2*>(row + 8 * sub);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c2 = ((i < 2 ? c.x : c.y) >> (16 * (i & 1))) & 0xFFFFu;
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c2, __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            w[i] = pack_bf16(f.x * s, f.y * s);
        }
    } else {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(row + 4 * sub);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int lo = (int)(c << (28 - 8 * i)) >> 28, hi = (int)(c << (24 - 8 * i)) >> 28;
            w[i] = pack_bf16((float)lo * s, (float)hi * s);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int FMT, int D, bool WRITE>
__global__ void __launch_bounds__(256) kv_copy_kernel(const KvCopyParams p) {
    constexpr int kLanes = D / 8;  // lanes of a row
    const unsigned i = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;  // row: token and head (below 2^31)
    const int sub = threadIdx.x % kLanes;
    const bool live = i < (unsigned)p.T * (unsigned)p.H_kv;
    const int t = live ? i / (unsigned)p.H_kv : 0, h = live ? i - t * (unsigned)p.H_kv : 0;
    int slot = live ? p.slots[t] : -1;
    if (slot >= p.n_slots) {
        if (sub == 0) record_error(p.hdr, kErrBadSlot);
        slot = -1;
    }
    const bool put = slot >= 0;
    const int page = put ? slot >> p.page_log2 : 0, at = put ? slot & (p.page - 1) : 0;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (WRITE) {
        if (put) {
            k = *reinterpret_cast<const uint4*>(p.k + t * p.ldk + h * D + 8 * sub);
            v = *reinterpret_cast<const uint4*>(p.v + t * p.ldv + h * D + 8 * sub);
        }
        store_row<FMT, D>(k, p.kr, page, h, at, p.page, p.H_kv, sub, put);
        store_row<FMT, D>(v, p.vr, page, h, at, p.page, p.H_kv, sub, put);
    } else if (live) {
        if (put) {
            k = load_row<FMT>(p.kr, page, h, at, p.page, p.H_kv, sub);
            v = load_row<FMT>(p.vr, page, h, at, p.page, p.H_kv, sub);
        }
        reinterpret_cast<uint4*>(p.k_out)[(int64_t)i * kLanes + sub] = k;
        reinterpret_cast<uint4*>(p.v_out)[(int64_t)i * kLanes + sub] = v;
    }
}

template <bool WRITE>
cudaError_t launch_copy(const KvCopyParams& p, const moe_kv_dims_t& d, cudaStream_t st) {
    const int rows = 256 / (d.D / 8);  // of a CTA
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
