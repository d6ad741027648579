// Rotary positions: the table of cosines and sines, and rows turned by it as they
// are read, on their way to a buffer or into the paged cache.
//
// Turning moves bytes: a row's elements once in and once out, and one table row per token. The
// bound is DRAM bandwidth, and for a few tokens the launch and two dependent loads (position, table
// row).  Rows come through shared memory, each lane copying what it will itself turn, three rows ahead: 65537 tokens
// of 32 + 2 * 8 heads of 128 into a bf16 cache take 238 us, a copy's bandwidth (loads in registers, at most two rows
// of a lane on the way: 302).  D / 16 lanes take a row, each two pieces of 16 bytes: in the half layout piece j and
// piece j + rot / 16, so that both elements of a pair meet in one lane; in the other layout a piece holds
// whole pairs.  A lane's eight angles are the same for every head of a token, so a group of lanes keeps
// them in registers and walks a token's heads: its queries, then its keys, then its values.
#include <cmath>

#include "kv_codes.cuh"
#include "rope.cuh"

namespace moe {
namespace {

struct RopeParams {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv, ldo;  // elements from token to token
    uint16_t* out;
    const int32_t *pos, *slots;
    moe_rope_t rope;
    KvRows kr, vr;
    WsHeader* hdr;
    int T, H, H_kv, page_log2, n_slots;
    int groups;  // groups of lanes that share a token's heads
};

__device__ __forceinline__ void unpack(uint4 x, float (&f)[8]) {
    f[0] = bf16_lo(x.x); f[1] = bf16_hi(x.x); f[2] = bf16_lo(x.y); f[3] = bf16_hi(x.y);
    f[4] = bf16_lo(x.z); f[5] = bf16_hi(x.z); f[6] = bf16_lo(x.w); f[7] = bf16_hi(x.w);
}
__device__ __forceinline__ uint4 packed(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void load4(const float* p, float* f) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// One pair turned.  Products and sums are rounded one by one, so that any program that takes the
// same steps in fp32 gets the same codes: a fused product would move the last bit.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = u;
}

// A lane's two pieces of a head: normalised with weights w (where norm), and turned (where live).
template <int D, bool PAIRS>
__device__ __forceinline__ void turn_row(float (&f)[2][8], bool norm, float eps, const float (&w)[2][8],
                                         const bool (&live)[2], const float (&c)[8], const float (&s)[8], unsigned mask) {
    constexpr int kLanes = D / 16;
    if (norm) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += f[j][i] * f[j][i];
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
        const float r = rsqrtf(sum * (1.0f / D) + eps);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] = f[j][i] * r * w[j][i];
    }
    if (PAIRS) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (live[j]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) turn(f[j][2 * i], f[j][2 * i + 1], c[4 * j + i], s[4 * j + i]);
            }
    } else if (live[0]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(f[0][i], f[1][i], c[i], s[i]);
    }
}

// A lane's two pieces of a key, not yet rounded, as a row of the cache.
template <int FMT, int D>
__device__ __forceinline__ void store_key(const float (&f)[2][8], uint8_t* row, float* scale, const int (&at)[2],
                                          bool first, unsigned mask) {
    constexpr int kLanes = D / 16;
    if (FMT == kKvBf16) {
#pragma unroll
        for (int j = 0; j < 2; ++j) reinterpret_cast<uint4*>(row)[at[j]] = packed(f[j]);
        return;
    }
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[j][i]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
    const float s = __fdiv_rn(m, FMT == kKvE4m3 ? 448.0f : 7.0f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float y[8];
        // (keys are a small share of the rows: a division each costs nothing that shows)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = s > 0.0f ? __fdiv_rn(f[j][i], s) : 0.0f;
        // The recipe's clamp: a turned key may be so small that its scale is a few units of 2^-149, rounded by up to half of
        // one, and quotients reach 10.  A normal scale needs none.  (NaN stays; E4M3's conversion saturates by itself.)
        if (FMT == kKvInt4 && s < 0x1p-126f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] > 7.0f ? 7.0f : y[i] < -8.0f ? -8.0f : y[i];
        }
        const uint2 c = codes_of<FMT>(y);
        if (FMT == kKvE4m3) reinterpret_cast<uint2*>(row)[at[j]] = c;
        else reinterpret_cast<uint32_t*>(row)[at[j]] = c.x;
    }
    if (first) *scale = s;
}

// FMT < 0: rows of q only, no cache.
template <int FMT, int D, bool PAIRS>
__global__ void __launch_bounds__(256, 3) rope_kernel(const RopeParams p) {
    constexpr int kLanes = D / 16, kGroups = 256 / kLanes;  // groups of a CTA
    constexpr int kAhead = 3;                               // rows on the way
    __shared__ uint4 ring[kAhead + 1][2][256];
    const int sub = threadIdx.x % kLanes;
    const unsigned mask = ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
    const int64_t g = (int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes;
    const int t = (int)(g / p.groups), first = (int)(g - (int64_t)t * p.groups);
    if (t >= p.T) return;
    // this lane's pieces of a row, and whether they are turned
    // (neighbouring lanes' pieces lie together in either case: their loads and stores are whole sectors)
    const int half = p.rope.rot / 16;  // pieces of half of what is turned
    int at[2];
    bool live[2];
    if (PAIRS) {
        at[0] = sub;
        at[1] = sub + kLanes;
        live[0] = at[0] < 2 * half;
        live[1] = at[1] < 2 * half;
    } else {
        live[0] = live[1] = sub < half;
        at[0] = live[0] ? sub : sub + half;
        at[1] = live[0] ? sub + half : sub + kLanes;
    }
    // The group's rows, queries then keys then values, come through shared memory, each lane its own pieces: the first
    // of them are on the way while the position and its angles are fetched.
    const int k0 = p.H, v0 = FMT < 0 ? p.H : p.H + p.H_kv, rows = FMT < 0 ? p.H : p.H + 2 * p.H_kv;
    auto fetch = [&](int i) {
        const int h = first + i * p.groups;
        if (h < rows) {
            const bool value = h >= v0;  // (in the order of store_row)
            const uint4* row = reinterpret_cast<const uint4*>(
                h < k0 ? p.q + t * p.ldq + (int64_t)h * D
                       : value ? p.v + t * p.ldv + (int64_t)(h - v0) * D : p.k + t * p.ldk + (int64_t)(h - k0) * D);
            copy_async<16>(&ring[i % (kAhead + 1)][0][threadIdx.x], row + (value ? sub : at[0]));
            copy_async<16>(&ring[i % (kAhead + 1)][1][threadIdx.x], row + (value ? sub + kLanes : at[1]));
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i);

    const int pos = __ldg(p.pos + t);
    int slot = FMT < 0 ? -1 : __ldg(p.slots + t);
    bool skip = pos < 0;
    if (pos >= p.rope.n_pos) {
        if (first == 0 && sub == 0) record_error(p.hdr, kErrBadPos);
        skip = true;
    }
    if (FMT >= 0 && slot >= p.n_slots) {
        if (!skip && first == 0 && sub == 0) record_error(p.hdr, kErrBadSlot);
        slot = -1;
    }
    if (skip) {
        copy_wait<0>();
        return;
    }
    float c[8], s[8];
    {
        const float* row = p.rope.table + (int64_t)pos * p.rope.rot;
        const float* other = row + p.rope.rot / 2;
        if (PAIRS) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (live[j]) {
                    load4(row + 4 * at[j], c + 4 * j);
                    load4(other + 4 * at[j], s + 4 * j);
                }
        } else if (live[0]) {
            load8(row + 8 * sub, c);
            load8(other + 8 * sub, s);
        }
        if (p.rope.flags & MOE_ROPE_INVERSE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = -s[i];
        }
    }
    const float eps = p.rope.eps;
    float w[2][8];
    auto load_weights = [&](const float* norm) {
        if (norm) {
            load8(norm + 8 * at[0], w[0]);
            load8(norm + 8 * at[1], w[1]);
        }
    };
    load_weights(first < k0 ? p.rope.q_norm : p.rope.k_norm);
    const int page = slot >> p.page_log2, in_page = slot & ((1 << p.page_log2) - 1);
    auto scale_at = [&](int head) { return (((int64_t)page * p.H_kv + head) << p.page_log2) + in_page; };
    uint16_t* out = p.out + t * p.ldo;

    int i = 0;
    for (int h = first; h < rows; h += p.groups, ++i) {
        fetch(i + kAhead);
        copy_wait<kAhead>();
        const uint4 x[2] = {ring[i % (kAhead + 1)][0][threadIdx.x], ring[i % (kAhead + 1)][1][threadIdx.x]};
        if (h < k0 || h < v0) {
            if (FMT >= 0 && h >= k0) {
                if (slot < 0) break;
                if (h - p.groups < k0 && h != first) load_weights(p.rope.k_norm);
            }
            float f[2][8];
            unpack(x[0], f[0]);
            unpack(x[1], f[1]);
            turn_row<D, PAIRS>(f, (h < k0 ? p.rope.q_norm : p.rope.k_norm) != nullptr, eps, w, live, c, s, mask);
            if (h < k0) {
                uint4* o = reinterpret_cast<uint4*>(out + (int64_t)h * D);
                o[at[0]] = packed(f[0]);
                o[at[1]] = packed(f[1]);
            } else if constexpr (FMT >= 0) {
                store_key<FMT, D>(f, p.kr.q + p.kr.offset(page, h - k0, in_page), p.kr.s + scale_at(h - k0), at, sub == 0,
                                  mask);
            }
        } else if constexpr (FMT >= 0) {
            if (slot < 0) break;
            float m = 0.0f;
            if (FMT != kKvBf16) {
                uint32_t a = absmax_pair(x[0], x[1]);
                a = max_bf16x2(a, __byte_perm(a, a, 0x1032));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) a = max_bf16x2(a, __shfl_xor_sync(mask, a, o));
                m = fmaxf(bf16_lo(a), 0.0f);  // (a row of NaN alone has none)
            }
            store_row<FMT, D>(x, m, p.vr.q + p.vr.offset(page, h - v0, in_page), p.vr.s + scale_at(h - v0), sub);
        }
    }
    copy_wait<0>();
}

// Groups of lanes per token: one for each row while that leaves SMs without work, else as many as
// share a warp, so that a token's angles are loaded once or twice.
int groups_of(int T, int rows, int D) {
    const int warp = 32 / (D / 16);
    int64_t g = rows;
    while (g > warp && (int64_t)T * g * (D / 16) > (int64_t)sm_count() * 2048) g = (g + 1) / 2;
    return (int)g;
}

template <int FMT>
cudaError_t launch_fmt(const RopeParams& p, int D, cudaStream_t st) {
    const int kGroups = 256 / (D / 16);
    const unsigned grid = (unsigned)(((int64_t)p.T * p.groups + kGroups - 1) / kGroups);
    const bool pairs = p.rope.flags & MOE_ROPE_PAIRS;
    if (D == 128) {
        if (pairs) rope_kernel<FMT, 128, true><<<grid, 256, 0, st>>>(p);
        else rope_kernel<FMT, 128, false><<<grid, 256, 0, st>>>(p);
    } else {
        if (pairs) rope_kernel<FMT, 64, true><<<grid, 256, 0, st>>>(p);
        else rope_kernel<FMT, 64, false><<<grid, 256, 0, st>>>(p);
    }
    return cudaGetLastError();
}

// ---------------------------------------------------------------- the table
constexpr int kMaxPairs = 128;

struct TableParams {
    float* table;
    uint64_t turn[kMaxPairs];  // each pair's turns per position, in 2^-64
    int64_t pos0, n_pos;
    int half;
    float magnitude;
};

// sin(pi x) and cos(pi x) for |x| <= 1/4 by their Taylor series in fp32: the first term left out is below 2^-28, and the
// leading product takes pi in two parts, so that what is left is the roundings of the last two steps.
__device__ __forceinline__ void sincos_pi(float x, float& s, float& c) {
    const float y = x * x;
    float p = fmaf(y, 8.2145886611e-2f, -5.9926452932e-1f);   // pi^9 / 9!, pi^7 / 7!
    p = fmaf(y, p, 2.5501640399f);                            // pi^5 / 5!
    p = fmaf(y, p, -5.1677127800f);                           // pi^3 / 3!
    s = fmaf(x, 3.1415927410f, x * fmaf(y, p, -8.7422780126e-8f));
    float q = fmaf(y, -2.5806891390e-2f, 2.3533063036e-1f);   // pi^10 / 10!, pi^8 / 8!
    q = fmaf(y, q, -1.3352627689f);                           // pi^6 / 6!
    q = fmaf(y, q, 4.0587121264f);                            // pi^4 / 4!
    q = fmaf(y, q, -4.9348022005f);                           // pi^2 / 2
    c = fmaf(y, q, 1.0f);
}

// Angles in turns, as 64-bit fractions: the product with a position drops whole turns by itself and
// is off by position * 2^-65 of one.  What is left is taken to the nearest quarter turn, so that
// the rest, at most an eighth, keeps 24 bits as a float.  A thread makes four cosines and four sines of a few rows:
// 131072 positions of 128 15.3 us, 4.4 TB/s of stores.  Neither the stores nor the arithmetic (issue 56%, ALU 52%) bound it, but the
// pairs' turns, which each lane takes out of the parameters at a place of its own: the unit that serves such loads one address
// after another is busy for 65% of the time, and most waits are for it.
constexpr int kTableRows = 4;  // rows of a thread
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableParams p) {
    const int j = threadIdx.x * 4;
    uint64_t a[4], step[4];
    int64_t r = ((int64_t)blockIdx.x * kTableRows) * blockDim.y + threadIdx.y;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        a[n] = p.turn[j + n] * (uint64_t)(p.pos0 + r);
        step[n] = p.turn[j + n] * (uint64_t)blockDim.y;
    }
#pragma unroll
    for (int k = 0; k < kTableRows; ++k, r += blockDim.y) {
        if (r >= p.n_pos) return;
        float c[4], s[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            // the high word holds all that fp32 can, the rest of an eighth of a turn in 29 bits
            const uint32_t high = (uint32_t)(a[n] >> 32), quarter = (high + (1u << 29)) >> 30;
            const float x = (float)(int32_t)(high - (quarter << 30)) * 0x1p-31f;  // half turns
            float sx, cx;
            sincos_pi(x, sx, cx);
            const float sv = quarter & 1 ? cx : sx, cv = quarter & 1 ? sx : cx;
            s[n] = p.magnitude * (quarter & 2 ? -sv : sv);
            c[n] = p.magnitude * ((quarter + 1) & 2 ? -cv : cv);
            a[n] += step[n];
        }
        float* row = p.table + r * 2 * p.half + j;
        *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4*>(row + p.half) = make_float4(s[0], s[1], s[2], s[3]);
    }
}

}  // namespace

double rope_frequency(const moe_rope_config_t& g, int i) {
    const double kTurn = 6.283185307179586476925;
    const double f = std::pow(g.base, -2.0 * i / g.rot);
    double scaled = 0.0;  // share of f / factor
    if (g.scaling == MOE_ROPE_LINEAR) scaled = 1.0;
    else if (g.scaling == MOE_ROPE_RAMP) {
        auto pair = [&](double t) { return g.rot * std::log(g.orig_len / (kTurn * t)) / (2.0 * std::log(g.base)); };
        const double a = std::fmax(std::floor(pair(g.hi)), 0.0), b = std::fmin(std::ceil(pair(g.lo)), g.rot - 1.0);
        scaled = std::fmin(std::fmax((i - a) / std::fmax(b - a, 0.001), 0.0), 1.0);
    } else if (g.scaling == MOE_ROPE_BAND) {
        scaled = 1.0 - std::fmin(std::fmax((g.orig_len * f / kTurn - g.lo) / (g.hi - g.lo), 0.0), 1.0);
    }
    return scaled == 0.0 ? f : (1.0 - scaled) * f + scaled * (f / g.factor);
}

cudaError_t launch_rope_table(const moe_rope_config_t& g, int32_t pos0, int32_t n_pos, float* table,
                              cudaStream_t st) {
    TableParams p{};
    p.table = table;
    p.pos0 = pos0;
    p.n_pos = n_pos;
    p.half = g.rot / 2;
    p.magnitude = (float)g.magnitude;
    for (int i = 0; i < p.half; ++i)  // (at most 1 / 2 pi of a turn: it fits)
        p.turn[i] = (uint64_t)std::nearbyint(std::ldexp(rope_frequency(g, i) / 6.283185307179586476925, 64));
    const dim3 threads(p.half / 4, 256 / (p.half / 4));
    const int rows = kTableRows * threads.y;  // of a CTA
    rope_table_kernel<<<(unsigned)(((int64_t)n_pos + rows - 1) / rows), threads, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rope_rows(const uint16_t* x, int64_t ldx, const int32_t* pos, int32_t T, int32_t H, int32_t D,
                             const moe_rope_t& rope, uint16_t* out, int64_t ldo, WsHeader* hdr, cudaStream_t st) {
    RopeParams p{};
    p.q = x;
    p.ldq = ldx;
    p.out = out;
    p.ldo = ldo;
    p.pos = pos;
    p.rope = rope;
    p.hdr = hdr;
    p.T = T;
    p.H = H;
    p.groups = groups_of(T, H, D);
    return launch_fmt<-1>(p, D, st);
}

cudaError_t launch_rope_kv_write(const RopeWriteArgs& a, cudaStream_t st) {
    RopeParams p{};
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.ldq = a.ldq;
    p.ldk = a.ldk;
    p.ldv = a.ldv;
    p.ldo = a.ldo;
    p.out = a.out;
    p.pos = a.pos;
    p.slots = a.slots;
    p.rope = a.rope;
    p.kr = kv_rows(a.cache, true);
    p.vr = kv_rows(a.cache, false);
    p.hdr = a.hdr;
    p.T = a.d.T;
    p.H = a.d.H;
    p.H_kv = a.d.H_kv;
    p.page_log2 = __builtin_ctz(a.d.page);
    p.n_slots = a.d.n_pages * a.d.page;
    p.groups = groups_of(p.T, p.H + 2 * p.H_kv, a.d.D);
    switch (a.d.format) {
        case kKvBf16: return launch_fmt<kKvBf16>(p, a.d.D, st);
        case kKvE4m3: return launch_fmt<kKvE4m3>(p, a.d.D, st);
        case kKvInt4: return launch_fmt<kKvInt4>(p, a.d.D, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
