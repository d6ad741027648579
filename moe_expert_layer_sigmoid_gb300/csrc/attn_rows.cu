// Attention of few rows: decode steps and short drafts, 16 rows (tokens x query
// heads of one key/value head) per unit.
//
// Each cached byte is used for 16 rows only, so the kernel is bound by the
// cache's bytes from HBM: the design keeps copies in flight and the work per byte small.
// A CTA is four warps of compute and one that issues TMA copies into a ring of
// stages, two CTAs per SM.  Every warp takes its own quarter of a stage's
// keys through scores, softmax and values with no exchange with the others;
// the warps' (maximum, sum, output) are joined once per unit.
//
// Products run on the warp-level tensor cores, m16n8k16 with bf16 operands:
//   S[16 x 8 keys]  += Q[16 x 16 of D] K^T     K from shared memory by ldmatrix
//   O[16 x 8 of D]  += P[16 x 16 keys] V       P straight from S's registers,
//                                             V by ldmatrix.trans
// Codes are turned into bf16 in registers.  A contraction may run in any
// order, so the k index is permuted to whatever order the unpacking leaves:
// ldmatrix hands lane (g, t) four bytes of key g, which for E4M3 are elements
// 4t .. 4t+3 (bytes 0, 2 and 1, 3 become the two register pairs of a k16
// step), for int4 elements 8t .. 8t+7 (nibble i with nibble i + 4); the query
// fragments are loaded in that order.  For values the transposed load gives
// each lane the same bytes of keys 2t and 2t+1, the pairing the B operand
// needs, and the permutation falls on the output columns.
// The key scales multiply the scores and the value scales the weights, so the
// codes enter the products exactly.
//
// The running maximum is only raised when some score exceeds it by 2^8: a
// warp vote decides, and most tiles need neither the shuffles nor the rescaling
// of the output.  Weights stay below 2^8 and the sums are fp32, so nothing is lost.
#include "attn.cuh"

namespace moe {
namespace {

constexpr int kRowsWarps = 5;              // four of compute, one of copies
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr int kRows = 16;                  // rows of a unit

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// E4M3 codes in bytes 0 and 2 (odd = false) or 1 and 3 of w as two bf16.  The
// code's sign goes to the top and its seven other bits to the exponent's low
// bits and the fraction's top: a bf16 of 2^-120 times the value (subnormals
// included), which one exact product restores.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, bool odd) {
    const uint32_t mag = odd ? (w >> 4) & 0x07F007F0u : (w << 4) & 0x07F007F0u;
    const uint32_t sgn = odd ? w & 0x80008000u : (w << 8) & 0x80008000u;
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(mag | sgn), "r"(0x7B807B80u));
    return r;
}
// Nibbles i and i + 4 of w (two's complement) as two bf16: 128 + (n + 8) by its
// bits, then less 136.
__device__ __forceinline__ uint32_t int4_pair(uint32_t w, int i) {
    uint32_t t, r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(t) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43084308u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(t), "r"(0x3F803F80u), "r"(0xC308C308u));
    return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Shapes of one instantiation.
template <int FMT, int D>
struct RowsShape {
    static constexpr int kRowB = kv_row_bytes(FMT, D);          // bytes of a cache row
    static constexpr int kBoxB = kRowB < 128 ? kRowB : 128;     // of a box's row: the swizzle span
    static constexpr int kHalves = kRowB / kBoxB;
    // keys of a stage: 32 KB of keys and values, 128 keys at most
    static constexpr int kTk = 2 * kRowB * 128 <= 32768 ? 128 : 64;
    static constexpr int kKw = kTk / 4;                         // keys of a warp
    static constexpr int kTileB = kTk * kRowB;                  // bytes of a stage's keys
    static constexpr int kScB = FMT == kKvBf16 ? 0 : kTk * 4;   // and of their scales
    static constexpr int kStages = 98304 / (2 * kTileB) < 8 ? 98304 / (2 * kTileB) : 8;
    static constexpr int kChunks = kRowB / 16;                  // 16-byte chunks of a row
    static constexpr int kEl = D / kChunks;                     // elements of a chunk: 8, 16, 32
    static constexpr int kNt = D / 8;                           // output column tiles
    // shared memory: tiles, scales, the join's buffer, barriers
    static constexpr int kOffSc = kStages * 2 * kTileB;
    static constexpr int kOffJoin = kOffSc + kStages * 2 * kScB;
    static constexpr int kOffMl = kOffJoin + kRows * D * 4;
    static constexpr int kOffBar = kOffMl + 4 * kRows * 8;
    static constexpr int kOffMisc = kOffBar + 2 * kStages * 8;
    static constexpr int kSmem = kOffMisc + 16;
    static_assert(kSmem <= 115712, "two CTAs share an SM's shared memory");
};

// Byte offset of a 16-byte chunk of a row inside a tile as TMA leaves it.
template <int BOXB, int TK>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    constexpr int kPer = BOXB / 16;
    const int half = chunk / kPer, c = chunk % kPer;
    const int x = BOXB == 128 ? row & 7 : BOXB == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    return half * (TK * BOXB) + row * BOXB + ((c ^ x) << 4);
}

// A unit's rows as one lane sees them (rows g and g + 8).
struct RowInfo {
    int64_t q[2];     // row of out / lse: token * H + head, -1 where there is none
    int pos[2];       // last key it sees
    int first[2];     // first key it sees
};

template <int FMT, int D>
__global__ void __launch_bounds__(kRowsThreads, 2)
attn_rows_kernel(const __grid_constant__ AttnParams p) {
    using S = RowsShape<FMT, D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
    auto full = [&](int s) { return smem_u32(bars + s); };
    auto empty = [&](int s) { return smem_u32(bars + S::kStages + s); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc);
    volatile int* last_flag = abort_flag + 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 4);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const Share sh = deal<kRowsThreads>(p, smem);
    if (sh.w0 >= sh.w1) return;
    __syncthreads();
    WsHeader* hdr = p.a.hdr;

    if (warp == 4) {
        // ---------------------------------------------------------------- copies
        const int page = 1 << p.c.page_log2;
        const int box_rows = page < S::kTk ? page : S::kTk;
        const int boxes = S::kTk / box_rows;     // boxes of a tile: one per page, or one
        Unit u = sh.u;
        int64_t unit0 = sh.unit0;
        uint32_t it = 0;
        bool ok = true;
        int ids = 0, ids_next = 0, ids_at = -1;  // 32 page ids from page ids_at on
        do {
            int tile, end;
            unit_share(p, sh, u, unit0, tile, end);
            const int hk = u.hs / p.c.subs;
            const int32_t* row = p.a.pages + (int64_t)u.b * p.a.d.max_pages;
            const int pg0 = u.key0 >> p.c.page_log2;
            const int pg1 = (int)(((int64_t)u.key1 + page - 1) >> p.c.page_log2);  // pages [pg0, pg1) are seen
            auto fetch = [&](int at) {
                const int i = at + lane;
                return i >= pg0 && i < pg1 ? __ldg(row + i) : 0;
            };
            ids_at = -1;
            for (; tile < end; ++tile, ++it) {
                const int s = it % S::kStages;
                const int key = (u.tile0 + tile) * S::kTk;
                const int pg = key >> p.c.page_log2;  // first page of the tile
                if (ids_at < 0 || pg >= ids_at + 32) {
                    const int at = pg & ~31;
                    ids = ids_at >= 0 && at == ids_at + 32 ? ids_next : fetch(at);
                    ids_at = at;
                    ids_next = fetch(at + 32);
                }
                // (a tile's pages lie in one aligned group of 32: at most 8, a power of two)
                const int mine = __shfl_sync(0xFFFFFFFFu, ids, (pg + lane) & 31);
                const bool live = lane < boxes && pg + lane >= pg0 && pg + lane < pg1 &&
                                  key + lane * box_rows < u.key1;
                const uint32_t n_live = __popc(__ballot_sync(0xFFFFFFFFu, live));
                if (!mbar_wait(empty(s), ((it / S::kStages) & 1) ^ 1, abort_flag, hdr)) {
                    ok = false;
                    break;
                }
                const uint32_t box_bytes = box_rows * S::kRowB, sc_bytes = FMT == kKvBf16 ? 0 : box_rows * 4;
                if (lane == 0) mbar_expect_tx(full(s), n_live * 2 * (box_bytes + sc_bytes));
                __syncwarp();
                if (live) {
                    int id = mine;
                    if (id < 0 || id >= p.a.d.n_pages) {
                        record_error(hdr, kErrBadPage);
                        id = 0;
                    }
                    const int at = key & (page - 1);  // 0 unless a page holds several tiles
                    const uint32_t dk = sbase + s * 2 * S::kTileB + lane * box_rows * S::kBoxB;
#pragma unroll
                    for (int h = 0; h < S::kHalves; ++h) {
                        const uint32_t d = dk + h * S::kTk * S::kBoxB;
                        const int x = h * S::kBoxB / (FMT == kKvBf16 ? 2 : 1);
                        tma_load_4d(d, &p.tm_k, x, at, hk, id, full(s));
                        tma_load_4d(d + S::kTileB, &p.tm_v, x, at, hk, id, full(s));
                    }
                    if (FMT != kKvBf16) {
                        const int64_t o = ((int64_t)id * p.a.d.H_kv + hk) * page + at;
                        const uint32_t ds = sbase + S::kOffSc + s * 2 * S::kScB + lane * box_rows * 4;
                        bulk_load(ds, p.a.cache.ks + o, sc_bytes, full(s));
                        bulk_load(ds + S::kScB, p.a.cache.vs + o, sc_bytes, full(s));
                    }
                }
                __syncwarp();
            }
        } while (ok && next_unit(p, sh, u, unit0));
        // after an abort: no copy may be in flight when the CTA ends
        if (!ok)
            for (uint32_t k = it > S::kStages ? it - S::kStages : 0; k < it; ++k)
                mbar_drain(full(k % S::kStages), (k / S::kStages) & 1, hdr);
        return;
    }

    // -------------------------------------------------------------------- compute
    const int g = lane >> 2, t = lane & 3;
    constexpr int kSteps = D / 16;              // k16 steps of a score
    constexpr int kNk = S::kKw / 8;             // key tiles of a warp
    Unit u = sh.u;
    int64_t unit0 = sh.unit0;
    uint32_t it = 0;
    bool ok = true;
    const float sc = p.scale_log2;
    float* join = reinterpret_cast<float*>(smem + S::kOffJoin);
    float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);  // [warp][row]: maximum, sum
    do {
        int tile, end;
        unit_share(p, sh, u, unit0, tile, end);
        if (tile >= end) continue;
        const bool whole = tile == 0 && end == u.tiles;
        // the lane's two rows
        RowInfo ri;
        const int hk = u.hs / p.c.subs, sub = u.hs % p.c.subs;
        const int G = p.a.d.H / p.a.d.H_kv;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i, tok = u.rt * p.c.tq + r / p.c.hg, hd = sub * p.c.hg + r % p.c.hg;
            const bool live = r < p.c.tq * p.c.hg && tok < u.n && hd < G;
            ri.q[i] = live ? (int64_t)(u.tok0 + tok) * p.a.d.H + hk * G + hd : -1;
            ri.pos[i] = live ? u.len - u.n + tok : -1;
            ri.first[i] = p.a.d.window ? max(0, ri.pos[i] - p.a.d.window + 1) : 0;
        }
        // query fragments, in the order that the codes unpack to
        uint32_t qf[kSteps][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t tok = ri.q[i] >= 0 ? ri.q[i] / p.a.d.H : 0, hd = ri.q[i] >= 0 ? ri.q[i] % p.a.d.H : 0;
            const uint16_t* q = p.a.q + tok * p.a.ldq + hd * D;
            const bool live = ri.q[i] >= 0;
#pragma unroll
            for (int c = 0; c < S::kChunks; ++c) {
                if constexpr (FMT == kKvBf16) {
                    // chunk c: k pair (2t, 2t + 1) of half c & 1 of step c / 2
                    qf[c / 2][2 * (c & 1) + i] =
                        live ? __ldg(reinterpret_cast<const uint32_t*>(q + 8 * c + 2 * t)) : 0;
                } else if constexpr (FMT == kKvE4m3) {
                    const uint2 x = live ? __ldg(reinterpret_cast<const uint2*>(q + 16 * c + 4 * t))
                                         : make_uint2(0, 0);
                    qf[c][i] = __byte_perm(x.x, x.y, 0x5410);      // elements 0, 2
                    qf[c][2 + i] = __byte_perm(x.x, x.y, 0x7632);  // elements 1, 3
                } else {
                    const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(q + 32 * c + 8 * t))
                                         : make_uint4(0, 0, 0, 0);
                    qf[2 * c][i] = __byte_perm(x.x, x.z, 0x5410);          // 0, 4
                    qf[2 * c][2 + i] = __byte_perm(x.x, x.z, 0x7632);      // 1, 5
                    qf[2 * c + 1][i] = __byte_perm(x.y, x.w, 0x5410);      // 2, 6
                    qf[2 * c + 1][2 + i] = __byte_perm(x.y, x.w, 0x7632);  // 3, 7
                }
            }
        }
        float o[S::kNt][4];
#pragma unroll
        for (int j = 0; j < S::kNt; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        float m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};
        // keys that every row of the unit sees need no mask
        const int inner0 = p.a.d.window ? max(0, u.len - u.n + min(u.n, u.rt * p.c.tq + p.c.tq) - p.a.d.window) : 0;
        const int inner1 = u.len - u.n + u.rt * p.c.tq + 1;  // [inner0, inner1)

        for (; tile < end; ++tile, ++it) {
            const int s = it % S::kStages;
            // once a wait gave up the flag is set; the warps then run on without waiting, in step
            // with each other, to the end
            if (ok) ok = mbar_wait(full(s), (it / S::kStages) & 1, abort_flag, hdr);
            const int kw0 = warp * S::kKw;                       // the warp's first key in the tile
            const int key = (u.tile0 + tile) * S::kTk + kw0;
            if (key < u.key1 && key + S::kKw > u.key0) {
                const uint32_t kt = sbase + s * 2 * S::kTileB, vt = kt + S::kTileB;
                float sv[kNk][4];
#pragma unroll
                for (int j = 0; j < kNk; ++j) sv[j][0] = sv[j][1] = sv[j][2] = sv[j][3] = 0.0f;
                // scores: chunks of 16 bytes, four per ldmatrix
                if constexpr (FMT == kKvBf16) {
#pragma unroll
                    for (int j = 0; j < kNk; ++j)
#pragma unroll
                        for (int c = 0; c < S::kChunks; c += 4) {
                            uint32_t r[4];
                            ldsm4(r, kt + chunk_at<S::kBoxB, S::kTk>(kw0 + 8 * j + (lane & 7), c + (lane >> 3)));
                            mma16816(sv[j], qf[c / 2], r[0], r[1]);
                            mma16816(sv[j], qf[c / 2 + 1], r[2], r[3]);
                        }
                } else if constexpr (S::kChunks >= 4) {
#pragma unroll
                    for (int j = 0; j < kNk; ++j)
#pragma unroll
                        for (int c = 0; c < S::kChunks; c += 4) {
                            uint32_t r[4];
                            ldsm4(r, kt + chunk_at<S::kBoxB, S::kTk>(kw0 + 8 * j + (lane & 7), c + (lane >> 3)));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (FMT == kKvE4m3) {
                                    mma16816(sv[j], qf[c + i], e4m3_pair(r[i], false), e4m3_pair(r[i], true));
                                } else {
                                    mma16816(sv[j], qf[2 * (c + i)], int4_pair(r[i], 0), int4_pair(r[i], 1));
                                    mma16816(sv[j], qf[2 * (c + i) + 1], int4_pair(r[i], 2), int4_pair(r[i], 3));
                                }
                            }
                        }
                } else {  // two chunks (int4, D = 64): two key tiles per ldmatrix
#pragma unroll
                    for (int j = 0; j < kNk; j += 2) {
                        uint32_t r[4];
                        ldsm4(r, kt + chunk_at<S::kBoxB, S::kTk>(kw0 + 8 * (j + (lane >> 4)) + (lane & 7), (lane >> 3) & 1));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = i & 1;
                            mma16816(sv[j + i / 2], qf[2 * c], int4_pair(r[i], 0), int4_pair(r[i], 1));
                            mma16816(sv[j + i / 2], qf[2 * c + 1], int4_pair(r[i], 2), int4_pair(r[i], 3));
                        }
                    }
                }
                // to the exponent's domain: scale * log2(e), the keys' scales, the masks
                const float* ks = reinterpret_cast<const float*>(smem + S::kOffSc + s * 2 * S::kScB) + kw0;
                const bool inner = key >= inner0 && key + S::kKw <= inner1;
                float mx[2] = {kNoMax, kNoMax};
#pragma unroll
                for (int j = 0; j < kNk; ++j) {
                    float2 f = make_float2(sc, sc);
                    if (FMT != kKvBf16) {
                        f = *reinterpret_cast<const float2*>(ks + 8 * j + 2 * t);
                        f.x *= sc;
                        f.y *= sc;
                    }
                    sv[j][0] *= f.x;
                    sv[j][1] *= f.y;
                    sv[j][2] *= f.x;
                    sv[j][3] *= f.y;
                    if (!inner) {
                        const int k0 = key + 8 * j + 2 * t;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = k0 + (e & 1), i = e >> 1;
                            if (k > ri.pos[i] || k < ri.first[i]) sv[j][e] = -INFINITY;
                        }
                    }
                    mx[0] = fmaxf(mx[0], fmaxf(sv[j][0], sv[j][1]));
                    mx[1] = fmaxf(mx[1], fmaxf(sv[j][2], sv[j][3]));
                }
                if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] + 8.0f || mx[1] > m[1] + 8.0f)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 2));
                        const float mn = fmaxf(m[i], mx[i]), a = ex2(m[i] - mn);
                        m[i] = mn;
                        l[i] *= a;
#pragma unroll
                        for (int j = 0; j < S::kNt; ++j) {
                            o[j][2 * i] *= a;
                            o[j][2 * i + 1] *= a;
                        }
                    }
                }
                // weights; their sum takes them unrounded and without the values' scales
                const float* vs = ks + S::kTk;
                uint32_t pf[kNk / 2][4];
#pragma unroll
                for (int j = 0; j < kNk; ++j) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float p0 = ex2(sv[j][2 * i] - m[i]), p1 = ex2(sv[j][2 * i + 1] - m[i]);
                        l[i] += p0 + p1;
                        if (FMT != kKvBf16) {
                            const float2 f = *reinterpret_cast<const float2*>(vs + 8 * j + 2 * t);
                            p0 *= f.x;
                            p1 *= f.y;
                        }
                        pf[j / 2][2 * (j & 1) + i] = bf16_pair(p0, p1);
                    }
                }
                // keys outside [key0, key1) are nobody's: their slots may hold anything, so the
                // values (and their scales) are cleared, not just weighted with 0
                const bool edge = key < u.key0 || key + S::kKw > u.key1;
                uint32_t vmask[kNk];
                if (edge) {
#pragma unroll
                    for (int j = 0; j < kNk; ++j) {
                        const int k0 = key + 8 * j + 2 * t;
                        vmask[j] = (k0 >= u.key0 && k0 < u.key1 ? 0x0000FFFFu : 0u) |
                                   (k0 + 1 >= u.key0 && k0 + 1 < u.key1 ? 0xFFFF0000u : 0u);
                        if (FMT != kKvBf16) {
                            pf[j / 2][2 * (j & 1)] &= vmask[j];
                            pf[j / 2][2 * (j & 1) + 1] &= vmask[j];
                        }
                    }
                }
#pragma unroll
                for (int kk = 0; kk < kNk / 2; ++kk)
#pragma unroll
                    for (int c = 0; c < S::kChunks; c += 2) {
                        // chunks c and c + 1 of keys 16 kk .. + 7 and + 8 .. + 15
                        uint32_t r[4];
                        ldsm4t(r, vt + chunk_at<S::kBoxB, S::kTk>(kw0 + 16 * kk + (lane & 15), c + (lane >> 4)));
                        if (edge) {
                            r[0] &= vmask[2 * kk];
                            r[1] &= vmask[2 * kk + 1];
                            r[2] &= vmask[2 * kk];
                            r[3] &= vmask[2 * kk + 1];
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t lo = r[2 * i], hi = r[2 * i + 1];
                            if constexpr (FMT == kKvBf16) {
                                mma16816(o[c + i], pf[kk], lo, hi);
                            } else if constexpr (FMT == kKvE4m3) {
                                const int j = 2 * (c + i);
                                mma16816(o[j], pf[kk], e4m3_pair(lo, false), e4m3_pair(hi, false));
                                mma16816(o[j + 1], pf[kk], e4m3_pair(lo, true), e4m3_pair(hi, true));
                            } else {
#pragma unroll
                                for (int n = 0; n < 4; ++n)
                                    mma16816(o[4 * (c + i) + n], pf[kk], int4_pair(lo, n), int4_pair(hi, n));
                            }
                        }
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
        }

        // ------------------------------------------------------ join the four warps
        // (row g: registers 0, 1; row g + 8: 2, 3; the same lanes hold them in every warp)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
            if (t == 0) ml[warp * kRows + g + 8 * i] = make_float2(m[i], l[i]);
        }
        compute_sync();
        float M[2], L[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            M[i] = kNoMax;
            L[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) M[i] = fmaxf(M[i], ml[k * kRows + g + 8 * i].x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = ml[k * kRows + g + 8 * i];
                L[i] += x.y * ex2(x.x - M[i]);
            }
            const float a = ex2(m[i] - M[i]);
#pragma unroll
            for (int j = 0; j < S::kNt; ++j) {
                o[j][2 * i] *= a;
                o[j][2 * i + 1] *= a;
            }
        }
        float4* jb = reinterpret_cast<float4*>(join);
        // 1 -> 0, 3 -> 2, then 2 -> 0: a fixed order
#pragma unroll
        for (int round = 0; round < 3; ++round) {
            const int from = round == 0 ? 1 : round == 1 ? 3 : 2, to = round == 1 ? 2 : 0;
            if (warp == from)
#pragma unroll
                for (int j = 0; j < S::kNt; ++j)
                    jb[j * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
            compute_sync();
            if (warp == to)
#pragma unroll
                for (int j = 0; j < S::kNt; ++j) {
                    const float4 x = jb[j * 32 + lane];
                    o[j][0] += x.x;
                    o[j][1] += x.y;
                    o[j][2] += x.z;
                    o[j][3] += x.w;
                }
            compute_sync();
        }
        bool write = whole;
        if (!whole) {
            // a partial result: slot 0 of a CTA for a unit that an earlier CTA began, else slot 1
            const int c = blockIdx.x, c0 = share_owner(sh.W, sh.R, unit0 + p.c.unit_cost);
            const int c1 = share_owner(sh.W, sh.R, unit0 + p.c.unit_cost + u.tiles - 1);
            constexpr int kPart = kRows * D + 2 * kRows;
            if (warp == 0) {
                float* part = p.part + (int64_t)(2 * c + (c == c0)) * kPart;
                float4* po = reinterpret_cast<float4*>(part);
#pragma unroll
                for (int j = 0; j < S::kNt; ++j)
                    __stcg(po + j * 32 + lane, make_float4(o[j][0], o[j][1], o[j][2], o[j][3]));
                if (t == 0) {
                    float2* pm = reinterpret_cast<float2*>(part + kRows * D);
                    __stcg(pm + g, make_float2(M[0], L[0]));
                    __stcg(pm + g + 8, make_float2(M[1], L[1]));
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const unsigned seen = atomicAdd(p.counters + c0, 1u);
                    const bool last = seen == (unsigned)(c1 - c0);
                    if (last) p.counters[c0] = 0;
                    *last_flag = last;
                }
                __syncwarp();
                write = *last_flag != 0;
                if (write) {
                    __threadfence();
                    M[0] = M[1] = kNoMax;
                    for (int k = c0; k <= c1; ++k) {
                        const float2* pm = reinterpret_cast<const float2*>(
                            p.part + (int64_t)(2 * k + (k == c0)) * kPart + kRows * D);
                        M[0] = fmaxf(M[0], __ldcg(&pm[g].x));
                        M[1] = fmaxf(M[1], __ldcg(&pm[g + 8].x));
                    }
                    L[0] = L[1] = 0.0f;
#pragma unroll
                    for (int j = 0; j < S::kNt; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
                    for (int k = c0; k <= c1; ++k) {
                        const float* q = p.part + (int64_t)(2 * k + (k == c0)) * kPart;
                        const float2* pm = reinterpret_cast<const float2*>(q + kRows * D);
                        const float2 x0 = __ldcg(pm + g), x1 = __ldcg(pm + g + 8);
                        const float a0 = ex2(x0.x - M[0]), a1 = ex2(x1.x - M[1]);
                        L[0] += x0.y * a0;
                        L[1] += x1.y * a1;
                        const float4* po = reinterpret_cast<const float4*>(q);
#pragma unroll
                        for (int j = 0; j < S::kNt; ++j) {
                            const float4 x = __ldcg(po + j * 32 + lane);
                            o[j][0] += x.x * a0;
                            o[j][1] += x.y * a0;
                            o[j][2] += x.z * a1;
                            o[j][3] += x.w * a1;
                        }
                    }
                }
            }
        }
        if (warp == 0 && write) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (ri.q[i] < 0) continue;
                const float inv = L[i] > 0.0f ? 1.0f / L[i] : 0.0f;
                uint16_t* out = p.a.out + ri.q[i] * D;
// of each chunk the lane holds kEl / 4 consecutive columns, over its kEl / 8 tiles
                constexpr int kJ = S::kEl / 8;
#pragma unroll
                for (int c = 0; c < S::kChunks; ++c) {
                    uint32_t x[kJ];
#pragma unroll
                    for (int k = 0; k < kJ; ++k) {  // columns 2k, 2k + 1: tile k % kJ, register k / kJ
                        const int k0 = 2 * k, k1 = 2 * k + 1;
                        x[k] = bf16_pair(o[c * kJ + k0 % kJ][2 * i + k0 / kJ] * inv,
                                         o[c * kJ + k1 % kJ][2 * i + k1 / kJ] * inv);
                    }
                    uint16_t* to = out + c * S::kEl + 2 * kJ * t;
                    if constexpr (kJ == 1) *reinterpret_cast<uint32_t*>(to) = x[0];
                    else if constexpr (kJ == 2) *reinterpret_cast<uint2*>(to) = make_uint2(x[0], x[1]);
                    else *reinterpret_cast<uint4*>(to) = make_uint4(x[0], x[1], x[2], x[3]);
                }
                if (p.a.lse && t == 0)
                    p.a.lse[ri.q[i]] = L[i] > 0.0f ? (M[i] + log2f(L[i])) * kLn2 : -INFINITY;
            }
        }
    } while (next_unit(p, sh, u, unit0));
}

template <int FMT, int D>
cudaError_t launch(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, float* part,
                   unsigned* counters, cudaStream_t st) {
    using S = RowsShape<FMT, D>;
    AttnParams p;
    p.a = a;
    const int G = a.d.H / a.d.H_kv;
    p.c.hg = std::min(G, kRows);
    p.c.tq = kRows / p.c.hg;
    p.c.subs = (G + kRows - 1) / kRows;
    p.c.hs = a.d.H_kv * p.c.subs;
    p.c.tk_log2 = S::kTk == 128 ? 7 : 6;
    p.c.page_log2 = __builtin_ctz(a.d.page);
    p.c.unit_cost = 1;
    p.c.min_share = 2;
    p.c.rows_lo = rows_lo;
    p.c.rows_hi = rows_hi;
    p.part = part;
    p.counters = counters;
    p.scale_log2 = a.scale * kLog2e;
    if (!make_kv_map(&p.tm_k, a.cache.k, a, S::kBoxB, std::min(a.d.page, S::kTk)) ||
        !make_kv_map(&p.tm_v, a.cache.v, a, S::kBoxB, std::min(a.d.page, S::kTk)))
        return cudaErrorInvalidValue;
    const void* kern = reinterpret_cast<const void*>(&attn_rows_kernel<FMT, D>);
    cudaError_t e = ensure_dynamic_smem(kern, S::kSmem);
    if (e != cudaSuccess) return e;
    attn_rows_kernel<FMT, D><<<2 * sm_count(), kRowsThreads, S::kSmem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attn_rows_part_bytes(const moe_kv_dims_t& d) {
    return (size_t)(2 * 2 * sm_count()) * (kRows * d.D + 2 * kRows) * sizeof(float);
}

cudaError_t launch_attn_rows(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, float* part,
                             unsigned* counters, cudaStream_t st) {
    const bool wide = a.d.D == 128;
    switch (a.d.format) {
        case kKvBf16:
            return wide ? launch<kKvBf16, 128>(a, rows_lo, rows_hi, part, counters, st)
                        : launch<kKvBf16, 64>(a, rows_lo, rows_hi, part, counters, st);
        case kKvE4m3:
            return wide ? launch<kKvE4m3, 128>(a, rows_lo, rows_hi, part, counters, st)
                        : launch<kKvE4m3, 64>(a, rows_lo, rows_hi, part, counters, st);
        case kKvInt4:
            return wide ? launch<kKvInt4, 128>(a, rows_lo, rows_hi, part, counters, st)
                        : launch<kKvInt4, 64>(a, rows_lo, rows_hi, part, counters, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
