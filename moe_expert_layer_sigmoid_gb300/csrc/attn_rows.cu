// Attention of few rows: decode steps and short drafts, 8 or 16 rows (tokens x
// query heads of one key/value head) per unit.
//
// Each cached byte is used for few rows only, so the floor is the cache's bytes
// from HBM; what stands in the way is the work per byte in the SM, so the design keeps
// copies in flight and that work small.  A CTA is four warps of compute and one that issues
// TMA copies into a ring of stages, three CTAs per SM (two with 16 rows, four with int4 rows of 64).  Every
// warp takes its own quarter of a stage's keys through scores, softmax and values
// with no exchange with the others; the warps' (maximum, sum, output) are joined once
// per unit.
//
// Products run on the warp-level tensor cores, m16n8k16, keys (and output columns) along
// the 16 and the few rows along the 8, so that no product is spent on rows that are not there:
//   S^T[16 keys x 8 rows] += K[16 keys x 16 of D] Q^T      K by ldmatrix
//   O^T[16 of D x 8 rows] += V^T[16 of D x 16 keys] P^T    V by ldmatrix.trans, P^T from S^T's
//                                                          registers by movmatrix
// The key scales multiply the scores and the value scales the weights, so codes enter the
// products exactly.  They are turned into operands in registers; a contraction may run in
// any order, so the k index (and for values the order of the output columns) is
// permuted to whatever the unpacking leaves:
//   E4M3 keys: f16 by the conversion of two codes; the query row is scaled by the power of two
//     that puts its largest element into [2^14, 2^15), where f16 holds every bf16 from 2^-31 of it up and
//     is off by 2^-39 of it at most below (its last bit is 2^-24).
//   int4 keys: the nibble n + 8 alone is the f16 subnormal (n + 8) 2^-24 (2^-20 four bits up):
//     one mask each, the queries take the other scale and the accumulators start at -8 sum q.  Half of the
//     query's elements are held at 2^-4 of the others, so the two limits are 2^-27 and 2^-35; and the sums
//     round by |q| (|n| + 16) instead of |q n|, which bf16 weights hide (their rounding is 2^-8) unless one
//     element outweighs the others by a thousand and meets codes of 0.
//   E4M3 values: the two codes of a column pair side by side, then by way of f16 and fp32 to bf16, exact at
//     every step (moving the bits takes fewer instructions, but all on one pipe).
//   int4 values: 128 + (n + 8) by its bits, less 136.
// Weights are bf16: they need its range.
//
// The running maximum is only raised when some score exceeds it by 2^8: a warp vote decides, and
// most tiles need neither the shuffles nor the rescaling of the output.  Weights stay below 2^8
// and the sums are fp32, so nothing is lost.
//
// Measured (GB300, whole call): 191 thousand E4M3 keys in three sequences, 8 key/value heads of 128, 77 us, 5.3 TB/s,
// 78% of a copy's bandwidth (issue slots 46%, ALU 46%).  128 sequences of up to 8190 int4 keys, D = 64,
// 36 us: issue-bound (54%, ALU 49%).  29 sequences of 71 to 4009 bf16 keys 31 us, 3.9 TB/s: latency of
// dealing, first loads and joins (issue 22%).  The forms of 16 rows and D = 128 spill (E4M3 64 bytes stored and
// 96 loaded, int4 124 and 144, bf16 12 and 12 at 168 registers), the others do not.
#include "attn.cuh"

namespace moe {
namespace {

constexpr int kRowsWarps = 5;              // four of compute, one of copies
constexpr int kRowsThreads = kRowsWarps * 32;

template <bool F16>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, const uint32_t* b) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
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

// An 8 x 8 matrix of 16-bit elements across the warp (lane (g, t): row g, columns 2t, 2t + 1), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Two E4M3 codes to two f16.
__device__ __forceinline__ uint32_t e4m3_f16(uint16_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
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
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two E4M3 codes to two bf16.
__device__ __forceinline__ uint32_t e4m3_bf16(uint16_t w) {
    const uint32_t h = e4m3_f16(w);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return bf16_pair(f.x, f.y);
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 .. 127

// Shapes of one instantiation; R8: blocks of eight rows.
template <int FMT, int D, int R8>
struct RowsShape {
    static constexpr int kRows = 8 * R8;
    // per SM, by registers; a fourth for narrow int4 heads, the work per byte of which is the largest (128
    // sequences: int4 39.4 -> 36.8 us with four, E4M3 41.2 -> 43.3, bf16 54 either way)
    static constexpr int kCtas = R8 == 2 ? 2 : FMT == kKvInt4 && D == 64 ? 4 : 3;
    static constexpr int kRowB = kv_row_bytes(FMT, D);          // bytes of a cache row
    static constexpr int kBoxB = kRowB < 128 ? kRowB : 128;     // of a box's row: the swizzle span
    static constexpr int kHalves = kRowB / kBoxB;
    static constexpr int kTk = FMT == kKvBf16 ? 64 : 128;       // keys of a stage
    static constexpr int kKm = kTk / 64;                        // blocks of 16 keys of a warp
    static constexpr int kTileB = kTk * kRowB;                  // bytes of a stage's keys
    static constexpr int kScB = FMT == kKvBf16 ? 0 : kTk * 4;   // and of their scales
    static constexpr int kRing = kCtas == 4 ? 40960 : kCtas == 3 ? 65536 : 98304;
    static constexpr int kStages = kRing / (2 * kTileB) < 8 ? kRing / (2 * kTileB) : 8;
    static constexpr int kChunks = kRowB / 16;                  // 16-byte chunks of a row
    static constexpr int kDm = D / 16;                          // blocks of 16 output columns
    static constexpr int kLd = D + 4;                           // row stride of the join's buffer
    // shared memory: tiles, scales, the join's buffer, barriers
    static constexpr int kOffSc = kStages * 2 * kTileB;
    static constexpr int kOffJoin = kOffSc + kStages * 2 * kScB;
    static constexpr int kOffMl = kOffJoin + kRows * kLd * 4;
    static constexpr int kOffBar = kOffMl + 4 * kRows * 8;
    static constexpr int kOffMisc = kOffBar + 2 * kStages * 8;
    static constexpr int kSmem = kOffMisc + 16 + sizeof(Share);
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM share its shared memory");
    static_assert(kSmem >= deal_bytes(kRowsThreads), "scratch");
    static constexpr int kPart = kRows * D + 2 * kRows;         // floats of a partial result
};

// Byte offset of a 16-byte chunk of a row inside a tile as TMA leaves it.
template <int BOXB, int TK>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    constexpr int kPer = BOXB / 16;
    const int half = chunk / kPer, c = chunk % kPer;
    const int x = BOXB == 128 ? row & 7 : BOXB == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    return half * (TK * BOXB) + row * BOXB + ((c ^ x) << 4);
}

// The output column of a lane's accumulators (block m, upper half or not).
template <int FMT>
__device__ __forceinline__ int out_col(int m, int half, int g) {
    if (FMT == kKvBf16) return 16 * m + 8 * half + g;
    if (FMT == kKvE4m3) return 16 * m + 2 * g + half;
    return 32 * (m / 2) + 4 * g + 2 * (m & 1) + half;
}

template <int FMT, int D, int R8>
__global__ void __launch_bounds__(kRowsThreads, RowsShape<FMT, D, R8>::kCtas)
attn_rows_kernel(const __grid_constant__ AttnParams p) {
    using S = RowsShape<FMT, D, R8>;
    constexpr int kRows = S::kRows;
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
    const uint32_t withheld = withheld_stage(p.a.hdr);
    // (the share stays in shared memory: it is looked at once per unit, and registers are short)
    Share& sh = *reinterpret_cast<Share*>(smem + S::kOffMisc + 16);
    {
        const Share mine = deal<kRowsThreads>(p, smem);
        if (mine.w0 >= mine.w1) {
            pdl_wait();
            return;
        }
        if (threadIdx.x == 0) sh = mine;
    }
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
            const int pg1 = tiles_until(u.key1, p.c.page_log2);  // pages [pg0, pg1) are seen
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
                if (!warp_wait(empty(s), ((it / S::kStages) & 1) ^ 1, abort_flag, hdr)) {
                    ok = false;
                    break;
                }
                const uint32_t box_bytes = box_rows * S::kRowB, sc_bytes = FMT == kKvBf16 ? 0 : box_rows * 4;
                if (lane == 0) mbar_expect_tx(full(s), n_live * 2 * (box_bytes + sc_bytes));
                __syncwarp();
                if (live && it + 1 != withheld) {
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
    const int g = lane >> 2, t = lane & 3, tid = threadIdx.x;
    constexpr int kSteps = D / 16;              // k16 steps of a score
    constexpr int kDm = S::kDm, kKm = S::kKm;
    Unit u = sh.u;
    int64_t unit0 = sh.unit0;
    uint32_t it = 0;
    bool ok = true;
    const float sc = p.scale_log2;
    float* join = reinterpret_cast<float*>(smem + S::kOffJoin);
    float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);  // [warp][row]: maximum, sum
    const int G = p.a.d.H / p.a.d.H_kv;
    do {
        int tile, end;
        unit_share(p, sh, u, unit0, tile, end);
        if (tile >= end) continue;
        const bool whole = tile == 0 && end == u.tiles;
        const int hk = u.hs / p.c.subs, sub = u.hs % p.c.subs;
        // row r of the unit: its token in the sequence and its query head, -1 where there is none
        auto token_of = [&](int r) {
            const int tok = u.rt * p.c.tq + r / p.c.hg;
            return r < p.c.tq * p.c.hg && tok < u.n && sub * p.c.hg + r % p.c.hg < G ? tok : -1;
        };
        auto head_of = [&](int r) { return hk * G + sub * p.c.hg + r % p.c.hg; };
        // query fragments (row g of each block), in the order that the codes unpack to
        uint32_t qf[kSteps][R8][2];
        float rs[R8][2], off[R8][2];  // of rows 2t, 2t + 1 of a block: factor and start of the scores
#pragma unroll
        for (int n = 0; n < R8; ++n) {
            const int tok = token_of(8 * n + g);
            const bool live = tok >= 0;
            const uint16_t* q = p.a.q + (int64_t)(u.tok0 + max(tok, 0)) * p.a.ldq + head_of(8 * n + g) * D;
            rs[n][0] = rs[n][1] = sc;
            off[n][0] = off[n][1] = 0.0f;
            if constexpr (FMT == kKvBf16) {
#pragma unroll
                for (int c = 0; c < S::kChunks; ++c)
                    qf[c / 2][n][c & 1] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + 8 * c + 2 * t)) : 0;
            } else {
                // elements kPer t .. of each chunk of 4 kPer
                constexpr int kPer = FMT == kKvE4m3 ? 4 : 8;
                uint32_t x[S::kChunks][kPer / 2];
#pragma unroll
                for (int c = 0; c < S::kChunks; ++c) {
                    if constexpr (FMT == kKvE4m3) {
                        const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(q + 16 * c + 4 * t)) : make_uint2(0, 0);
                        x[c][0] = v.x, x[c][1] = v.y;
                    } else {
                        const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(q + 32 * c + 8 * t)) : make_uint4(0, 0, 0, 0);
                        x[c][0] = v.x, x[c][1] = v.y, x[c][2] = v.z, x[c][3] = v.w;
                    }
                }
                uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
                for (int c = 0; c < S::kChunks; ++c)
#pragma unroll
                    for (int k = 0; k < kPer / 2; ++k)
                        top = max(top, max(x[c][k] & 0x7FFFu, (x[c][k] >> 16) & 0x7FFFu));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int e = min(126, 14 - ((int)(top >> 7) - 127));  // the largest comes to [2^14, 2^15)
                const float up = pow2(e);
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < S::kChunks; ++c) {
                    if constexpr (FMT == kKvE4m3) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            qf[c][n][k] = f16_pair(bf16_lo(x[c][k]) * up, bf16_hi(x[c][k]) * up);
                    } else {
                        float f[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            f[2 * k] = bf16_lo(x[c][k]) * up;
                            f[2 * k + 1] = bf16_hi(x[c][k]) * up;
                        }
                        // nibbles 0, 4 and 2, 6 are read in bits 0-3 of their words, 1, 5 and 3, 7 in bits
                        // 4-7, where they count 16 times as much
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float d = k & 1 ? 0.0625f : 1.0f;
                            const uint32_t h = f16_pair(f[k] * d, f[k + 4] * d);
                            qf[2 * c + k / 2][n][k & 1] = h;
                            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h));
                            sum += (b.x + b.y) / d;
                        }
                    }
                }
                if constexpr (FMT == kKvInt4) {
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                }
                const float down = sc * pow2(max(-126, -e));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    rs[n][i] = __shfl_sync(0xFFFFFFFFu, down, 4 * (2 * t + i)) * (FMT == kKvInt4 ? 16777216.0f : 1.0f);
                    if constexpr (FMT == kKvInt4)
                        off[n][i] = __shfl_sync(0xFFFFFFFFu, sum, 4 * (2 * t + i)) * (-8.0f / 16777216.0f);
                }
            }
        }
        // rows 2t, 2t + 1 of each block: the keys they see
        int pos[R8][2], first[R8][2];
#pragma unroll
        for (int n = 0; n < R8; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = token_of(8 * n + 2 * t + i);
                pos[n][i] = tok >= 0 ? u.len - u.n + tok : -1;
                first[n][i] = first_key(pos[n][i], p.a.d.window);
            }
        float o[kDm][R8][4];
#pragma unroll
        for (int j = 0; j < kDm; ++j)
#pragma unroll
            for (int n = 0; n < R8; ++n) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.0f;
        float m[R8][2], l[R8][2];
#pragma unroll
        for (int n = 0; n < R8; ++n) {
            m[n][0] = m[n][1] = kNoMax;
            l[n][0] = l[n][1] = 0.0f;
        }
        // keys that every row of the unit sees need no mask
        const int inner0 = first_key(u.len - u.n + min(u.n, u.rt * p.c.tq + p.c.tq) - 1, p.a.d.window);
        const int inner1 = max(0, u.len - u.n + u.rt * p.c.tq + 1);  // [inner0, inner1)

        for (; tile < end; ++tile, ++it) {
            const int s = it % S::kStages;
            // once a wait gave up the flag is set; the warps then run on without waiting, in step
            // with each other, to the end.  They hand no stage back: one whose copies never came must
            // not be armed a second time (its barrier's phase is still open), so the copies stop too
            if (ok) ok = mbar_wait(full(s), (it / S::kStages) & 1, abort_flag, hdr);
            const int kw0 = warp * 16 * kKm;                       // the warp's first key in the tile
            const int key = (u.tile0 + tile) * S::kTk + kw0;
            if (tile_meets(key, 16 * kKm, u.key0, u.key1)) {
                const uint32_t kt = sbase + s * 2 * S::kTileB, vt = kt + S::kTileB;
                float sv[kKm][R8][4];
#pragma unroll
                for (int km = 0; km < kKm; ++km)
#pragma unroll
                    for (int n = 0; n < R8; ++n) {
                        sv[km][n][0] = sv[km][n][2] = off[n][0];
                        sv[km][n][1] = sv[km][n][3] = off[n][1];
                    }
#pragma unroll
                for (int km = 0; km < kKm; ++km)
#pragma unroll
                    for (int c = 0; c < S::kChunks; c += 2) {
                        // r: keys 0-7 and 8-15 of chunk c, then of chunk c + 1
                        uint32_t r[4];
                        ldsm4(r, kt + chunk_at<S::kBoxB, S::kTk>(kw0 + 16 * km + (lane & 15), c + (lane >> 4)));
                        if constexpr (FMT == kKvBf16) {
#pragma unroll
                            for (int n = 0; n < R8; ++n) mma16816<false>(sv[km][n], r, qf[c / 2][n]);
                        } else if constexpr (FMT == kKvE4m3) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t x = r[2 * i], y = r[2 * i + 1];
                                const uint32_t a[4] = {e4m3_f16((uint16_t)x), e4m3_f16((uint16_t)y),
                                                       e4m3_f16((uint16_t)(x >> 16)), e4m3_f16((uint16_t)(y >> 16))};
#pragma unroll
                                for (int n = 0; n < R8; ++n) mma16816<true>(sv[km][n], a, qf[c + i][n]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t x = r[2 * i] ^ 0x88888888u, y = r[2 * i + 1] ^ 0x88888888u;
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t xs = x >> (8 * h), ys = y >> (8 * h);
                                    const uint32_t a[4] = {xs & 0x000F000Fu, ys & 0x000F000Fu, xs & 0x00F000F0u,
                                                           ys & 0x00F000F0u};
#pragma unroll
                                    for (int n = 0; n < R8; ++n) mma16816<true>(sv[km][n], a, qf[2 * (c + i) + h][n]);
                                }
                            }
                        }
                    }
                // to the exponent's domain: scale * log2(e), the keys' scales, the masks
                const float* ks = reinterpret_cast<const float*>(smem + S::kOffSc + s * 2 * S::kScB) + kw0 + g;
                const bool inner = tile_inside(key, 16 * kKm, inner0, inner1);
                const bool edge = !tile_inside(key, 16 * kKm, u.key0, u.key1);
                float mx[R8][2], vw[kKm][2];
#pragma unroll
                for (int n = 0; n < R8; ++n) mx[n][0] = mx[n][1] = kNoMax;
#pragma unroll
                for (int km = 0; km < kKm; ++km)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // keys g and g + 8 of the block
                        const int k = key + 16 * km + 8 * h + g;
                        if constexpr (FMT != kKvBf16) {
                            // keys outside [key0, key1) are nobody's: their scales may be anything
                            vw[km][h] = edge && (k < u.key0 || k >= u.key1) ? 0.0f : ks[S::kTk + 16 * km + 8 * h];
                        }
                        const float f = FMT != kKvBf16 ? ks[16 * km + 8 * h] : 1.0f;
#pragma unroll
                        for (int n = 0; n < R8; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float& x = sv[km][n][2 * h + i];
                                x *= FMT != kKvBf16 ? rs[n][i] * f : sc;
                                if (!inner && (k > pos[n][i] || k < first[n][i])) x = -INFINITY;
                                mx[n][i] = fmaxf(mx[n][i], x);
                            }
                    }
                bool raise = false;
#pragma unroll
                for (int n = 0; n < R8; ++n) raise |= mx[n][0] > m[n][0] + 8.0f || mx[n][1] > m[n][1] + 8.0f;
                if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                    for (int n = 0; n < R8; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float x = mx[n][i];
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
                            const float mn = fmaxf(m[n][i], x), a = ex2(m[n][i] - mn);
                            m[n][i] = mn;
                            l[n][i] *= a;
#pragma unroll
                            for (int j = 0; j < kDm; ++j) {
                                o[j][n][i] *= a;
                                o[j][n][2 + i] *= a;
                            }
                        }
                }
                // weights; their sum takes them unrounded and without the values' scales
                uint32_t pb[kKm][R8][2];
#pragma unroll
                for (int km = 0; km < kKm; ++km)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < R8; ++n) {
                            float p0 = ex2(sv[km][n][2 * h] - m[n][0]), p1 = ex2(sv[km][n][2 * h + 1] - m[n][1]);
                            l[n][0] += p0;
                            l[n][1] += p1;
                            if constexpr (FMT != kKvBf16) {
                                p0 *= vw[km][h];
                                p1 *= vw[km][h];
                            }
                            pb[km][n][h] = transposed(bf16_pair(p0, p1));
                        }
#pragma unroll
                for (int km = 0; km < kKm; ++km) {
                    // what nobody's slots hold is cleared, not just weighted with 0 (int4 codes are finite
                    // whatever they are)
                    uint32_t vm[2] = {~0u, ~0u};
                    if (FMT != kKvInt4 && edge) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int k = key + 16 * km + 8 * h + 2 * t;
                            vm[h] = (k >= u.key0 && k < u.key1 ? 0x0000FFFFu : 0u) |
                                    (k + 1 >= u.key0 && k + 1 < u.key1 ? 0xFFFF0000u : 0u);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < S::kChunks; c += 2) {
                        uint32_t r[4];
                        ldsm4t(r, vt + chunk_at<S::kBoxB, S::kTk>(kw0 + 16 * km + (lane & 15), c + (lane >> 4)));
                        if (FMT != kKvInt4 && edge) {
                            r[0] &= vm[0], r[2] &= vm[0];
                            r[1] &= vm[1], r[3] &= vm[1];
                        }
                        if constexpr (FMT == kKvBf16) {
                            const uint32_t a[4] = {r[0], r[2], r[1], r[3]};
#pragma unroll
                            for (int n = 0; n < R8; ++n) mma16816<false>(o[c / 2][n], a, pb[km][n]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t x = r[2 * i], y = r[2 * i + 1];
                                if constexpr (FMT == kKvE4m3) {
                                    // bytes 0 and 2 (column 2g of keys 2t, 2t + 1), then 1 and 3 (column 2g + 1)
                                    const uint32_t xp = __byte_perm(x, 0, 0x3120), yp = __byte_perm(y, 0, 0x3120);
                                    const uint32_t a[4] = {e4m3_bf16((uint16_t)xp), e4m3_bf16((uint16_t)(xp >> 16)),
                                                           e4m3_bf16((uint16_t)yp), e4m3_bf16((uint16_t)(yp >> 16))};
#pragma unroll
                                    for (int n = 0; n < R8; ++n) mma16816<false>(o[c + i][n], a, pb[km][n]);
                                } else {
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        const uint32_t a[4] = {int4_pair(x, 2 * h), int4_pair(x, 2 * h + 1),
                                                               int4_pair(y, 2 * h), int4_pair(y, 2 * h + 1)};
#pragma unroll
                                        for (int n = 0; n < R8; ++n) mma16816<false>(o[2 * (c + i) + h][n], a, pb[km][n]);
                                    }
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(empty(s));
        }

        // ------------------------------------------------------ join the four warps
#pragma unroll
        for (int n = 0; n < R8; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], d);
                if (g == 0) ml[warp * kRows + 8 * n + 2 * t + i] = make_float2(m[n][i], l[n][i]);
            }
        compute_sync();
        auto joined = [&](int r) {  // maximum and sum of row r over the warps
            float M = kNoMax, L = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) M = fmaxf(M, ml[k * kRows + r].x);
#pragma unroll
            for (int k = 0; k < 4; ++k) L += ml[k * kRows + r].y * ex2(ml[k * kRows + r].x - M);
            return make_float2(M, L);
        };
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {  // one warp after the other: a fixed order
            if (warp == k) {
#pragma unroll
                for (int n = 0; n < R8; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = 8 * n + 2 * t + i;
                        const float a = ex2(m[n][i] - joined(r).x);
                        float* to = join + r * S::kLd;
#pragma unroll
                        for (int j = 0; j < kDm; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float& x = to[out_col<FMT>(j, h, g)];
                                const float y = o[j][n][2 * h + i] * a;
                                x = k ? x + y : y;
                            }
                    }
            }
            compute_sync();
        }
        // The unit's result, or this CTA's part of it: thread by thread, eight columns of a row
        constexpr int kPieces = kRows * D / 8;
        auto put = [&](int piece, const float* f, float2 st) {
            const int r = piece / (D / 8), col = piece % (D / 8) * 8, tok = token_of(r);
            if (tok < 0) return;
            const float inv = st.y > 0.0f ? 1.0f / st.y : 0.0f;
            const int64_t row = (int64_t)(u.tok0 + tok) * p.a.d.H + head_of(r);
            *reinterpret_cast<uint4*>(p.a.out + row * D + col) =
                make_uint4(bf16_pair(f[0] * inv, f[1] * inv), bf16_pair(f[2] * inv, f[3] * inv),
                           bf16_pair(f[4] * inv, f[5] * inv), bf16_pair(f[6] * inv, f[7] * inv));
            if (p.a.lse && col == 0) p.a.lse[row] = st.y > 0.0f ? (st.x + log2f(st.y)) * kLn2 : -INFINITY;
        };
        auto mine = [&](int piece, float* f) {
            const float4* q = reinterpret_cast<const float4*>(join + piece / (D / 8) * S::kLd + piece % (D / 8) * 8);
            const float4 x = q[0], y = q[1];
            f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
        };
        if (whole) {
            for (int i = tid; i < kPieces; i += 128) {
                float f[8];
                mine(i, f);
                put(i, f, joined(i / (D / 8)));
            }
        } else {
            // a partial result: slot 0 of a CTA for a unit that an earlier CTA began, else slot 1.  The CTA
            // that comes last joins them; if the others have all come its own need not go through memory.
            const int c = blockIdx.x, c0 = share_owner(sh.W, sh.R, unit0 + p.c.unit_cost);
            const int c1 = share_owner(sh.W, sh.R, unit0 + p.c.unit_cost + u.tiles - 1);
            const unsigned others = c1 - c0;
            unsigned* arrived = p.counters + c0;
            auto part = [&](int k) { return p.part + (int64_t)(2 * k + (k == c0)) * S::kPart; };
            if (tid == 0) {
                unsigned n;
                asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(n) : "l"(arrived) : "memory");
                *last_flag = n == others;
            }
            compute_sync();
            bool last = *last_flag;
            if (!last) {
                float* q = part(c);
                for (int i = tid; i < kPieces; i += 128) {
                    float f[8];
                    mine(i, f);
                    float4* to = reinterpret_cast<float4*>(q + i * 8);
                    __stcg(to, make_float4(f[0], f[1], f[2], f[3]));
                    __stcg(to + 1, make_float4(f[4], f[5], f[6], f[7]));
                }
                if (tid < kRows) __stcg(reinterpret_cast<float2*>(q + kRows * D) + tid, joined(tid));
                compute_sync();
                if (tid == 0) {
                    __threadfence();  // the whole group's writes: they come before it by the barrier
                    *last_flag = atomicAdd(arrived, 1u) == others;
                    __threadfence();
                }
                compute_sync();
                last = *last_flag;
            }
            if (last) {
                if (tid == 0) *arrived = 0;
                for (int i = tid; i < kPieces; i += 128) {
                    const int r = i / (D / 8);
                    auto stat = [&](int k) {
                        return k == c ? joined(r) : __ldcg(reinterpret_cast<const float2*>(part(k) + kRows * D) + r);
                    };
                    float2 st = make_float2(kNoMax, 0.0f);
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k) st.x = fmaxf(st.x, stat(k).x);
                    float f[8] = {};
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k) {
                        const float2 e = stat(k);
                        const float a = ex2(e.x - st.x);
                        st.y += e.y * a;
                        float v[8];
                        if (k == c) mine(i, v);
                        else {
                            const float4* q = reinterpret_cast<const float4*>(part(k) + i * 8);
                            const float4 x = __ldcg(q), y = __ldcg(q + 1);
                            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] += v[j] * a;
                    }
                    put(i, f, st);
                }
            }
        }
        compute_sync();  // the buffers are free for the next unit
    } while (next_unit(p, sh, u, unit0));
    pdl_wait();  // behind the chunks' kernel: what follows this one may count on both
}

template <int FMT, int D, int R8>
cudaError_t launch(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, bool behind, float* part,
                   unsigned* counters, cudaStream_t st) {
    using S = RowsShape<FMT, D, R8>;
    AttnParams p;
    p.a = a;
    const int G = a.d.H / a.d.H_kv;
    p.c.hg = std::min(G, S::kRows);
    p.c.tq = S::kRows / p.c.hg;
    p.c.subs = (G + S::kRows - 1) / S::kRows;
    p.c.hs = a.d.H_kv * p.c.subs;
    p.c.tk_log2 = __builtin_ctz(S::kTk);
    p.c.page_log2 = __builtin_ctz(a.d.page);
    // (drafts, a wide int4 step and a bf16 step take 65.2, 35.8 and 31.6 us at 2, 63.6, 35.3 and 31.1 at 3,
    // 63.6, 36.7 and 31.2 at 4, 65.4, 37.1 and 31.3 at 6)
    p.c.unit_cost = 3;
    p.c.min_share = 4;
    p.c.rows_lo = rows_lo;
    p.c.rows_hi = rows_hi;
    p.part = part;
    p.counters = counters;
    p.scale_log2 = a.scale * kLog2e;
    if (!make_kv_map(&p.tm_k, a.cache.k, a, S::kBoxB, std::min(a.d.page, S::kTk)) ||
        !make_kv_map(&p.tm_v, a.cache.v, a, S::kBoxB, std::min(a.d.page, S::kTk)))
        return cudaErrorInvalidValue;
    const void* kern = reinterpret_cast<const void*>(&attn_rows_kernel<FMT, D, R8>);
    cudaError_t e = ensure_dynamic_smem(kern, S::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(S::kCtas * sm_count());
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_rows_kernel<FMT, D, R8>, p);
}

template <int FMT, int D>
cudaError_t launch_for(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, bool eight, bool behind, float* part,
                       unsigned* counters, cudaStream_t st) {
    return eight ? launch<FMT, D, 1>(a, rows_lo, rows_hi, behind, part, counters, st)
                 : launch<FMT, D, 2>(a, rows_lo, rows_hi, behind, part, counters, st);
}

}  // namespace

size_t attn_rows_part_bytes(const moe_kv_dims_t& d) {
    // two slots for each of up to four CTAs per SM with 8 rows, or two with 16
    return (size_t)(2 * sm_count()) * std::max(4 * 8, 2 * 16) * (d.D + 2) * sizeof(float);
}

cudaError_t launch_attn_rows(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, bool eight, bool behind, float* part,
                             unsigned* counters, cudaStream_t st) {
    const bool wide = a.d.D == 128;
    switch (a.d.format) {
        case kKvBf16:
            return wide ? launch_for<kKvBf16, 128>(a, rows_lo, rows_hi, eight, behind, part, counters, st)
                        : launch_for<kKvBf16, 64>(a, rows_lo, rows_hi, eight, behind, part, counters, st);
        case kKvE4m3:
            return wide ? launch_for<kKvE4m3, 128>(a, rows_lo, rows_hi, eight, behind, part, counters, st)
                        : launch_for<kKvE4m3, 64>(a, rows_lo, rows_hi, eight, behind, part, counters, st);
        case kKvInt4:
            return wide ? launch_for<kKvInt4, 128>(a, rows_lo, rows_hi, eight, behind, part, counters, st)
                        : launch_for<kKvInt4, 64>(a, rows_lo, rows_hi, eight, behind, part, counters, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
