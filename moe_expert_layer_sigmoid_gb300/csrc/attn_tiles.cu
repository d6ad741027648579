// Attention of many rows (chunks of a prompt, drafts) on the tcgen05 tensor
// cores: 128 rows (tokens x query heads of one key/value head) per accumulator,
// two accumulators per CTA, one CTA per SM.
//
// A key tile of 128 keys is two products, S = Q K^T (128 x 128 x D, both operands
// in shared memory) and O += P V (P in TMEM, V in shared memory, row-major as the
// cache holds it: the MN-major operand form).  At D = 128 each takes 512 tensor
// cycles, so the softmax of a tile (128 exponentials per row) has to hide behind
// the other accumulator's products: while warpgroup A turns its S into P, the
// tensor core works on B's P V and next Q K^T, and the other way round.
// Streams A and B are
//   - two row tiles of one unit walking the same key tiles, when the unit has
//     more than 128 rows (each K and V tile is read once for both), or
//   - even and odd key tiles of one row tile, joined at the end, when it has not.
//
// TMEM (512 columns): S of A and B at 0 and 128, O at 256 and 384.  P (bf16, two
// keys per column) overwrites S, each half of the keys its own half's first columns; the
// next S of a stream is issued after the P V that reads P, and the tensor core runs one
// thread's products in order.
//
// Two threads own a row, each half of a tile's keys, no shuffles.  A tile takes one pass over S, with the
// running maximum as it stands; a barrier with a vote tells whether some score exceeds it by 2^8 (rows that
// no token fills have no vote: their queries are whatever lies in shared memory, and the others' maxima, so their
// rounding, would depend on it), and in those few tiles (S is still whole: P is stored after the vote) the halves exchange their maxima, O is
// rescaled (read, scaled and written back in TMEM) and the pass done again.  When S of tile i is ready,
// P V of tile i - 1 is too, so O may be touched without a further wait.  The loop's issue slots and
// registers are what the tensor core waits for most, so S is read 32 columns at a time and the
// arithmetic is packed two to an instruction.
//
// Quantised caches: TMA brings the codes to a ring of their own, two warpgroups (one for keys, one for
// values) turn them into bf16 tiles.  Key scales multiply the scores, value scales the weights, so
// codes enter the products exactly.
//
// Warps: 0 copies, 1 products (and TMEM), 2-3 none, 4-11 stream A, 12-19 stream B (in each
// four warps for the first 64 keys of a tile and four for the last), 20-23 conversion
// of keys, 24-27 of values.
//
// Measured (GB300, 2048 tokens, D = 128): behind 27,953 keys 730 to 754 us in bf16 (by clocks), 1290 to
// 1334 TFLOP/s, 66 to 68% of a library product's rate; 1020 us in E4M3, 953 TFLOP/s, and 986 in int4, where the
// conversion's warps take issue slots (53% used against 40%) from the softmax.  With no keys before it
// 57 us: 14 pairs of key tiles per CTA, which the long chunk walks in half of that, so the rest is what a
// CTA does before and after its walk.  All forms spill in the softmax's loop (coded caches 328 bytes stored and
// 448 loaded at 72 registers, bf16 80 and 124 at 96).
#include <atomic>
#include <type_traits>

#include "attn.cuh"
#include "umma.cuh"

namespace moe {
namespace {

constexpr int kTileRows = 128;
constexpr int kTk = 128;  // keys of a tile

template <int FMT, int D>
struct TilesShape {
    static constexpr bool kQuant = FMT != kKvBf16;
    static constexpr int kThreads = kQuant ? 896 : 640;
    static constexpr int kRowB = kv_row_bytes(FMT, D);
    static constexpr int kBoxB = kRowB < 128 ? kRowB : 128;
    static constexpr int kTileB = kTk * D * 2;                // a bf16 tile
    static constexpr int kSlots = kQuant ? 3 : 4;             // bf16 tiles of keys or values
    // Tiles of codes.  No more than bf16 slots: a tile's codes are only there (CodeRing's barriers tell
    // exactly) once the tile three before it is converted, for which the slot's product before that was done.
    // So the wait for the bf16 slot of a tile cannot take the release before the last for the last.
    static constexpr int kRaws = kQuant ? 3 : 0;
    static_assert(kRaws <= kSlots, "phases");
    using Ring = CodeRing<kQuant ? kRaws : 1>;
    static constexpr int kRawFulls = kQuant ? Ring::kFull : 0;
    static constexpr int kRawB = kTk * kRowB;
    // Key and value scales of a tile.  Four slots: while V of tile i is in use (K of tile i + 2 would take its
    // place) no codes after K of tile i + 3 are loaded.
    static constexpr int kScB = kQuant ? 2 * kTk * 4 : 0;
    static constexpr int kScSlots = 4;
    // registers per thread: control, streams, conversion; in 128-thread groups they add up to
    // what the launch holds (96 x 640 or 72 x 896)
    static constexpr int kRegCtl = kQuant ? 56 : 96, kRegStream = kQuant ? 88 : 96, kRegConv = 48;
    static_assert(kRegCtl + 4 * kRegStream + (kQuant ? 2 * kRegConv : 0) <= (kQuant ? 504 : 480), "register split");
    static constexpr int kOffQ = 0;
    static constexpr int kOffKv = kOffQ + 2 * kTileRows * D * 2;
    static constexpr int kOffRaw = kOffKv + kSlots * kTileB;
    static constexpr int kOffSc = kOffRaw + kRaws * kRawB;
    // output rows on their way from registers to coalesced stores: 16 rows x 32 bytes per warp
    static constexpr int kOffStage = kOffSc + kScSlots * kScB;
    static constexpr int kOffMl = kOffStage + 16 * 512;  // the streams' maxima and sums: [stream][half][row]
    static constexpr int kOffBar = kOffMl + 4 * kTileRows * 8;
    // barriers: FULL, EMPTY [kSlots]; RAWF [kRawFulls], RAWE [kRaws]; SF, PF, OD [2]; QF, QE, TD
    static constexpr int kBarFull = 0, kBarEmpty = kSlots, kBarRawF = 2 * kSlots, kBarRawE = kBarRawF + kRawFulls,
                         kBarSf = kBarRawE + kRaws, kBarPf = kBarSf + 2, kBarOd = kBarPf + 2,
                         kBarQf = kBarOd + 2, kBarQe = kBarQf + 1, kBarTd = kBarQe + 1, kNumBars = kBarTd + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmem = kOffMisc + 16 + sizeof(Share);
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
    // a partial result: both streams' rows, O as float4 columns of 128 rows, then maximum and sum
    static constexpr int kPartStream = kTileRows * D + 2 * kTileRows;
    static constexpr int kPart = 2 * kPartStream;
};
constexpr int kPartSlots = 2;  // per CTA: a unit begun before, a unit ended after

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two floats in one 64-bit register, for the packed forms: one instruction for both.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(uint32_t lo, uint32_t hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ f2 pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ void split(f2 x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void lds_f2x2(uint32_t addr, f2& a, f2& b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// A pair of consecutive E4M3 codes (the low or the high half of w) as two bf16, exact at every step: by
// way of f16 and fp32, as those conversions spread over more pipes than moving the bits does (0.77
// pairs of a warp per clock and SM against 0.50).
__device__ __forceinline__ uint32_t e4m3_two(uint32_t w, bool high) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(high ? w >> 16 : w)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return bf16x2_of(f.x, f.y);
}
// Nibbles 2i and 2i + 1 of w (two's complement) as two bf16: 128 + (n + 8) by its bits, less 136.
__device__ __forceinline__ uint32_t int4_two(uint32_t w, int i) {
    const uint32_t b = w >> (8 * i);
    uint32_t t, r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(t) : "r"((b & 0xFu) | (b << 12)), "r"(0x000F000Fu), "r"(0x43084308u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(t), "r"(0x3F803F80u), "r"(0xC308C308u));
    return r;
}

// One CTA's stretch of a unit: which key tiles each stream takes.
struct Stretch {
    int t0, t1;        // tiles of the unit, relative to u.tile0
    int lo[2], hi[2];  // of them, those with keys for the stream's rows
    bool split;        // even and odd tiles of one row tile instead of two row tiles
    __device__ __forceinline__ bool act(int x, int i) const {
        if (split && ((i - t0) & 1) != x) return false;
        return i >= lo[x] && i < hi[x];
    }
};

__device__ __forceinline__ Stretch stretch(const AttnParams& p, const Share& sh, const Unit& u, int64_t unit0) {
    Stretch s;
    unit_share(p, sh, u, unit0, s.t0, s.t1);
    const int half = p.c.tq / 2, i0 = u.rt * p.c.tq, have = min(p.c.tq, u.n - i0);
    s.split = have <= half;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        // the stream's tokens [a, b) of the sequence, their keys [k0, k1)
        const int a = i0 + (s.split ? 0 : x * half), b = min(u.n, s.split ? i0 + have : a + half);
        const int k1 = max(0, u.len - u.n + b);
        const int k0 = first_key(u.len - u.n + a, p.a.d.window);
        s.lo[x] = max(s.t0, k0 / kTk - u.tile0);
        s.hi[x] = k1 > k0 ? min(s.t1, tiles_until(k1, 7) - u.tile0) : s.lo[x];
    }
    return s;
}

template <int FMT, int D>
__global__ void __launch_bounds__(TilesShape<FMT, D>::kThreads, 1)
attn_tiles_kernel(const __grid_constant__ AttnParams p) {
    using S = TilesShape<FMT, D>;
    constexpr int kSlots = S::kSlots;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
    volatile int* last_flag = abort_flag + 1;
    WsHeader* hdr = p.a.hdr;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(bar(S::kBarFull + s), S::kQuant ? 4 : 1);
            mbar_init(bar(S::kBarEmpty + s), 1);
        }
        for (int s = 0; s < S::kRawFulls; ++s) mbar_init(bar(S::kBarRawF + s), 1);
        for (int s = 0; s < S::kRaws; ++s) mbar_init(bar(S::kBarRawE + s), 4);
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(S::kBarSf + x), 1);
            mbar_init(bar(S::kBarPf + x), 8);
            mbar_init(bar(S::kBarOd + x), 1);
        }
        mbar_init(bar(S::kBarQf), 1);
        mbar_init(bar(S::kBarQe), 1);
        mbar_init(bar(S::kBarTd), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_trigger();  // the kernel of few rows may start where this one leaves room
    const uint32_t withheld = withheld_stage(hdr);
    // (the share stays in shared memory: it is looked at once per unit, and registers are short)
    Share& sh = *reinterpret_cast<Share*>(smem + S::kOffMisc + 16);
    {
        const Share mine = deal<S::kThreads>(p, smem);
        if (mine.w0 >= mine.w1) return;
        if (threadIdx.x == 0) sh = mine;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Unit u = sh.u;
    int64_t unit0 = sh.unit0;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegCtl));
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            const int page = 1 << p.c.page_log2;
            const int box_rows = page < kTk ? page : kTk;
            const int boxes = kTk / box_rows;
            using Ring = typename S::Ring;
            constexpr uint32_t kRing = S::kQuant ? S::kRaws : kSlots;
            // the barrier and its parity that copy k completes
            auto full = [&](uint32_t k) { return bar(S::kQuant ? S::kBarRawF + Ring::full(k) : S::kBarFull + k % kSlots); };
            auto parity = [&](uint32_t k) { return S::kQuant ? Ring::full_parity(k) : (k / kSlots) & 1; };
            uint32_t it = 0;   // slots filled
            uint32_t tiles = 0, n_q = 0;
            bool ok = true;
            const int half = p.c.tq / 2;
            do {
                int tile, end;
                unit_share(p, sh, u, unit0, tile, end);
                if (tile >= end) continue;
                const int hk = u.hs;
                // the queries, {64 columns, heads, tokens} boxes: row r of a stream is token r / heads,
                // head r % heads.  Rows of other sequences' tokens may come along: rows do not mix.
                if (!warp_wait(bar(S::kBarQe), (n_q & 1) ^ 1, abort_flag, hdr)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int tok = u.tok0 + u.rt * p.c.tq, tok1 = tok + (u.n - u.rt * p.c.tq > half ? half : 0);
                    mbar_expect_tx(bar(S::kBarQf), 2 * (D / 64) * half * p.c.hg * 128);
                    for (int h = 0; h < 2 * (D / 64); ++h) {
                        const int x = h / (D / 64), c = h % (D / 64);
                        tma_load_3d(sbase + S::kOffQ + x * kTileRows * D * 2 + c * (128 * 128), &p.tm_q, c * 64,
                                    hk * p.c.hg, x ? tok1 : tok, bar(S::kBarQf));
                    }
                }
                ++n_q;
                __syncwarp();
                const int32_t* row = p.a.pages + (int64_t)u.b * p.a.d.max_pages;
                const int pg0 = u.key0 >> p.c.page_log2;
                const int pg1 = tiles_until(u.key1, p.c.page_log2);
                auto fetch = [&](int at) {
                    const int i = at + lane;
                    return i >= pg0 && i < pg1 ? __ldg(row + i) : 0;
                };
                int ids = 0, ids_next = 0, ids_at = -1;  // 32 page ids from page ids_at on
                for (; tile < end && ok; ++tile, ++tiles) {
                    const int key = (u.tile0 + tile) * kTk;
                    const int pg = key >> p.c.page_log2;
                    if (ids_at < 0 || pg >= ids_at + 32) {
                        const int at = pg & ~31;
                        ids = ids_at >= 0 && at == ids_at + 32 ? ids_next : fetch(at);
                        ids_at = at;
                        ids_next = fetch(at + 32);
                    }
                    int id = __shfl_sync(0xFFFFFFFFu, ids, (pg + lane) & 31);
                    const bool live = lane < boxes && pg + lane >= pg0 && pg + lane < pg1 &&
                                      key + lane * box_rows < u.key1;
                    if (live && (id < 0 || id >= p.a.d.n_pages)) {
                        record_error(hdr, kErrBadPage);
                        id = 0;
                    }
                    const uint32_t n_live = __popc(__ballot_sync(0xFFFFFFFFu, live));
                    const int at = key & (page - 1);
#pragma unroll
                    for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
                        const int s = it % kRing;  // (its wait takes one phase after the other)
                        if (!warp_wait(bar((S::kQuant ? S::kBarRawE : S::kBarEmpty) + s),
                                       S::kQuant ? Ring::free_parity(it) : ((it / kSlots) & 1) ^ 1, abort_flag, hdr)) {
                            ok = false;
                            break;
                        }
                        const uint32_t done = full(it);
                        const uint32_t sc_bytes = S::kQuant ? box_rows * 4 : 0;
                        if (lane == 0) mbar_expect_tx(done, n_live * (box_rows * S::kRowB + sc_bytes));
                        __syncwarp();
                        if (live && it + 1 != withheld) {
                            const CUtensorMap* tm = kv ? &p.tm_v : &p.tm_k;
                            const uint32_t d = sbase + (S::kQuant ? S::kOffRaw + s * S::kRawB : S::kOffKv + s * S::kTileB) +
                                               lane * box_rows * S::kBoxB;
#pragma unroll
                            for (int h = 0; h < S::kRowB / S::kBoxB; ++h)
                                tma_load_4d(d + h * kTk * S::kBoxB, tm, h * S::kBoxB / (S::kQuant ? 1 : 2), at, hk, id, done);
                            if (S::kQuant)
                                bulk_load(sbase + S::kOffSc + (tiles % S::kScSlots) * S::kScB + kv * kTk * 4 + lane * box_rows * 4,
                                          (kv ? p.a.cache.vs : p.a.cache.ks) + ((int64_t)id * p.a.d.H_kv + hk) * page + at,
                                          sc_bytes, done);
                        }
                        __syncwarp();
                    }
                }
            } while (ok && next_unit(p, sh, u, unit0));
            if (!ok && n_q) mbar_drain(bar(S::kBarQf), (n_q - 1) & 1, hdr);
            if (!ok)  // no copy may be in flight when the CTA ends
                for (uint32_t k = it > kRing ? it - kRing : 0; k < it; ++k)
                    mbar_drain(full(k), parity(k), hdr);
        } else if (warp == 1) {
            // ---------------------------------------------------------- products
            // The whole warp follows the loop, so that its values are uniform; one thread issues.
            const uint32_t id_qk = idesc_bf16(128, kTk), id_pv = idesc_bf16_bmn(128, D);
            const uint32_t q_lo = desc_lo_sw128(sbase + S::kOffQ), k_lo = desc_lo_sw128(sbase + S::kOffKv);
            const uint32_t v_lo = desc_lo_sw128_mn(sbase + S::kOffKv, kTk * 128);
            uint32_t it0 = 0;    // slot index of the stretch's first key tile
            uint32_t n_pf[2] = {0, 0}, n_q = 0;
            bool ok = true;
            bool fresh[2];       // no product in the stream's O yet
            auto wait = [&](int b, uint32_t par) {
                if (ok) ok = warp_wait(bar(b), par & 1, abort_flag, hdr);
                tc_fence_after();
                return ok;
            };
            // K of relative tile i is the slot 2 i after it0, V the next
            auto full = [&](uint32_t k) { return wait(S::kBarFull + k % kSlots, k / kSlots); };
            auto release = [&](uint32_t k) {
                if (elect_one()) mma_commit(bar(S::kBarEmpty + k % kSlots));
                __syncwarp();
            };
            auto qk = [&](int x, uint32_t k) {
                const uint32_t a = q_lo + x * (kTileRows * D * 2 / 16), b = k_lo + (k % kSlots) * (S::kTileB / 16);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t o = ((ks / 4) * (128 * 128) + (ks % 4) * 32) / 16;
                        mma_ss_lo(tmem + x * 128, a + o, b + o, id_qk, ks > 0);
                    }
                    mma_commit(bar(S::kBarSf + x));
                }
                __syncwarp();
            };
            auto pv = [&](int x, uint32_t k) {
                const uint32_t b = v_lo + (k % kSlots) * (S::kTileB / 16);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kTk / 16; ++ks)
                        mma_ts_lo(tmem + 256 + x * 128, tmem + x * 128 + ks / 4 * 64 + ks % 4 * 8, b + ks * (16 * 128 / 16), id_pv,
                                  ks > 0 || !fresh[x]);
                }
                __syncwarp();
                fresh[x] = false;
            };
            do {
                const Stretch s = stretch(p, sh, u, unit0);
                if (s.t0 >= s.t1) continue;
                auto kslot = [&](int i) { return it0 + 2 * (uint32_t)(i - s.t0); };
                fresh[0] = fresh[1] = true;
                // first products; a stream whose first tile comes later starts in the loop
                if (!wait(S::kBarQf, n_q++) || !full(kslot(s.t0))) break;
                if (s.act(0, s.t0)) qk(0, kslot(s.t0));
                if (s.act(1, s.t0)) qk(1, kslot(s.t0));
                release(kslot(s.t0));
                if (s.split && s.t0 + 1 < s.t1) {
                    if (!full(kslot(s.t0 + 1))) break;
                    if (s.act(1, s.t0 + 1)) qk(1, kslot(s.t0 + 1));
                    release(kslot(s.t0 + 1));
                }
                // behind the unit's last scores the place of its queries is free
                const int stride = s.split ? 2 : 1;
                auto queries_done = [&] {
                    if (elect_one()) mma_commit(bar(S::kBarQe));
                    __syncwarp();
                };
                if (s.t1 - s.t0 <= stride) queries_done();
                for (int i = s.t0; i < s.t1; ++i) {
                    if (!full(kslot(i) + 1)) break;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (s.act(x, i)) {
                            if (!wait(S::kBarPf + x, n_pf[x]++)) break;
                            pv(x, kslot(i) + 1);
                            if (!s.act(x, i + stride)) {  // the stream's output of the unit is whole
                                if (elect_one()) mma_commit(bar(S::kBarOd + x));
                                __syncwarp();
                            }
                        }
                        if (!s.split && s.act(x, i + 1)) {
                            if (!full(kslot(i + 1))) break;
                            qk(x, kslot(i + 1));
                        }
                    }
                    if (!ok) break;
                    release(kslot(i) + 1);
                    if (!s.split && i + 1 < s.t1) {
                        if (!full(kslot(i + 1))) break;
                        release(kslot(i + 1));
                    } else if (s.split && i + 2 < s.t1) {
                        if (!full(kslot(i + 2))) break;
                        const int x = (i - s.t0) & 1;
                        if (s.act(x, i + 2)) {
                            if (x) qk(1, kslot(i + 2));
                            else qk(0, kslot(i + 2));
                        }
                        release(kslot(i + 2));
                    }
                    if (i + stride == s.t1 - 1) queries_done();
                }
                if (!ok) break;
                it0 = kslot(s.t1);
            } while (next_unit(p, sh, u, unit0));
            if (!ok) {  // products in flight end before TMEM is given back
                if (elect_one()) mma_commit(bar(S::kBarTd));
                __syncwarp();
                mbar_drain(bar(S::kBarTd), 0, hdr);
            }
        }
    } else if (warp < 20) {
        // ----------------------------------------------------------------- streams
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegStream));
        const int x = warp >= 12, hf = (warp >> 2) & 1 ^ 1;   // stream, half of the key tile's columns
        const int r = (warp & 3) * 32 + lane;                 // row
        const uint32_t trow = tmem + ((uint32_t)(warp & 3) << 21);  // the warp's 32 lanes
        const uint32_t ts = trow + x * 128, to = trow + 256 + x * 128;
        // (not 0, so that a masked score stays infinite)
        const bool neg = p.scale_log2 < 0.0f;
        const float sc = fmaxf(fabsf(p.scale_log2), 1e-37f);
        const int G = p.a.d.H / p.a.d.H_kv, half = p.c.tq / 2;
        uint8_t* stage = smem + S::kOffStage + (warp - 4) * 512;
        float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);
        float* top = reinterpret_cast<float*>(ml + 2 * x * kTileRows) + r;  // + half * rows: halves' maxima
        uint32_t n_sf = 0, n_od = 0, tiles0 = 0;  // tiles0: tiles of the CTA before this stretch
        bool ok = true;
        auto wait = [&](int b, uint32_t par) {  // once a wait gave up the streams run on, in step
            if (ok) ok = mbar_wait(bar(b), par & 1, abort_flag, hdr);
        };
        auto stream_sync = [&] { asm volatile("bar.sync %0, 256;" ::"r"(2 + x) : "memory"); };
        auto all_sync = [&] { asm volatile("bar.sync 1, 512;" ::: "memory"); };
        int64_t orow;       // this thread's row of out and lse: token * H + head, -1: none
        int pos, first;     // keys it sees: first .. pos
        auto rows_of = [&](const Unit& v, bool split) {
            const int tok = v.rt * p.c.tq + (split ? 0 : x * half) + r / G, hd = v.hs * G + r % G;
            const bool live = r < half * G && tok < v.n;
            orow = live ? (int64_t)(v.tok0 + tok) * p.a.d.H + hd : -1;
            pos = live ? v.len - v.n + tok : -1;
            first = first_key(pos, p.a.d.window);
        };
        // 16 columns of the warp's rows (bf16 pairs) to `out`, by way of shared memory, 16 rows at a time:
        // each two lanes store 32 bytes of a row
        auto put = [&](const uint32_t* e, int col) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (lane >> 4 == h) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4*>(stage + (lane & 15) * 32 + ((k ^ ((lane >> 2) & 1)) << 4)) =
                            make_uint4(e[4 * k], e[4 * k + 1], e[4 * k + 2], e[4 * k + 3]);
                }
                __syncwarp();
                const int rr = lane >> 1, c = lane & 1;
                const int64_t row = __shfl_sync(0xFFFFFFFFu, orow, 16 * h + rr);
                const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 32 + ((c ^ ((rr >> 2) & 1)) << 4));
                if (row >= 0) *reinterpret_cast<uint4*>(p.a.out + row * D + col + 8 * c) = v;
                __syncwarp();
            }
        };
        do {
            const Stretch s = stretch(p, sh, u, unit0);
            if (s.t0 >= s.t1) continue;
            rows_of(u, s.split);
            const bool whole = s.t0 == 0 && s.t1 == u.tiles;
            float m = kNoMax, l = 0.0f;
            // keys that all of the stream's rows see need no mask
            const int i0 = u.rt * p.c.tq + (s.split ? 0 : x * half);
            const int inner1 = max(0, u.len - u.n + i0 + 1);
            const int inner0 = first_key(u.len - u.n + min(u.n, i0 + half) - 1, p.a.d.window);
            // the stream's tiles: i0 .. (every other one with one row tile)
            const int step = s.split ? 2 : 1;
            const int beg = s.split ? s.t0 + x : x ? s.lo[1] : s.lo[0], end = x ? s.hi[1] : s.hi[0];
            uint32_t from = (uint32_t)(u.tile0 + beg) * kTk;  // the tile's first key (past the last tile it may be 2^31)
            uint32_t vk = 2 * (tiles0 + (uint32_t)(beg - s.t0)) + 1;  // the value tile's slot index
            // keys outside [key0, key1) are nobody's: their slots may hold anything.  bf16 values are cleared
            // there, not just weighted with 0, by the first stream that takes the tile: by B where A has none.
            const int key0 = u.key0, key1 = u.key1;
            const int clear0 = s.split || x == 0 ? 0 : s.hi[0];
#pragma unroll 1
            for (int i = beg; i < end; i += step, from += step * kTk, vk += 2 * step) {
                const int key = (int)from;
                wait(S::kBarSf + x, n_sf++);
                tc_fence_after();
                if (!S::kQuant && !tile_inside(key, kTk, key0, key1) && (i >= clear0 || (x == 1 && i < s.lo[0]))) {
                    wait(S::kBarFull + vk % kSlots, vk / kSlots);
                    if (key + r < key0 || key + r >= key1) {
                        uint8_t* z = smem + S::kOffKv + (vk % kSlots) * S::kTileB + r * 128;
#pragma unroll
                        for (int c = hf * (D / 16); c < (hf + 1) * (D / 16); ++c)
                            *reinterpret_cast<uint4*>(z + (c / 8) * (128 * 128) + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async();
                }
                const bool inner = tile_inside(key, kTk, inner0, inner1);
                // quantised: the half's key scales (times the call's; in place since before the products
                // that S comes from), then its value scales
                const uint32_t ksc = sbase + S::kOffSc + ((vk / 2) % S::kScSlots) * S::kScB + 256 * hf;
                // 32 of the half's 64 scores, masked; a negative scale turns their sign
                auto scores = [&](uint32_t* vr, int c) {
                    tmem_ld_x32(ts + 64 * hf + 32 * c, vr);
                    tmem_wait_ld32(vr);
                    float* v = reinterpret_cast<float*>(vr);
                    if (neg) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = -v[k];
                    }
                    if (!inner) {
                        // bit k: column k is seen
                        const int at = key + 64 * hf + 32 * c, h = pos - at, g = first - at;
                        const uint32_t see = (h >= 31 ? ~0u : h < 0 ? 0u : (2u << h) - 1) &
                                             (g <= 0 ? ~0u : g > 31 ? 0u : ~0u << g);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(see >> k & 1)) v[k] = -INFINITY;
                    }
                };
                // the factors of four of them into the exponent's domain
                auto factors = [&](int c, int k, f2& f0, f2& f1) {
                    if (S::kQuant) lds_f2x2(ksc + 128 * c + 16 * k, f0, f1);
                    else f0 = f1 = pair(sc, sc);
                };
                if (S::kQuant) wait(S::kBarFull + vk % kSlots, vk / kSlots);  // for the value scales
                uint32_t pk[32];
                f2 l0, l1;
                int raise = i == beg;
#pragma unroll 1
                for (int k2 = 0; k2 < 2; ++k2) {
                    if (raise) {
                        float mx = kNoMax;
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t vr[32];
                            scores(vr, c);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                f2 f0, f1;
                                float e0, e1, e2, e3;
                                factors(c, k, f0, f1);
                                split(mul2(pair(vr[4 * k], vr[4 * k + 1]), f0), e0, e1);
                                split(mul2(pair(vr[4 * k + 2], vr[4 * k + 3]), f1), e2, e3);
                                mx = max3(mx, e0, e1);
                                mx = max3(mx, e2, e3);
                            }
                        }
                        top[hf * kTileRows] = mx;
                        stream_sync();
                        mx = fmaxf(top[0], top[kTileRows]);
                        // (a little above the largest score, so that no rounding of a product lets the exact
                        // one in the fma come out above it)
                        const float mn = mx > m ? mx + fabsf(mx) * 1.2e-7f : m, a = ex2(m - mn);
                        m = mn;
                        l *= a;
                        if (i > beg) {  // P V of the tile before is done: S of this one came after it
#pragma unroll 1
                            for (int c = hf * (D / 2); c < (hf + 1) * (D / 2); c += 16) {
                                uint32_t o[16];
                                tmem_ld_x16(to + c, o);
                                tmem_wait_ld16(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                                tmem_st_x16(to + c, o);
                            }
                        }
                    }
                    const f2 nm = pair(-m, -m);
                    float t0 = kNoMax, t1 = kNoMax;
                    l0 = l1 = pair(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t vr[32];
                        scores(vr, c);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            f2 f0, f1;
                            float e0, e1, e2, e3;
                            factors(c, k, f0, f1);
                            split(fma2(pair(vr[4 * k], vr[4 * k + 1]), f0, nm), e0, e1);
                            split(fma2(pair(vr[4 * k + 2], vr[4 * k + 3]), f1, nm), e2, e3);
                            t0 = max3(t0, e0, e1);
                            t1 = max3(t1, e2, e3);
                            f2 a = pair(ex2(e0), ex2(e1)), b = pair(ex2(e2), ex2(e3));
                            l0 = add2(l0, a);
                            l1 = add2(l1, b);
                            if (S::kQuant) {
                                lds_f2x2(ksc + 512 + 128 * c + 16 * k, f0, f1);
                                a = mul2(a, f0);
                                b = mul2(b, f1);
                            }
                            split(a, e0, e1);
                            split(b, e2, e3);
                            pk[16 * c + 2 * k] = bf16x2_of(e0, e1);
                            pk[16 * c + 2 * k + 1] = bf16x2_of(e2, e3);
                        }
                    }
                    asm volatile(
                        "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 256, p;\n"
                        " selp.b32 %0, 1, 0, q;\n}"
                        : "=r"(raise)
                        : "r"((int)(pos >= 0 && fmaxf(t0, t1) > 8.0f)), "r"(2 + x)
                        : "memory");
                    if (!raise) break;
                }
                // over the first of the half's own scores
                tmem_st_x32(ts + 64 * hf, pk);
                {
                    float a0, a1;
                    split(add2(l0, l1), a0, a1);
                    l += a0 + a1;
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::kBarPf + x));
            }
            const bool any = beg < end;
            tiles0 += s.t1 - s.t0;
            if (any) wait(S::kBarOd + x, n_od++);
            // maxima and sums of the halves (and, with one row tile, of both streams)
            ml[(2 * x + hf) * kTileRows + r] = make_float2(m, l);
            if (s.split) all_sync();
            else stream_sync();
            tc_fence_after();
            // The CTA's own result of the stretch, unnormalised: a0 * (this stream's output), or with one
            // row tile a0 * (A's) + a1 * (B's).  This thread takes the columns [cb, ce) of its row.
            float M = m, L = ml[2 * x * kTileRows + r].y + ml[(2 * x + 1) * kTileRows + r].y, a0 = 1.0f, a1 = 0.0f;
            bool use0 = any, use1 = false;  // (the same for the whole warp: by the stretch, not by a row's values)
            uint32_t o0 = to, o1 = to;
            int cb = hf * (D / 2), ce = cb + D / 2;
            if (s.split) {
                constexpr int kQ = D / 4 < 32 ? 32 : D / 4;
                cb = min(D, (2 * x + hf) * kQ);
                ce = min(D, cb + kQ);
                const float2 e0 = ml[r], e1 = ml[2 * kTileRows + r];
                M = fmaxf(e0.x, e1.x);
                a0 = ex2(e0.x - M);
                a1 = ex2(e1.x - M);
                L = (e0.y + ml[kTileRows + r].y) * a0 + (e1.y + ml[3 * kTileRows + r].y) * a1;
                use0 = s.act(0, s.t0);
                use1 = s.act(1, s.t0 + 1);
                o0 = trow + 256;
                o1 = trow + 384;
            }
            auto own = [&](int col, float* f) {  // columns col .. col + 15
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = 0.0f;
                if (use0) {
                    tmem_ld_x16(o0 + col, o);
                    tmem_wait_ld16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(o[e]) * a0;
                }
                if (use1) {
                    tmem_ld_x16(o1 + col, o);
                    tmem_wait_ld16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] += __uint_as_float(o[e]) * a1;
                }
            };
            auto finish = [&](const float* f, int col, float inv) {
                uint32_t e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] = bf16x2_of(f[2 * k] * inv, f[2 * k + 1] * inv);
                put(e, col);
            };
            bool join = false;
            const int c = blockIdx.x;
            int c0 = c, c1 = c;
            const bool stats = s.split ? x == 0 && hf == 0 : hf == 0;  // the thread that speaks for its row
            if (!whole) {
                // A partial result; the CTA that comes last to the unit joins them.  If the others
                // have all come its own need not go through memory.
                c0 = share_owner(sh.W, sh.R, unit0 + p.c.unit_cost);
                c1 = share_owner(sh.W, sh.R, unit0 + p.c.unit_cost + u.tiles - 1);
                const unsigned others = c1 - c0;
                unsigned* arrived = p.counters + c0;
                if (threadIdx.x == 128) {
                    unsigned n;
                    asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(n) : "l"(arrived) : "memory");
                    *last_flag = n == others;
                }
                all_sync();
                join = *last_flag;
                if (!join) {
                    float* part = p.part + ((int64_t)kPartSlots * c + (c == c0)) * S::kPart + (s.split ? 0 : x) * S::kPartStream;
                    float4* po = reinterpret_cast<float4*>(part);
#pragma unroll 1
                    for (int col = cb; col < ce; col += 16) {
                        float f[16];
                        own(col, f);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            __stcg(po + (col / 4 + e) * kTileRows + r, make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]));
                    }
                    if (stats) __stcg(reinterpret_cast<float2*>(part + kTileRows * D) + r, make_float2(M, L));
                    all_sync();
                    if (threadIdx.x == 128) {
                        __threadfence();  // the whole group's writes: they come before it by the barrier
                        *last_flag = atomicAdd(arrived, 1u) == others;
                        __threadfence();
                    }
                    all_sync();
                    join = *last_flag;
                }
                if (join && threadIdx.x == 128) *arrived = 0;
            }
            if (whole) {
                const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll 1
                for (int col = cb; col < ce; col += 16) {
                    float f[16];
                    own(col, f);
                    finish(f, col, inv);
                }
            } else if (join) {
                auto part = [&](int k) {
                    return p.part + ((int64_t)kPartSlots * k + (k == c0)) * S::kPart + (s.split ? 0 : x) * S::kPartStream;
                };
                auto stat = [&](int k) {  // maximum and sum of part k
                    return k == c ? make_float2(M, L) : __ldcg(reinterpret_cast<const float2*>(part(k) + kTileRows * D) + r);
                };
                float Mj = kNoMax, Lj = 0.0f;
#pragma unroll 4
                for (int k = c0; k <= c1; ++k) Mj = fmaxf(Mj, stat(k).x);
#pragma unroll 4
                for (int k = c0; k <= c1; ++k) {
                    const float2 e = stat(k);
                    Lj += e.y * ex2(e.x - Mj);
                }
                const float inv = Lj > 0.0f ? 1.0f / Lj : 0.0f;
#pragma unroll 1
                for (int col = cb; col < ce; col += 16) {
                    float f[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = 0.0f;
#pragma unroll 1
                    for (int k = c0; k <= c1; ++k) {
                        const float a = ex2(stat(k).x - Mj);
                        float g[16];
                        if (k == c) own(col, g);
                        else {
                            const float4* q = reinterpret_cast<const float4*>(part(k)) + (col / 4) * kTileRows + r;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 v = __ldcg(q + e * kTileRows);
                                g[4 * e] = v.x, g[4 * e + 1] = v.y, g[4 * e + 2] = v.z, g[4 * e + 3] = v.w;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] += g[e] * a;
                    }
                    finish(f, col, inv);
                }
                M = Mj;
                L = Lj;
            }
            if ((whole || join) && orow >= 0 && p.a.lse && stats)
                p.a.lse[orow] = L > 0.0f ? (M + log2f(L)) * kLn2 : -INFINITY;
            // Every thread has read the outputs, sums and flags that are not its own: the next unit's products
            // (which wait for P of its first tiles), sums and flags come after this point.
            tc_fence_before();
            if (s.split || !whole) all_sync();
            else stream_sync();
        } while (next_unit(p, sh, u, unit0));
    } else {
        // -------------------------------------------------------------- conversion
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegConv));
        if constexpr (S::kQuant) {
            using Ring = typename S::Ring;
            const int r = threadIdx.x & 127, kv = warp >= 24;  // row (key) of the tile; keys or values
            uint32_t it = kv, tiles = 0;
            bool ok = true;
            do {
                int tile, end;
                unit_share(p, sh, u, unit0, tile, end);
                for (; tile < end; ++tile, ++tiles, it += 2) {
                    const int key = (u.tile0 + tile) * kTk + r;
                    const bool seen = key >= u.key0 && key < u.key1;
                    const int sl = it % kSlots, rw = Ring::slot(it);
                    if (ok) ok = mbar_wait(bar(S::kBarRawF + Ring::full(it)), Ring::full_parity(it), abort_flag, hdr);
                    if (ok) ok = mbar_wait(bar(S::kBarEmpty + sl), ((it / kSlots) & 1) ^ 1, abort_flag, hdr);
                    const uint8_t* raw = smem + S::kOffRaw + rw * S::kRawB + r * S::kRowB;
                    uint8_t* slot = smem + S::kOffKv + sl * S::kTileB + r * 128;
                    const int sw = S::kBoxB == 128 ? r & 7 : S::kBoxB == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
                    // the keys' scales take the call's along (its size, and not 0: see the streams); nobody's
                    // key may have anything in its slot
                    float* scale = reinterpret_cast<float*>(smem + S::kOffSc + (tiles % S::kScSlots) * S::kScB) + kv * kTk + r;
                    if (!kv) *scale = seen ? fmaxf(*scale * fabsf(p.scale_log2), 1e-37f) : 1.0f;
                    else if (!seen) *scale = 0.0f;
                    constexpr int kIn = S::kRowB / 16, kAt = kIn < 4 ? kIn : 4;  // 16-byte chunks of codes: of a row, at a time
                    constexpr int kPer = FMT == kKvE4m3 ? 2 : 4;                 // output chunks of an input chunk
#pragma unroll 1
                    for (int c0 = 0; c0 < kIn; c0 += kAt) {
                        uint4 in4[kAt];
#pragma unroll
                        for (int c = 0; c < kAt; ++c)
                            in4[c] = seen ? *reinterpret_cast<const uint4*>(raw + (((c0 + c) ^ sw) << 4)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int c = 0; c < kAt; ++c) {
                            const uint32_t in[4] = {in4[c].x, in4[c].y, in4[c].z, in4[c].w};
#pragma unroll
                            for (int k = 0; k < kPer; ++k) {
                                uint4 o;
                                if constexpr (FMT == kKvE4m3)
                                    o = make_uint4(e4m3_two(in[2 * k], false), e4m3_two(in[2 * k], true),
                                                   e4m3_two(in[2 * k + 1], false), e4m3_two(in[2 * k + 1], true));
                                else
                                    o = make_uint4(int4_two(in[k], 0), int4_two(in[k], 1), int4_two(in[k], 2), int4_two(in[k], 3));
                                const int oc = (c0 + c) * kPer + k;
                                *reinterpret_cast<uint4*>(slot + (oc / 8) * (128 * 128) + (((oc & 7) ^ (r & 7)) << 4)) = o;
                            }
                        }
                    }
                    fence_async();
                    __syncwarp();
                    // (nothing is handed on after an abort: codes that never came must not be asked for a
                    // second time while their barrier's phase is open)
                    if (lane == 0 && ok) {
                        mbar_arrive(bar(S::kBarFull + sl));
                        mbar_arrive(bar(S::kBarRawE + rw));
                    }
                }
            } while (next_unit(p, sh, u, unit0));
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int FMT, int D>
cudaError_t launch(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, float* part,
                   unsigned* counters, cudaStream_t st) {
    using S = TilesShape<FMT, D>;
    AttnParams p;
    p.a = a;
    const int G = a.d.H / a.d.H_kv;
    p.c.hg = G;
    p.c.tq = 2 * (kTileRows / G);
    p.c.subs = 1;
    p.c.hs = a.d.H_kv;
    p.c.tk_log2 = 7;
    p.c.page_log2 = __builtin_ctz(a.d.page);
    // (a 2048-token chunk and a mixed batch take 57.4 and 48.2 us at 2, 56.9 and 48.0 at 3, 57.4 and 47.9 at 4, 60.4
    // and 48.1 at 6)
    p.c.unit_cost = 3;
    p.c.min_share = 4;
    p.c.rows_lo = rows_lo;
    p.c.rows_hi = rows_hi;
    p.part = part;
    p.counters = counters;
    p.scale_log2 = a.scale * kLog2e;
    if (!make_kv_map(&p.tm_k, a.cache.k, a, S::kBoxB, std::min(a.d.page, kTk)) ||
        !make_kv_map(&p.tm_v, a.cache.v, a, S::kBoxB, std::min(a.d.page, kTk)))
        return cudaErrorInvalidValue;
    {
        // queries {D, H, T}; one token needs no token stride
        const int64_t ld = a.d.T > 1 ? a.ldq : (int64_t)a.d.H * D;
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.d.H, (cuuint64_t)a.d.T};
        const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kTileRows / G)};
        if (!make_map_nd(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    const void* kern = reinterpret_cast<const void*>(&attn_tiles_kernel<FMT, D>);
    cudaError_t e = ensure_dynamic_smem(kern, S::kSmem);
    if (e != cudaSuccess) return e;
    // the streams' register share is drawn from what the launch holds: check it once
    static std::atomic<int> regs{0};
    if (!regs.load(std::memory_order_relaxed)) {
        cudaFuncAttributes at{};
        if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
        regs.store(at.numRegs, std::memory_order_relaxed);
    }
    const int need = S::kRegCtl + 4 * S::kRegStream + (S::kQuant ? 2 * S::kRegConv : 0);
    if (need * 128 > regs.load(std::memory_order_relaxed) * S::kThreads) return cudaErrorInvalidConfiguration;
    attn_tiles_kernel<FMT, D><<<sm_count(), S::kThreads, S::kSmem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attn_tiles_part_bytes(const moe_kv_dims_t& d) {
    return (size_t)kPartSlots * sm_count() * 2 * (kTileRows * d.D + 2 * kTileRows) * sizeof(float);
}

cudaError_t launch_attn_tiles(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, float* part,
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
