// Shared by the attention kernels: how a call's work is cut into tiles and
// dealt to CTAs on the device, and the join of partial results.
//
// The unit is one (sequence, row tile, head slot): a row tile is `tq`
// consecutive new tokens of the sequence, a head slot the query heads of one
// key/value head that share a tile (row r of the tile is token r / hg, head
// r % hg of the slot).  A unit walks the tiles of `tk` keys that its rows see.
// The units' tiles, in the order sequence, row tile, head slot, key tile, form
// one line of W tiles; CTA c of R takes tiles [c W / R, (c + 1) W / R).  So every
// CTA gets the same share of keys whatever the lengths are, and a unit cut by
// a border is joined from its CTAs' partial results (running maximum, sum and
// unnormalised output).  A CTA leaves at most two partials: of the unit it
// starts in the middle of, and of the unit it ends in the middle of, so the
// workspace does not grow with the batch.  The CTA that arrives last at a unit
// joins it, in CTA order, so the result does not depend on who is last.
// Lengths are read on the device only: a captured call follows them.
#pragma once

#include "kv.cuh"
#include "tma.cuh"

namespace moe {

constexpr float kNoMax = -3.402823466e38f;  // running maximum before any key
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How a kernel cuts the call (host side constants of one launch).
struct AttnCut {
    int tq;        // tokens per row tile
    int hg;        // query heads per head slot
    int subs;      // head slots per key/value head
    int hs;        // head slots: H_kv * subs
    int tk_log2;   // keys per tile
    int page_log2;
    int min_tiles;  // fewest tiles that a CTA is worth starting for
    // sequences with rows_lo < n * (H / H_kv) <= rows_hi are this launch's
    int64_t rows_lo, rows_hi;
};

struct AttnParams {
    CUtensorMap tm_k, tm_v;
    CUtensorMap tm_q;     // the tcgen05 kernel's
    AttnArgs a;
    AttnCut c;
    float* part;          // partial results, two slots for each CTA
    unsigned* counters;   // arrivals, one for each CTA
    float scale_log2;     // scale * log2(e)
};

// A unit's place and keys.
struct Unit {
    int b, rt, hs;
    int n, len, tok0;   // sequence: new tokens, length, first token's row
    int key0, key1;     // keys that its rows see: [key0, key1), empty if key1 <= key0
    int tile0, tiles;   // key tiles: [tile0, tile0 + tiles), at least one
};

// Sequence b's new tokens and length; n = 0 for one that is not this launch's.
__device__ __forceinline__ void load_seq(const AttnParams& p, int b, int& tok0, int& n, int& len) {
    tok0 = __ldg(p.a.q_off + b);
    const int t1 = __ldg(p.a.q_off + b + 1);
    len = __ldg(p.a.kv_len + b);
    n = t1 - tok0;
    if (tok0 < 0 || n < 0 || t1 > p.a.d.T || len < 0 ||
        (int64_t)len > ((int64_t)p.a.d.max_pages << p.c.page_log2)) {
        if (n != 0) record_error(p.a.hdr, kErrBadSeq);
        n = 0;
    }
    const int64_t rows = (int64_t)n * (p.a.d.H / p.a.d.H_kv);
    if (rows <= p.c.rows_lo || rows > p.c.rows_hi) n = 0;
}

__device__ __forceinline__ void unit_keys(const AttnParams& p, Unit& u) {
    const int i0 = u.rt * p.c.tq, i1 = min(u.n, i0 + p.c.tq) - 1;
    u.key1 = max(0, u.len - u.n + i1 + 1);
    u.key0 = p.a.d.window ? max(0, u.len - u.n + i0 - p.a.d.window + 1) : 0;
    u.tile0 = u.key0 >> p.c.tk_log2;
    u.tiles = max(1, (int)(((int64_t)u.key1 + (1 << p.c.tk_log2) - 1) >> p.c.tk_log2) - u.tile0);
}

__device__ __forceinline__ int row_tiles(const AttnParams& p, int n) {
    return (n + p.c.tq - 1) / p.c.tq;
}

// Tiles of one sequence, over its row tiles and one head slot.
__device__ __forceinline__ int64_t seq_tiles(const AttnParams& p, int n, int len) {
    int64_t s = 0;
    Unit u;
    u.n = n;
    u.len = len;
    const int rts = row_tiles(p, n);
    for (u.rt = 0; u.rt < rts; ++u.rt) {
        unit_keys(p, u);
        s += u.tiles;
    }
    return s;
}

// A CTA's share and its first unit.
struct Share {
    int64_t W;        // tiles of the launch
    int64_t w0, w1;   // this CTA's
    int64_t unit0;    // index of the first unit's first tile
    int R;            // CTAs that take part
    Unit u;           // the first unit
};

__device__ __forceinline__ int64_t share_start(int64_t W, int R, int c) { return (W * c) / R; }
// The CTA that holds tile w.
__device__ __forceinline__ int share_owner(int64_t W, int R, int64_t w) {
    return (int)(((w + 1) * R - 1) / W);
}

// Every thread of the CTA calls this; `sm` is scratch of (threads / 32 + 4) int64.
// Sums the sequences' tiles in order (each thread a run of sequences), deals
// the line and finds the unit that holds this CTA's first tile.
template <int THREADS>
__device__ Share deal(const AttnParams& p, int64_t* sm) {
    constexpr int kWarps = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = p.a.d.B, per = (B + THREADS - 1) / THREADS;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        int tok0, n, len;
        load_seq(p, b, tok0, n, len);
        mine += n ? seq_tiles(p, n, len) * p.c.hs : 0;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    int64_t before = 0, W = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += sm[i];
        W += sm[i];
    }
    before += incl - mine;
    Share s;
    s.W = W;
    s.R = (int)min((int64_t)gridDim.x, max((int64_t)1, W / p.c.min_tiles));
    const bool idle = (int)blockIdx.x >= s.R || W == 0;
    s.w0 = idle ? 0 : share_start(W, s.R, blockIdx.x);
    s.w1 = idle ? 0 : share_start(W, s.R, blockIdx.x + 1);
    if (!idle && s.w0 >= before && s.w0 < before + mine) {
        for (int b = b0; b < b1; ++b) {
            int tok0, n, len;
            load_seq(p, b, tok0, n, len);
            const int64_t t = n ? seq_tiles(p, n, len) * p.c.hs : 0;
            if (s.w0 < before + t) {
                sm[kWarps] = b;
                sm[kWarps + 1] = before;
                break;
            }
            before += t;
        }
    }
    __syncthreads();
    if (!idle) {
        Unit& u = s.u;
        u.b = (int)sm[kWarps];
        int64_t at = sm[kWarps + 1];
        load_seq(p, u.b, u.tok0, u.n, u.len);
        for (u.rt = 0;; ++u.rt) {
            unit_keys(p, u);
            const int64_t t = (int64_t)u.tiles * p.c.hs;
            if (s.w0 < at + t || u.rt + 1 >= row_tiles(p, u.n)) break;
            at += t;
        }
        u.hs = (int)((s.w0 - at) / u.tiles);
        s.unit0 = at + (int64_t)u.hs * u.tiles;
    }
    return s;
}

// The unit after u (which is not the launch's last).
__device__ __forceinline__ void next_unit(const AttnParams& p, Unit& u) {
    if (++u.hs < p.c.hs) return;
    u.hs = 0;
    if (++u.rt >= row_tiles(p, u.n)) {
        u.rt = 0;
        do {
            if (++u.b >= p.a.d.B) return;
            load_seq(p, u.b, u.tok0, u.n, u.len);
        } while (u.n == 0);
    }
    unit_keys(p, u);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The map of a pool's rows: {row, slots of a page, heads, pages}, boxes of
// `box_bytes` x `box_rows`.
bool make_kv_map(CUtensorMap* m, const void* base, const AttnArgs& a, int box_bytes, int box_rows);

// Launchers.  `part` and `counters` lie in the workspace; the counters are zero
// between calls.
size_t attn_rows_part_bytes(const moe_kv_dims_t& d);
cudaError_t launch_attn_rows(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, float* part,
                             unsigned* counters, cudaStream_t st);
size_t attn_tiles_part_bytes(const moe_kv_dims_t& d);
cudaError_t launch_attn_tiles(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, float* part,
                              unsigned* counters, cudaStream_t st);

}  // namespace moe
