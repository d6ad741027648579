// Shared by the attention kernels: how a call's work is cut into tiles and
// dealt to CTAs on the device, and the join of partial results.
//
// The unit is one (sequence, row tile, head slot): a row tile is `tq`
// consecutive new tokens of the sequence, a head slot the query heads of one
// key/value head that share a tile (row r of the tile is token r / hg, head
// r % hg of the slot).  A unit walks the tiles of `tk` keys that its rows see.
// The units, in the order sequence, row tile, head slot, form one line of
// length W: each takes `unit_cost` places (what a unit costs besides its
// tiles, in tiles) and then one place for each key tile; CTA c of R takes the
// places [c W / R, (c + 1) W / R).  So every CTA gets the same share whatever
// the lengths are, and a unit cut by a border is joined from its CTAs' partial
// results (running maximum, sum and unnormalised output).  A CTA leaves at most
// two partials: of the unit it starts in the middle of, and of the unit it ends
// in the middle of, so the workspace does not grow with the batch.  The CTA
// that arrives last at a unit joins it, in CTA order, so the result does not
// depend on who is last.  Lengths are read on the device only: a captured call
// follows them.
#pragma once

#include "attn_index.h"
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
    int unit_cost;  // places of a unit besides its tiles
    int min_share;  // fewest places that a CTA is worth starting for
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
    n = 0;
    if (seq_ok(tok0, t1, len, p.a.d.T, (int64_t)p.a.d.max_pages << p.c.page_log2)) n = t1 - tok0;
    else if (t1 != tok0) record_error(p.a.hdr, kErrBadSeq);
    const int64_t rows = (int64_t)n * (p.a.d.H / p.a.d.H_kv);
    if (rows <= p.c.rows_lo || rows > p.c.rows_hi) n = 0;
}

__device__ __forceinline__ void unit_keys(const AttnParams& p, Unit& u) {
    const int i0 = u.rt * p.c.tq, i1 = min(u.n, i0 + p.c.tq) - 1;
    u.key1 = max(0, u.len - u.n + i1 + 1);
    u.key0 = first_key(u.len - u.n + i0, p.a.d.window);
    u.tile0 = u.key0 >> p.c.tk_log2;
    u.tiles = max(1, tiles_until(u.key1, p.c.tk_log2) - u.tile0);
}

__device__ __forceinline__ int row_tiles(const AttnParams& p, int n) {
    return (n + p.c.tq - 1) / p.c.tq;
}

// A CTA's share and its first unit.
struct Share {
    int64_t W;        // places of the launch
    int64_t w0, w1;   // this CTA's
    int64_t unit0;    // the first unit's first place
    int R;            // CTAs that take part
    Unit u;           // the first unit
};

// The CTA that holds place w.
__device__ __forceinline__ int share_owner(int64_t W, int R, int64_t w) {
    const int64_t n = (w + 1) * R - 1;
    return (int)(n >> 32 == 0 && W >> 32 == 0 ? (uint32_t)n / (uint32_t)W : n / W);
}

// Inclusive scan over the CTA; `sm` holds a value for each warp.
template <int THREADS, class T>
__device__ __forceinline__ T cta_scan(T x, T* sm, T& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T v = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += v;
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    total = 0;
    T before = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) before += sm[i];
        total += sm[i];
    }
    return before + x;
}

// Every thread of the CTA calls deal(); `scratch` is 8-aligned, of deal_bytes(THREADS), and nothing
// else uses it until the CTA's next __syncthreads.  Sums the places of the sequences, deals the line and
// finds the unit that holds this CTA's first place.  Everything a CTA does waits for it, and its code
// is cold when it runs, so the common cases (a sequence per thread at most, a line that 32 bits hold,
// and few row tiles per sequence or no more in all than threads) are kept short; deal_many is for
// the others (a 2048-token chunk waited 12,300 cycles for it; 160 decode sequences of 1638 E4M3 keys
// take 102.6 us, 161 of 1628 take 107.4).
constexpr int deal_bytes(int threads) { return 8 * (2 * (threads / 32) + 8) + 16 * threads; }

// The share of the line and its first unit, from the found one's first place of its row tile.
__device__ __forceinline__ void put_found(const AttnParams& p, int64_t* found, Unit& u, int64_t before, int64_t w0) {
    const int each = u.tiles + p.c.unit_cost;
    const int64_t off = w0 - before;
    u.hs = (int)(off >> 31 == 0 ? (uint32_t)off / (uint32_t)each : off / each);
    found[0] = before + (int64_t)u.hs * each;
    int* f = reinterpret_cast<int*>(found + 1);
    f[0] = u.b, f[1] = u.rt, f[2] = u.hs, f[3] = u.n, f[4] = u.len, f[5] = u.tok0;
}
__device__ __forceinline__ void get_found(const AttnParams& p, const int64_t* found, Share& s) {
    const int* f = reinterpret_cast<const int*>(found + 1);
    s.unit0 = found[0];
    s.u.b = f[0], s.u.rt = f[1], s.u.hs = f[2], s.u.n = f[3], s.u.len = f[4], s.u.tok0 = f[5];
    unit_keys(p, s.u);
}

// Any lengths: each thread a run of sequences to count the row tiles, then a run of row tiles to count
// the places.
template <int THREADS>
__device__ __noinline__ void deal_many(const AttnParams& p, int64_t* sm) {
    constexpr int kWarps = THREADS / 32;
    int* smr = reinterpret_cast<int*>(sm + kWarps);  // row tiles by warp
    int64_t* found = sm + 2 * kWarps;
    int* first = reinterpret_cast<int*>(found + 8);  // [threads]: row tiles before each thread's sequences
    const int tid = threadIdx.x, B = p.a.d.B, per = (B + THREADS - 1) / THREADS;
    Unit u;
    int rts = 0, n_rt;
    for (u.b = min(B, tid * per); u.b < min(B, tid * per + per); ++u.b) {
        load_seq(p, u.b, u.tok0, u.n, u.len);
        rts += row_tiles(p, u.n);
    }
    __syncthreads();
    first[tid] = cta_scan<THREADS>(rts, smr, n_rt) - rts;
    __syncthreads();
    const int pe = (n_rt + THREADS - 1) / THREADS, e0 = min(n_rt, tid * pe), e1 = min(n_rt, e0 + pe);
    int k = 0;  // the thread whose run of sequences has row tile e0
#pragma unroll 1
    for (int step = 512; step; step >>= 1)
        if (k + step < THREADS && first[k + step] <= e0) k += step;
    auto seek = [&] {  // u to row tile e0
        u.b = k * per;
        u.rt = e0 - first[k];
        load_seq(p, u.b, u.tok0, u.n, u.len);
        for (int r; u.rt >= (r = row_tiles(p, u.n));) {
            u.rt -= r;
            load_seq(p, ++u.b, u.tok0, u.n, u.len);
        }
    };
    auto step = [&] {
        if (++u.rt < row_tiles(p, u.n)) return;
        u.rt = 0;
        do {
            if (++u.b >= B) return;
            load_seq(p, u.b, u.tok0, u.n, u.len);
        } while (u.n == 0);
    };
    auto places = [&] {
        unit_keys(p, u);
        return (int64_t)(u.tiles + p.c.unit_cost) * p.c.hs;
    };
    int64_t mine = 0, W;
    if (e0 < e1) {
        seek();
        for (int e = e0;;) {
            mine += places();
            if (++e == e1) break;
            step();
        }
    }
    int64_t before = cta_scan<THREADS>(mine, sm, W) - mine;
    const int R = (int)min((int64_t)gridDim.x, max((int64_t)1, W / p.c.min_share));
    const bool idle = (int)blockIdx.x >= R || W == 0;
    const int64_t w0 = idle ? 0 : W * blockIdx.x / R;
    if (tid == 0) {
        found[4] = W;
        found[5] = R;
        found[6] = w0;
        found[7] = idle ? 0 : W * (blockIdx.x + 1) / R;
    }
    if (!idle && w0 >= before && w0 < before + mine) {
        seek();
        for (int64_t t; w0 >= before + (t = places());) {
            before += t;
            step();
        }
        put_found(p, found, u, before, w0);
    }
    __syncthreads();
}

template <int THREADS>
__device__ __forceinline__ Share deal(const AttnParams& p, void* scratch) {
    constexpr int kWarps = THREADS / 32;
    constexpr int kFew = 4;  // row tiles of a sequence that its thread may count alone
    int64_t* sm = static_cast<int64_t*>(scratch);
    int64_t* found = sm + 2 * kWarps;
    const int B = p.a.d.B;
    Share s;
    Unit& u = s.u;
    u.b = threadIdx.x;
    u.n = 0;
    if (u.b < B) load_seq(p, u.b, u.tok0, u.n, u.len);
    const int rts = row_tiles(p, u.n);
    uint64_t sum = 0;
    bool long_ = B > THREADS || rts > kFew;
    if (!long_)
#pragma unroll 1
        for (u.rt = 0; u.rt < rts; ++u.rt) {
            unit_keys(p, u);
            sum += (uint64_t)(u.tiles + p.c.unit_cost) * (unsigned)p.c.hs;
        }
    long_ |= sum >= 1u << 22;  // (below it no sum over the CTA passes 32 bits)
    unsigned mine = (unsigned)sum;
    unsigned W = 0, before = 0;
    bool many = __syncthreads_or(long_), each = false;  // each: a thread has one row tile, u
    if (!many) {
        before = cta_scan<THREADS>(mine, reinterpret_cast<unsigned*>(sm), W) - mine;
    } else if (B <= THREADS) {
        int n_rt;
        int4* seqs = reinterpret_cast<int4*>(found + 8);  // n, length, first token, row tiles before
        const int e = threadIdx.x, upto = cta_scan<THREADS>(rts, reinterpret_cast<int*>(sm + kWarps), n_rt);
        if (n_rt <= THREADS) {
            seqs[e] = make_int4(u.n, u.len, u.tok0, upto - rts);
            __syncthreads();
            u.n = 0;
            mine = 0;
            if (e < n_rt) {
                int lo = 0;
#pragma unroll 1
                for (int hi = B; hi - lo > 1;) {
                    const int mid = (lo + hi) >> 1;
                    if (seqs[mid].w <= e) lo = mid;
                    else hi = mid;
                }
                const int4 q = seqs[lo];
                u.b = lo;
                u.n = q.x, u.len = q.y, u.tok0 = q.z;
                u.rt = e - q.w;
                unit_keys(p, u);
                sum = (uint64_t)(u.tiles + p.c.unit_cost) * (unsigned)p.c.hs;
                mine = (unsigned)sum;
            }
            many = __syncthreads_or(e < n_rt && sum >= 1u << 22);
            each = true;
            if (!many) before = cta_scan<THREADS>(mine, reinterpret_cast<unsigned*>(sm), W) - mine;
        }
    }
    many |= W >= 1u << 22;  // W * R in 32 bits, up to 1024 CTAs
    if (many) {
        deal_many<THREADS>(p, sm);
        s.W = found[4];
        s.R = (int)found[5];
        s.w0 = found[6];
        s.w1 = found[7];
        get_found(p, found, s);
        return s;
    }
    s.W = W;
    const unsigned R = min(gridDim.x, max(1u, W / (unsigned)p.c.min_share));
    s.R = R;
    s.w0 = s.w1 = s.unit0 = 0;
    if (blockIdx.x >= R || W == 0) return s;
    const unsigned w0 = W * blockIdx.x / R;
    s.w0 = w0;
    s.w1 = (W * blockIdx.x + W) / R;
    if (w0 >= before && w0 < before + mine) {
        if (!each)
            for (u.rt = 0;; ++u.rt) {
                unit_keys(p, u);
                const unsigned t = (unsigned)(u.tiles + p.c.unit_cost) * (unsigned)p.c.hs;
                if (w0 < before + t) break;
                before += t;
            }
        put_found(p, found, u, before, w0);
    }
    __syncthreads();
    get_found(p, found, s);
    return s;
}

// The tiles [t0, t1) of unit u (whose first place is unit0) that are in this CTA's share.
__device__ __forceinline__ void unit_share(const AttnParams& p, const Share& s, const Unit& u,
                                           int64_t unit0, int& t0, int& t1) {
    const int64_t at = unit0 + p.c.unit_cost;
    t0 = (int)max((int64_t)0, s.w0 - at);
    t1 = (int)max((int64_t)0, min((int64_t)u.tiles, s.w1 - at));
}

// Moves u and unit0 on; false if no tile of the next unit is in the share.
__device__ __forceinline__ bool next_unit(const AttnParams& p, const Share& s, Unit& u, int64_t& unit0) {
    unit0 += u.tiles + p.c.unit_cost;
    if (unit0 + p.c.unit_cost >= s.w1) return false;
    if (++u.hs < p.c.hs) return true;
    u.hs = 0;
    if (++u.rt >= row_tiles(p, u.n)) {
        u.rt = 0;
        do {
            if (++u.b >= p.a.d.B) return false;
            load_seq(p, u.b, u.tok0, u.n, u.len);
        } while (u.n == 0);
    }
    unit_keys(p, u);
    return true;
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
// `eight`: units of eight rows instead of sixteen (at most eight query heads per key/value head).
// `behind`: launched right behind launch_attn_tiles on the same sequences' others: its CTAs may take the
// SMs that the chunks' CTAs leave, and it ends after them.
cudaError_t launch_attn_rows(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, bool eight, bool behind, float* part,
                             unsigned* counters, cudaStream_t st);
size_t attn_tiles_part_bytes(const moe_kv_dims_t& d);
cudaError_t launch_attn_tiles(const AttnArgs& a, int64_t rows_lo, int64_t rows_hi, float* part,
                              unsigned* counters, cudaStream_t st);

}  // namespace moe
