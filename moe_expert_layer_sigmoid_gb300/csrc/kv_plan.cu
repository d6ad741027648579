// Page planning: block tables and slot maps from request lengths.
//
// Three exclusive sums over the batch (pages given back, then tokens and pages of the
// sequences that can be served) place everything; what follows is a copy of ids, and a
// search in the sums for each token.  The bytes are few (8 per token): a call is a launch, the state's
// latency and the sums' (3.5 us for 32 sequences and a token each).  So it is one launch, of one CTA or, where tokens are many,
// of one cluster whose CTAs all make the same sums (the batch's lengths are a few KB) and share
// the copies and the tokens: nothing is handed from one CTA to another but the state itself, behind
// two cluster barriers.  No result depends on timing.
#include "kv.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;  // of a CTA, at most
constexpr int kRun = 4;            // neighbouring tokens of a thread

struct PlanParams {
    const int32_t* new_len;
    moe_kv_pages_t st;
    int32_t *q_off, *pos, *slots;
    WsHeader* hdr;
    int T, B, page_log2, n_pages, max_pages, window;
};

// One sequence's step, before it is known whether there is room.
struct Step {
    int after;       // its tokens before the new ones
    int first;       // the first page it holds from now on
    int lo, hi;      // entries whose pages go back
    int want, need;  // tokens and pages asked for
};

__device__ __forceinline__ int pages_of(int tokens, int lg) {
    return (int)(((unsigned)tokens + (1u << lg) - 1) >> lg);
}

__device__ __forceinline__ Step step_of(const PlanParams& p, int b, bool& bad) {
    const int n = p.new_len[b], L = p.st.kv_len[b], f = p.st.first[b];
    Step s{L, f, 0, 0, 0, 0};
    const int64_t most = (int64_t)p.max_pages << p.page_log2;
    if (L < 0 || L > most || f < 0 || f > pages_of(L, p.page_log2)) {
        bad = true;
        return s;
    }
    if (n < 0) {
        const int64_t left = (int64_t)L + n;
        const int after = left > 0 ? (int)left : 0;
        // the window's last keys went back with their pages: a shorter sequence would need some again
        if (after > 0 && ((int64_t)f << p.page_log2) > max(0, after - p.window + 1)) {
            bad = true;
            return s;
        }
        s.after = after;
        s.first = after > 0 ? f : 0;
        s.lo = max(pages_of(after, p.page_log2), f);
        s.hi = pages_of(L, p.page_log2);
        return s;
    }
    if (n > most - L) {
        bad = true;
        return s;
    }
    if (p.window > 0) s.first = max(f, max(0, L - p.window + 1) >> p.page_log2);
    s.lo = f;
    s.hi = s.first;
    s.want = n;
    s.need = pages_of(L + n, p.page_log2) - pages_of(L, p.page_log2);
    return s;
}

struct Sums {
    int64_t a, b, c;
};

// Inclusive sums over the warp's lanes.
__device__ __forceinline__ Sums warp_sums(Sums x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xFFFFFFFFu, x.a, o), b = __shfl_up_sync(0xFFFFFFFFu, x.b, o),
                      c = __shfl_up_sync(0xFFFFFFFFu, x.c, o);
        if (lane >= o) {
            x.a += a;
            x.b += b;
            x.c += c;
        }
    }
    return x;
}
__device__ __forceinline__ Sums of_lane(Sums x, int lane) {
    return Sums{__shfl_sync(0xFFFFFFFFu, x.a, lane), __shfl_sync(0xFFFFFFFFu, x.b, lane),
                __shfl_sync(0xFFFFFFFFu, x.c, lane)};
}

// Exclusive sums over the CTA's threads; `total` gets the sums of all.  (Each warp sums the warps' sums again, by lanes: one by
// one they were half of a call for 500 sequences.)
__device__ __forceinline__ Sums scan(Sums v, Sums* part, Sums& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const Sums x = warp_sums(v);
    __syncthreads();  // (the sums of an earlier scan have been read)
    if (lane == 31) part[warp] = x;
    __syncthreads();
    const Sums all = warp_sums(lane < warps ? part[lane] : Sums{0, 0, 0});
    total = of_lane(all, 31);
    const Sums before = of_lane(all, max(warp - 1, 0));
    Sums r{x.a - v.a, x.b - v.b, x.c - v.c};
    if (warp > 0) {
        r.a += before.a;
        r.b += before.b;
        r.c += before.c;
    }
    return r;
}

// The last b of [0, B) with off[b] <= i, off ascending from 0.
__device__ __forceinline__ int find(const int32_t* off, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// All CTAs of the launch (one cluster), their writes to global memory visible to each other.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
    extern __shared__ int32_t smem[];
    __shared__ Sums part[kPlanThreads / 32];
    int32_t* after = smem;             // [B] tokens before the new ones
    int32_t* held = after + p.B;       // [B] the first page held from now on
    int32_t* q_off = held + p.B;       // [B] first row (while summing: tokens asked for)
    int32_t* given = q_off + p.B;      // [B] first of the new pages in the order of taking (pages asked for)
    int32_t* back = given + p.B;       // [B] first of the returned pages in their list
    int32_t* lo = back + p.B;          // [B] entry of that page
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    const int kept = p.st.n_free[0];
    int errors = 0;
    // all CTAs' writes to the state visible to each other
    auto barrier = [&]() {
        __syncthreads();
        if (gridDim.x > 1) cluster_barrier();
    };

    Sums mine{0, 0, 0}, all;
    for (int b = b0; b < b1; ++b) {
        bool bad = false;
        const Step s = step_of(p, b, bad);
        if (bad) errors |= kErrBadSeq;
        after[b] = s.after;
        held[b] = s.first;
        q_off[b] = s.want;
        given[b] = s.need;
        back[b] = s.hi - s.lo;
        lo[b] = s.lo;
        mine.a += s.want;
        mine.b += s.need;
        mine.c += s.hi - s.lo;
    }
    Sums at = scan(mine, part, all);
    const int had = min(max(kept, 0), p.n_pages);
    const int returned = (int)min(all.c, (int64_t)(1 << 30));  // (of a state that is whole: at most n_pages)
    const int total = (int)min((int64_t)had + returned, (int64_t)p.n_pages);
    if (had != kept || had + (int64_t)returned > p.n_pages) errors |= kErrBadPage;
    int64_t gone = at.c;
    for (int b = b0; b < b1; ++b) {
        const int n = back[b];
        back[b] = (int)min(gone, (int64_t)(1 << 30));
        gone += n;
    }
    if (all.a > p.T || all.b > total) {
        // not all can be served: those that can are summed anew
        mine = Sums{0, 0, 0};
        for (int b = b0; b < b1; ++b) {
            const int want = q_off[b], need = given[b];
            at.a += want;
            at.b += need;
            if (at.a <= p.T && (need == 0 || at.b <= total)) {
                mine.a += want;
                mine.b += need;
            } else {
                if (want) errors |= kErrNoRoom;
                q_off[b] = given[b] = 0;
            }
        }
        at = scan(mine, part, all);
    }
    const int tokens = (int)all.a, taken = (int)all.b;
    for (int b = b0; b < b1; ++b) {
        const int want = q_off[b], need = given[b];
        q_off[b] = (int)at.a;
        given[b] = (int)at.b;
        at.a += want;
        at.b += need;
    }
    // Every CTA has read the state; now it changes.  (Entries that go back are read behind the barrier too, but
    // each by the one thread that then clears it.)
    barrier();

    const int threads = gridDim.x * blockDim.x, me = blockIdx.x * blockDim.x + threadIdx.x;
    for (int r = me; r < returned; r += threads) {
        const int b = find(back, p.B, r);
        int32_t* e = p.st.pages + (int64_t)b * p.max_pages + lo[b] + (r - back[b]);
        const int to = had + returned - 1 - r;
        if (to < p.n_pages) p.st.free_pages[to] = *e;
        *e = -1;
    }
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const int row = q_off[b], next = b + 1 < p.B ? q_off[b + 1] : tokens;
            p.q_off[b] = row;
            p.st.kv_len[b] = after[b] + (next - row);
            p.st.first[b] = held[b];
        }
        if (threadIdx.x == 0) {
            p.q_off[p.B] = tokens;
            p.st.n_free[0] = total - taken;
        }
        if (errors) record_error(p.hdr, errors);
    }
    if (returned > 0) barrier();
    for (int r = me; r < taken; r += threads) {
        const int b = find(given, p.B, r);
        p.st.pages[(int64_t)b * p.max_pages + pages_of(after[b], p.page_log2) + (r - given[b])] =
            p.st.free_pages[total - 1 - r];
    }
    // Rows of tokens, a run of neighbours to a thread: one search, then along the sequences; ids are fetched together.
    const int mask = (1 << p.page_log2) - 1;
    const bool wide = (reinterpret_cast<uintptr_t>(p.pos) | reinterpret_cast<uintptr_t>(p.slots)) % 16 == 0;
    for (int64_t t0 = (int64_t)me * kRun; t0 < p.T; t0 += (int64_t)threads * kRun) {
        int pos[kRun], id[kRun], slot[kRun];
        const int t = (int)t0;
        int b = t < tokens ? find(q_off, p.B, t) : p.B, end = t < tokens ? (b + 1 < p.B ? q_off[b + 1] : tokens) : 0;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            pos[i] = -1;
            const int32_t* from = p.st.n_free;  // (read for nothing where there is no token)
            if (t + i < tokens) {
                while (t + i >= end) {
                    ++b;
                    end = b + 1 < p.B ? q_off[b + 1] : tokens;
                }
                pos[i] = after[b] + (t + i - q_off[b]);
                const int entry = pos[i] >> p.page_log2, fresh = entry - pages_of(after[b], p.page_log2);
                from = fresh < 0 ? p.st.pages + (int64_t)b * p.max_pages + entry
                                 : p.st.free_pages + (total - 1 - (given[b] + fresh));
            }
            id[i] = *from;
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            slot[i] = -1;
            if (pos[i] >= 0) {
                if ((unsigned)id[i] < (unsigned)p.n_pages) slot[i] = (id[i] << p.page_log2) + (pos[i] & mask);
                else record_error(p.hdr, kErrBadPage);
            }
        }
        if (wide && t0 + kRun <= p.T) {
            *reinterpret_cast<int4*>(p.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                if (t0 + i < p.T) {
                    p.pos[t0 + i] = pos[i];
                    p.slots[t0 + i] = slot[i];
                }
        }
    }
}

}  // namespace

cudaError_t launch_kv_plan(const int32_t* new_len, const moe_kv_dims_t& d, const moe_kv_pages_t& st,
                           int32_t* q_off, int32_t* pos, int32_t* slots, WsHeader* hdr, cudaStream_t stream) {
    const PlanParams p{new_len, st, q_off, pos, slots, hdr, d.T, d.B, __builtin_ctz(d.page), d.n_pages,
                       d.max_pages, d.window};
    const size_t smem = 6 * sizeof(int32_t) * (size_t)d.B;
    cudaError_t err = ensure_dynamic_smem((const void*)kv_plan_kernel, smem + 1024);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    // One CTA, as large as the batch, or a cluster of eight where tokens are many (1 and 8 CTAs, us for two calls: 1600
    // tokens of 8 sequences 8.6, 10.1; 4000 of 20 12.1, 10.4; 35000 of 60 56, 15.5).
    const int rows = d.T / kRun + (d.T % kRun != 0);  // (T may be 2^31 - 1)
    cfg.gridDim = dim3(rows > 512 ? 8 : 1);
    cfg.blockDim = dim3(std::max(d.B, rows) <= 128 ? 128 : std::max(d.B, rows) <= 2048 ? 512 : kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cfg.gridDim.x;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, p);
}

}  // namespace moe
