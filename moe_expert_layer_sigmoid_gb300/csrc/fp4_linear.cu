// Projections with both operands in microscaled 4-bit floats: the tensor cores' block-scaled products
// (kind::mxf4nvf4, E2M1 x E2M1 with an E4M3 scale for each 16, fp32 accumulators in TMEM).
//
//   out[t][n] = (sum over blocks of bx bw (sum of 16 code products)) * s_x[t] * s_w[n]
// Code products and block scales meet inside the product, so codes go from memory to the tensor core as they are
// stored; the two row scales are applied once, to the finished sum.
//
// A tile has M = 128 rows of one operand and NT of the other, K in stages of 256 elements: 128 bytes of codes per
// row (TMA, 128-byte swizzle) and, for each 128 rows and 64 elements, 512 bytes of scales, which lie in memory
// in the order that tcgen05.cp spreads over TMEM (lane r % 32 and column r / 32 hold row r's four scales).  Four
// products of K = 64 per stage.  Two forms:
//  - narrow, for few tokens: M are weight rows, NT the smallest of 16, 32, 64 that holds the tokens; one tile per CTA.  What
//    bounds it is the time until the first weights arrive and the joining (16 tokens, N = 6144, K = 4096: 8.5 us with the
//    quantisation's 2.1; the weights are 2.1 us of DRAM time).
//  - wide, NT = 128: M are tokens, so that a lane of the epilogue holds 32 neighbours of an output row.
// A CTA has one tile.  Where wide tiles are more than SMs, pairs of CTAs take over (launch_pair_fp4).
// Where the tiles are too few for the SMs, K is cut among the CTAs of a cluster, which add their sums in
// the order of K through each other's shared memory.
//
// Warps: 0 copies, 1 allocates TMEM and issues the products, 2-9 the epilogue, two per quarter of TMEM's
// lanes.  The scales of a stage have TMEM columns of their own, which are free when the stage's shared memory is.
#include "fp4_mma.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 8, kEpiWarp0 = 2, kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kMaxSplits = 8, kMaxNarrow = 4;  // CTAs of a cluster

template <int NT, bool WIDE>
struct Shape {
    static constexpr int kA = 128 * kRowBytes, kB = NT * kRowBytes;
    static constexpr int kSfA = 4 * kAtom, kSfB = 4 * kAtom;
    static constexpr int kStage = kA + kB + kSfA + kSfB;
    static constexpr int kRoom = (WIDE ? 216 : 108) * 1024;
    static constexpr int kStages = kRoom / kStage < 6 ? kRoom / kStage : 6;
    static constexpr int kSfCols = 32;  // TMEM columns of a stage's scales
    static constexpr int kSfCol0 = NT;
    static constexpr int kTmemCols = WIDE ? 512 : 256;
    // FULL[stages], EMPTY[stages], AFULL (the tile's products are done), TD (those in flight at the end are)
    static constexpr int kFull = 0, kEmpty = kStages, kAFull = 2 * kStages, kTd = kAFull + 1;
    static constexpr int kBarAt = kStages * kStage;
    static constexpr int kMisc = kBarAt + 8 * (kTd + 1);
    static constexpr int kScales = (kMisc + 16 + 15) / 16 * 16;  // row scales of the NT rows (wide)
    static constexpr int kSmem = kScales + (WIDE ? NT * 4 : 0) + 1024;  // + alignment slack
    static_assert(kSmem <= (WIDE ? 227 : 113) * 1024 && kSfCol0 + kStages * kSfCols <= kTmemCols && kStage % 1024 == 0,
                  "");
    static_assert(NT * 128 * 4 <= kStages * kStage, "a tile's sums fit where the stages were");
};

struct LinearParams {
    Side m, n;
    uint16_t* out;
    WsHeader* hdr;
    int64_t ld;  // output channels, N of the call
    int K, splits;
};

struct Unit {
    int m, n;    // tiles of either side
    int k0, k1;  // stages
};
__device__ __forceinline__ Unit unit_of(const LinearParams& p, int u) {
    const int tile = u / p.splits, s = u - tile * p.splits, all = (p.K + kStageK - 1) / kStageK;
    Unit r;
    r.n = tile / p.m.tiles;
    r.m = tile - r.n * p.m.tiles;
    r.k0 = all * s / p.splits;  // (at most 256 * 8)
    r.k1 = all * (s + 1) / p.splits;
    return r;
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }
__device__ __forceinline__ void load_peer4(uint32_t addr, float* v) {
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float load_peer(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int NT, bool WIDE>
__global__ void __launch_bounds__(kThreads, WIDE ? 1 : 2) linear_kernel(const __grid_constant__ LinearParams p) {
    using S = Shape<NT, WIDE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    // (the shuffle tells the compiler that a warp has one number)
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    auto bar = [&](int i) { return sbase + S::kBarAt + 8 * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(bar(S::kFull + s), 1);
            mbar_init(bar(S::kEmpty + s), 1);
        }
        mbar_init(bar(S::kAFull), 1);
        mbar_init(bar(S::kTd), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&p.m.map);
        prefetch_tmap(&p.n.map);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(S::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int atoms = p.K / 64;  // scale atoms of a row tile
    const Unit u = unit_of(p, blockIdx.x);
    const bool shared = !WIDE || p.splits > 1;  // sums go through shared memory

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            // (One thread issues every copy of a stage: what it works out for each of them bounds the loop, so addresses are
            // counted up.)
            const uint32_t withheld = withheld_stage(p.hdr);
            const int last = (atoms + 3) / 4 - 1;  // the last stage of K, and its bytes of scales per 128 rows
            const uint32_t last_bytes = (atoms - 4 * last) * kAtom;
            uint32_t it = 0;
            // where the tile's rows and scales are, and the copies of a stage
            const int y_m = u.m * 128, y_n = u.n * NT;
            const uint8_t* sf_m = p.m.b + ((int64_t)u.m * atoms + 4 * u.k0) * kAtom;
            const uint8_t* sf_n = p.n.b + ((int64_t)(y_n / 128) * atoms + 4 * u.k0) * kAtom;
            auto load_m = [&](uint32_t at, uint32_t full, int x, uint32_t bytes, const uint8_t* sf) {
                tma_load_2d(at, &p.m.map, x, y_m, full);
                bulk_load(at + S::kA + S::kB, sf, bytes, full);
            };
            auto load_n = [&](uint32_t at, uint32_t full, int x, uint32_t bytes, const uint8_t* sf) {
                tma_load_2d(at + S::kA, &p.n.map, x, y_n, full);
                bulk_load(at + S::kA + S::kB + S::kSfA, sf, bytes, full);
            };
            // The weights of the first stages do not wait for the kernel before this one, which makes the tokens' codes.
            const uint32_t ahead = min(S::kStages, u.k1 - u.k0);
            for (uint32_t i = 0; i < ahead; ++i) {
                if (i + 1 == withheld) continue;
                const uint32_t at = sbase + i * S::kStage, full = bar(S::kFull + i);
                const int ks = u.k0 + i;
                const uint32_t bytes = ks == last ? last_bytes : 4 * kAtom;
                mbar_expect_tx(full, S::kA + S::kB + 2 * bytes);
                if (WIDE) load_n(at, full, ks * kRowBytes, bytes, sf_n + i * 4 * kAtom);
                else load_m(at, full, ks * kRowBytes, bytes, sf_m + i * 4 * kAtom);
            }
            pdl_wait();
            uint32_t s = 0, parity = 1, at = sbase, full = bar(S::kFull);
            int x = u.k0 * kRowBytes;
            for (int ks = u.k0; ks < u.k1; ++ks, ++it) {
                if (it >= ahead && !mbar_wait(full + 8 * S::kStages, parity, abort_flag, p.hdr)) break;  // (EMPTY)
                if (it + 1 != withheld) {  // (else its FULL phase never completes)
                    const uint32_t bytes = ks == last ? last_bytes : 4 * kAtom;
                    if (it >= ahead) mbar_expect_tx(full, S::kA + S::kB + 2 * bytes);
                    if (it >= ahead || WIDE) load_m(at, full, x, bytes, sf_m);
                    if (it >= ahead || !WIDE) load_n(at, full, x, bytes, sf_n);
                }
                x += kRowBytes;
                sf_m += 4 * kAtom;
                sf_n += 4 * kAtom;
                at += S::kStage;
                full += 8;
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                    at = sbase;
                    full = bar(S::kFull);
                }
            }
            // do not leave with copies in flight (without an abort their phases are complete)
            for (uint32_t j = it >= S::kStages ? it - S::kStages : 0; j < it; ++j)
                if (j + 1 != withheld) mbar_drain(bar(S::kFull + j % S::kStages), (j / S::kStages) & 1, p.hdr);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const uint32_t idesc = idesc_fp4(128, NT);
        const uint64_t ad0 = smem_desc_sw128(sbase), bd0 = smem_desc_sw128(sbase + S::kA);
        const uint64_t sd0 = scale_desc(sbase + S::kA + S::kB);
        uint32_t s = 0, parity = 0;
        bool ok = true;
        for (int ks = u.k0; ks < u.k1; ++ks) {
            if (!warp_wait(bar(S::kFull + s), parity, abort_flag, p.hdr)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                // (the lower 14 bits of a descriptor count 16 bytes, and a CTA's shared memory does not pass them)
                const uint64_t off = s * (S::kStage / 16), ad = ad0 + off, bd = bd0 + off, sd = sd0 + off;
                const uint32_t sfa = tmem + S::kSfCol0 + s * S::kSfCols, sfb = sfa + 16;
                const int nk = min(4, atoms - 4 * ks);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk >= nk) break;
                    copy_scales<1>(sfa + 4 * kk, sd + kk * (kAtom / 16));
                    copy_scales<1>(sfb + 4 * kk, sd + (S::kSfA + kk * kAtom) / 16);
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {  // 32 bytes = 2 address units per step
                    if (kk >= nk) break;
                    mma_fp4<1>(tmem, ad + 2 * kk, bd + 2 * kk, idesc, sfa + 4 * kk, sfb + 4 * kk,
                            ks > u.k0 || kk > 0);
                }
                mma_commit(bar(S::kEmpty + s));
            }
            __syncwarp();
            if (++s == S::kStages) {
                s = 0;
                parity ^= 1;
            }
        }
        if (ok && elect_one()) mma_commit(bar(S::kAFull));
        __syncwarp();
        // the products are done before the CTA frees TMEM
        if (elect_one()) mma_commit(bar(S::kTd));
        __syncwarp();
        mbar_drain(bar(S::kTd), 0, p.hdr);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        // (after a failed wait every warp goes on without the work, so that none waits at a barrier that the others left)
        const int q = warp & 3, part = (warp - kEpiWarp0) >> 2, me = threadIdx.x - 32 * kEpiWarp0;
        const int r = q * 32 + lane;  // row of the tile, TMEM lane
        const int64_t row = (int64_t)u.m * 128 + r, col0 = (int64_t)u.n * NT;
        const int cols = (int)min((int64_t)NT, p.n.rows - col0);
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
        float* cs = reinterpret_cast<float*>(smem + S::kScales);
        float rs = 0.0f;
        pdl_wait();
        if (!shared) {
            if (me < cols) cs[me] = __ldg(p.n.s + col0 + me);
            if (row < p.m.rows) rs = __ldg(p.m.s + row);
        }
        // (one warp waits for all: waiting warps take turns of the shared memory that copies and products use)
        bool ok = true;
        if (warp == kEpiWarp0) {
            ok = warp_wait(bar(S::kAFull), 0, abort_flag, p.hdr);
            tc_fence_after();
            tc_fence_before();
        }
        epi_sync();
        if (ok) ok = !__any_sync(0xFFFFFFFFu, *abort_flag);
        tc_fence_after();
        if (shared && ok) {
            constexpr int kChunk = NT < 32 ? NT : 32;
            for (int c0 = part * kChunk; c0 < cols; c0 += 2 * kChunk) {
                uint32_t v[kChunk];
                if constexpr (kChunk == 16) {
                    tmem_ld_x16(acc + c0, v);
                    tmem_wait_ld16(v);
                } else {
                    tmem_ld_x32(acc + c0, v);
                    tmem_wait_ld32(v);
                }
                float* to = reinterpret_cast<float*>(smem) + c0 * 128 + r;
#pragma unroll
                for (int j = 0; j < kChunk; ++j) to[j * 128] = __uint_as_float(v[j]);
            }
        } else if constexpr (WIDE) {
            if (ok) {
                const int64_t at = (int64_t)u.m * 128 + q * 32 + (lane & ~3);
                const int rows = (int)min((int64_t)4, p.m.rows - at), left = cols - 32 * part - 8 * (lane & 3);
                uint16_t* to = p.out + at * p.ld + col0 + 32 * part + 8 * (lane & 3);
#pragma unroll
                for (int k = 0; k < NT / 64; ++k) {
                    uint32_t v[32];
                    tmem_ld_x32(acc + 32 * (2 * k + part), v);
                    tmem_wait_ld32(v);
                    const float4* c = reinterpret_cast<const float4*>(cs + 32 * (2 * k + part));
                    uint4 x[4];  // 32 outputs, packed
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 a = c[2 * j], e = c[2 * j + 1];
                        auto f = [&](int i) { return __uint_as_float(v[8 * j + i]) * rs; };
                        x[j] = make_uint4(pack2(f(0) * a.x, f(1) * a.y), pack2(f(2) * a.z, f(3) * a.w),
                                          pack2(f(4) * e.x, f(5) * e.y), pack2(f(6) * e.z, f(7) * e.w));
                    }
                    store_run(x, to + 64 * k, p.ld, rows, left - 64 * k, lane);
                }
            }
        }
    }

    tc_fence_before();
    if (shared) {
        // Every warp's sums lie in shared memory as [NT][128]; the CTAs of a cluster share the adding and the stores.
        if (p.splits > 1) cluster_sync();
        else __syncthreads();
        if (warp >= kEpiWarp0) {
            const int64_t row0 = (int64_t)u.m * 128, col0 = (int64_t)u.n * NT;
            const int rows = (int)min((int64_t)128, p.m.rows - row0), cols = (int)min((int64_t)NT, p.n.rows - col0);
            const int rank = blockIdx.x % p.splits, me = threadIdx.x - 32 * kEpiWarp0;
            // a thread takes 8 outputs that lie together: 8 rows of a column (narrow), 8 columns of a row (wide)
            const int items = WIDE ? 128 * ((cols + 7) / 8) : 16 * cols;
            for (int i = rank * kEpiThreads + me; i < items; i += p.splits * kEpiThreads) {
                const int r = WIDE ? i % 128 : 8 * (i % 16), c = WIDE ? 8 * (i / 128) : i / 16;
                if (r >= rows) continue;
                float v[8];
                if constexpr (WIDE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
                    for (int s = 0; s < p.splits; ++s) {
                        const uint32_t from = p.splits > 1 ? peer_addr(sbase, s) : sbase;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += load_peer(from + 4 * ((c + j) * 128 + r));
                    }
                } else {
                    // (every CTA's part is on the way before the first is added: 64 tokens, N = 6144, K = 4096 8.0 to 7.7 us; with
                    // eight loads of the wide form for each it took longer)
                    float part[kMaxNarrow][8];
#pragma unroll
                    for (int s = 0; s < kMaxNarrow; ++s) {
                        if (s >= p.splits) break;
                        const uint32_t from = (p.splits > 1 ? peer_addr(sbase, s) : sbase) + 4 * (c * 128 + r);
                        load_peer4(from, part[s]);
                        load_peer4(from + 16, part[s] + 4);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = part[0][j];
#pragma unroll
                    for (int s = 1; s < kMaxNarrow; ++s) {
                        if (s >= p.splits) break;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += part[s][j];
                    }
                }
                const float own = __ldg(WIDE ? p.m.s + row0 + r : p.n.s + col0 + c);
                const float* others = WIDE ? p.n.s + col0 + c : p.m.s + row0 + r;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * own * __ldg(others + j);
                uint16_t* to = p.out + (WIDE ? (row0 + r) * p.ld + col0 + c : (col0 + c) * p.ld + row0 + r);
                *reinterpret_cast<uint4*>(to) =
                    make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
            }
        }
        __syncwarp();
        if (p.splits > 1) cluster_meet();  // no CTA leaves while another reads its sums
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmemCols) : "memory");
}

template <int NT, bool WIDE>
cudaError_t launch(LinearParams& p, const moe_fp4_t& x, const moe_fp4_t& w, int T, int N, cudaStream_t st) {
    using S = Shape<NT, WIDE>;
    if (!make_side(p.m, WIDE ? x : w, WIDE ? T : N, p.K, 128) || !make_side(p.n, WIDE ? w : x, WIDE ? N : T, p.K, NT))
        return cudaErrorInvalidValue;
    cudaError_t err = ensure_dynamic_smem((const void*)linear_kernel<NT, WIDE>, S::kSmem);
    if (err != cudaSuccess) return err;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int tiles = p.m.tiles * p.n.tiles, stages = (p.K + kStageK - 1) / kStageK;
    // K is cut while CTAs find an SM: in pairs all of them do, in fours 144 of 152, in eights 120 (each GPC holds whole
    // clusters; 16 of eight took twice the time of 8).  Narrow tiles are light enough for more CTAs than SMs, in pairs or where K is
    // long; joining wide ones costs as much as some ten stages.  Cuts of 1, 2, 4, us without the quantisation: 16 tokens, N = 2048, K = 4096 7.6, 5.8, 5.0; N = 6144
    // 7.8, 6.0, 6.6, K = 16384 20.6, 12.3, 9.6; N = 16384, K = 4096 7.8, 7.0, 13.2; 64 tokens, N = 4096 8.9, 6.9, 6.7; 128 tokens, N = 2048 7.8, 8.4, 7.2; K = 2048 5.6, 6.6, 6.0.
    p.splits = 1;
    for (int s = 2; s <= (WIDE ? kMaxSplits : kMaxNarrow); s *= 2) {
        const bool many = !WIDE && (s == 2 || stages >= 48);
        const int most = many ? sms * 7 / 4 : s == 2 ? sms : s == 4 ? sms * 7 / 8 : sms * 3 / 4;
        if (tiles * s <= most && stages >= 2 * s && (!WIDE || stages * (s - 1) / s >= 12)) p.splits = s;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tiles * p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<NT, WIDE>, p);
}

}  // namespace

cudaError_t launch_linear_fp4(moe_fp4_t x, moe_fp4_t w, int T, int N, int K, uint16_t* out, void* ws,
                              cudaStream_t st) {
    LinearParams p{};
    p.out = out;
    p.hdr = static_cast<WsHeader*>(ws);
    p.ld = N;
    p.K = K;
    if (T <= 16) return launch<16, false>(p, x, w, T, N, st);
    if (T <= 32) return launch<32, false>(p, x, w, T, N, st);
    if (T <= 64) return launch<64, false>(p, x, w, T, N, st);
    // Wide tiles that find an SM each (or share K) are done soonest; where there are more of them, the pairs' larger tiles move fewer
    // bytes.  Wide, pairs, us without the quantisation: 256 tokens, N = 8192, K = 512 4.3, 5.2; K = 2048 7.0, 7.1; N = 16384,
    // K = 512 6.3, 5.7; K = 2048 10.5, 7.7; 2048 tokens, N = 6144, K = 512 12.9, 10.3; K = 4096 36, 21.  The same for 65 to 128
    // tokens, where half of a pair's tile is empty, with the quantisation: 128 tokens, N = 19584, K = 512 8.7, 9.3; K = 4096 20.1, 19.9;
    // N = 32768 21.8, 21.8; N = 65536, K = 2048 28.2, 23.1; N = 152064, K = 4096 80, 67; 65 tokens, N = 32768 20.1, 20.4.
    const int64_t tiles = (int64_t)((T + 127) / 128) * ((N + 127) / 128);
    if (tiles > sm_count()) return launch_pair_fp4(x, w, T, N, K, out, ws, st);
    return launch<128, true>(p, x, w, T, N, st);
}

}  // namespace moe
