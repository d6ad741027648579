// Projections of many tokens in microscaled 4-bit floats: a pair of CTAs to a tile.
//
// A tile of 256 tokens by 256 weight rows belongs to two CTAs of a cluster, whose tensor cores work as one (cta_group::2):
// each holds half of the tokens and half of the weight rows of a stage, the scales of its tokens and of all weight rows, and
// the sums of its tokens.  So a CTA takes in 38 KB per stage of K = 256, where a tile of 128 by 256 of its own would take 54, and its
// tensor core reads 32 KB of codes instead of 48.  What bounds it is a stage's way round (0.32 us, 0.29
// without products, which take 0.2; 0.25 without the scales too) and what lies between two tiles: 2048 tokens, N = 6144, K = 4096 20.5 us,
// 5.0 PFLOP/s; 8192 tokens, N = K = 8192 152, 7.2 PFLOP/s.
//
// All of a stage's copies, of either CTA, are counted on one barrier of the leader (rank 0), which issues the products; their
// completion frees the stage in both.
//
// Warps of each CTA: 0, 10 and 11 copy; 1 allocates TMEM and, in the leader, issues the products; 2-9 the epilogue, two per quarter of
// TMEM's lanes.
#include "fp4_mma.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 8, kEpiWarp0 = 2;
constexpr int kCopyWarps = 3, kCopyWarp1 = kEpiWarp0 + kEpiWarps;  // warp 0 and those from kCopyWarp1 on
constexpr int kThreads = 32 * (kCopyWarp1 + kCopyWarps - 1);
constexpr int kTile = 256;                                 // tokens, and weight rows, of a pair's tile
constexpr int kA = 128 * kRowBytes, kB = 128 * kRowBytes;  // a CTA's halves of a stage
constexpr int kSfA = 4 * kAtom, kSfB = 8 * kAtom;          // scales of its tokens, of all weight rows
constexpr int kStage = kA + kB + kSfA + kSfB;
constexpr int kStages = 5;
constexpr int kSfCols = 16 + 32, kSfCol0 = kTile;  // TMEM columns of a stage's scales
constexpr int kTmemCols = 512;
// FULL[stages] (the leader's count), EMPTY[stages], AFULL, AEMPTY (the leader's counts), TD (the products in flight at the end)
constexpr int kFull = 0, kEmpty = kStages, kAFull = 2 * kStages, kAEmpty = kAFull + 1, kTd = kAEmpty + 1;
constexpr int kScalesAt = kStages * kStage;  // row scales of the weight rows, two tiles'
constexpr int kBarAt = kScalesAt + 2 * kTile * 4;
constexpr int kMisc = kBarAt + 8 * (kTd + 1);
constexpr int kSmem = kMisc + 16 + 1024;  // + alignment slack
static_assert(kSmem <= 227 * 1024 && kSfCol0 + kStages * kSfCols <= kTmemCols && kStage % 1024 == 0, "");

struct PairSide {
    CUtensorMap codes, scales;
    const float* s;
    int rows, tiles;  // tiles of 256 rows
};

struct PairParams {
    PairSide x, w;
    uint16_t* out;
    WsHeader* hdr;
    int64_t ld;
    int K;
};

// A copy of either CTA into its own shared memory, counted on a barrier of one of the two.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(cluster_bar)
        : "memory");
}
// Relaxed: what it tells, that TMEM has been read, is over when it is issued, and it hands nothing in memory over.  (With release, and
// a fence at the leader, it waited for the tile's stores before: in the first case above 25.2 us instead of 22.2.)
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// Arrive on the barriers of both CTAs once the pair's products issued so far are done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) pair_kernel(const __grid_constant__ PairParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    // (the shuffle tells the compiler that a warp has one number: copies of three roles took 10% longer without)
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = blockIdx.x & 1;
    auto bar = [&](int i) { return sbase + kBarAt + 8 * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMisc + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(kFull + s), kCopyWarps);
            mbar_init(bar(kEmpty + s), 1);
        }
        mbar_init(bar(kAFull), 1);
        mbar_init(bar(kAEmpty), 2 * kEpiWarps);
        mbar_init(bar(kTd), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&p.x.codes);
        prefetch_tmap(&p.x.scales);
        prefetch_tmap(&p.w.codes);
        prefetch_tmap(&p.w.scales);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_meet();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int units = p.x.tiles * p.w.tiles, first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int atoms = p.K / 64, stages = (p.K + kStageK - 1) / kStageK;

    if (warp == 0 || warp >= kCopyWarp1) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            // One thread copies the weight rows' codes, one the tokens', one the scales: issuing a copy takes a thread some 60 ns,
            // and all four of a stage by one thread bounded the loop.
            enum { kWeights, kTokens, kScaleTiles };
            const int role = warp == 0 ? kWeights : warp == kCopyWarp1 ? kTokens : kScaleTiles;
            const uint32_t withheld = withheld_stage(p.hdr);
            const uint32_t full0 = peer_addr(bar(kFull), 0);  // in the leader
            uint32_t it = 0;
            bool ok = true;
            int n = first / p.x.tiles, m = first - n * p.x.tiles;
            // K's last stage is filled up with zeros where K ends inside it, and rows past the last are zeros
            auto expect = [&](uint32_t i) {
                if (rank == 0) mbar_expect_tx(bar(kFull) + 8 * i, role == kWeights ? 2 * kB : role == kTokens ? 2 * kA : 2 * (kSfA + kSfB));
            };
            auto weights = [&](uint32_t at, uint32_t full, int ks) {
                if (role == kWeights) tma_load_2d_pair(at + kA, &p.w.codes, ks * kRowBytes, n * kTile + rank * 128, full);
                if (role == kScaleTiles)
                    tma_load_2d_pair(at + kA + kB + kSfA, &p.w.scales, ks * (4 * kAtom / 8), 2 * n, full);
            };
            auto tokens = [&](uint32_t at, uint32_t full, int ks) {
                if (role == kTokens) tma_load_2d_pair(at, &p.x.codes, ks * kRowBytes, m * kTile + rank * 128, full);
                if (role == kScaleTiles)
                    tma_load_2d_pair(at + kA + kB, &p.x.scales, ks * (4 * kAtom / 8), 2 * m + rank, full);
            };
            // The weights of the first stages do not wait for the kernel before this one, which makes the tokens' codes.
            uint32_t ahead = 0;
            if (first < units) {
                ahead = min(kStages, stages);
                for (uint32_t i = 0; i < ahead; ++i) {
                    if (i + 1 == withheld) continue;
                    expect(i);
                    weights(sbase + i * kStage, full0 + 8 * i, i);
                }
            }
            pdl_wait();
            uint32_t s = 0, parity = 1, at = sbase, full = full0, empty = bar(kEmpty);
            for (int u = first; u < units && ok; u += step) {
                if (u != first) {
                    n = u / p.x.tiles;
                    m = u - n * p.x.tiles;
                }
                for (int ks = 0; ks < stages; ++ks, ++it) {
                    if (it >= ahead && !mbar_wait(empty, parity, abort_flag, p.hdr)) {
                        ok = false;
                        break;
                    }
                    if (it + 1 != withheld) {  // (else its FULL phase never completes)
                        if (it >= ahead) {
                            expect(s);
                            weights(at, full, ks);
                        }
                        tokens(at, full, ks);
                    }
                    at += kStage;
                    full += 8;
                    empty += 8;
                    if (++s == kStages) {
                        s = 0;
                        parity ^= 1;
                        at = sbase;
                        full = full0;
                        empty = bar(kEmpty);
                    }
                }
            }
            // Do not leave with copies in flight: without an abort their phases are complete, as every product has been
            // waited for; after one the leader waits for its phases, which count the other's copies too (for what that one copies
            // past them see the end).
            if (rank == 0) {
                for (uint32_t j = it >= kStages ? it - kStages : 0; j < it; ++j)
                    if (j + 1 != withheld) mbar_drain(bar(kFull + j % kStages), (j / kStages) & 1, p.hdr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        if (rank == 0) {
            const uint32_t idesc = idesc_fp4(2 * 128, kTile);
            const uint64_t ad0 = smem_desc_sw128(sbase), bd0 = smem_desc_sw128(sbase + kA), sd0 = scale_desc(sbase + kA + kB);
            uint32_t s = 0, parity = 0, tc = 0;
            bool ok = true;
            for (int u = first; u < units && ok; u += step, ++tc) {
                if (!warp_wait(bar(kAEmpty), (tc & 1) ^ 1, abort_flag, p.hdr)) break;
                tc_fence_after();
                for (int ks = 0; ks < stages; ++ks) {
                    if (!warp_wait(bar(kFull + s), parity, abort_flag, p.hdr)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        // (the lower 14 bits of a descriptor count 16 bytes, and a CTA's shared memory does not pass them)
                        const uint64_t off = s * (kStage / 16), ad = ad0 + off, bd = bd0 + off, sd = sd0 + off;
                        const uint32_t sfa = tmem + kSfCol0 + s * kSfCols, sfb = sfa + 16;
                        const int nk = min(4, atoms - 4 * ks);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kk >= nk) break;
                            copy_scales<2>(sfa + 4 * kk, sd + kk * (kAtom / 16));
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                copy_scales<2>(sfb + 4 * (2 * kk + r), sd + (kSfA + (4 * r + kk) * kAtom) / 16);
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {  // 32 bytes = 2 address units per step
                            if (kk >= nk) break;
                            mma_fp4<2>(tmem, ad + 2 * kk, bd + 2 * kk, idesc, sfa + 4 * kk, sfb + 8 * kk, ks > 0 || kk > 0);
                        }
                        commit_both(bar(kEmpty + s));
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        parity ^= 1;
                    }
                }
                if (!ok) break;
                if (elect_one()) commit_both(bar(kAFull));
                __syncwarp();
            }
            // the products are done before either CTA frees TMEM
            if (elect_one()) commit_both(bar(kTd));
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // After a failed wait every warp keeps walking the units without the work, so that none waits
        // at a barrier that the others left.
        const int q = warp & 3, part = (warp - kEpiWarp0) >> 2, me = threadIdx.x - 32 * kEpiWarp0;
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + 32 * part, aempty = peer_addr(bar(kAEmpty), 0);
        bool ok = true;
        uint32_t tc = 0;
        pdl_wait();
        // a lane's row scale, and one of the weight rows', of a tile: fetched while the tile before is stored
        float c_next = 0.0f, r_next = 0.0f;
        auto fetch_scales = [&](int u) {
            if (u >= units) return;
            const int n = u / p.x.tiles, m = u - n * p.x.tiles;
            const int64_t row = (int64_t)m * kTile + rank * 128 + q * 32 + lane, col = (int64_t)n * kTile + me;
            if (row < p.x.rows) r_next = __ldg(p.x.s + row);
            if (col < p.w.rows) c_next = __ldg(p.w.s + col);
        };
        fetch_scales(first);
        for (int u = first; u < units; u += step, ++tc) {
            const int n = u / p.x.tiles, m = u - n * p.x.tiles;
            const int64_t row0 = (int64_t)m * kTile + rank * 128 + q * 32, col0 = (int64_t)n * kTile;
            const int cols = (int)min((int64_t)kTile, p.w.rows - col0);
            float* cs = reinterpret_cast<float*>(smem + kScalesAt) + (tc & 1) * kTile;
            cs[me] = c_next;
            const float rs = r_next;
            // (one warp waits for all: waiting warps take turns of the shared memory that copies and products use)
            if (warp == kEpiWarp0) {
                if (ok) ok = warp_wait(bar(kAFull), tc & 1, abort_flag, p.hdr);
                tc_fence_after();
                tc_fence_before();
            }
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
            if (ok) ok = !__any_sync(0xFFFFFFFFu, *abort_flag);
            // Nearly all of a lane's sums leave TMEM before they are packed, so that the next tile's products wait the least; the
            // last come while the first are packed, since registers hold no more.
            uint32_t v[4][32];
            uint4 x[4];  // 32 outputs, packed
            auto pack_run = [&](int k) {
                const float4* c = reinterpret_cast<const float4*>(cs + 32 * (2 * k + part));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 a = c[2 * j], b = c[2 * j + 1];
                    auto f = [&](int i) { return __uint_as_float(v[k][8 * j + i]) * rs; };
                    x[j] = make_uint4(pack2(f(0) * a.x, f(1) * a.y), pack2(f(2) * a.z, f(3) * a.w),
                                      pack2(f(4) * b.x, f(5) * b.y), pack2(f(6) * b.z, f(7) * b.w));
                }
            };
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 3; ++k) tmem_ld_x32(acc + 64 * k, v[k]);
#pragma unroll
                for (int k = 0; k < 3; ++k) tmem_wait_ld32(v[k]);
                tmem_ld_x32(acc + 64 * 3, v[3]);
                pack_run(0);
                tmem_wait_ld32(v[3]);
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) arrive_at(aempty);
            fetch_scales(u + step);
            if (!ok) continue;
            const int64_t at = row0 + (lane & ~3);
            const int rows = (int)min((int64_t)4, p.x.rows - at), left = cols - 32 * part - 8 * (lane & 3);
            uint16_t* to = p.out + at * p.ld + col0 + 32 * part + 8 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k > 0) pack_run(k);
                store_run(x, to + 64 * k, p.ld, rows, left - 64 * k, lane);
            }
        }
    }

    // Neither leaves while the other's arrivals or products may still come.  After an abort the leader may have given up at an
    // earlier stage than the other copied for, whose phases nobody can wait for then: its CTA stays for longer than a copy
    // takes.  (Its own flag is set by then: products that the leader leaves out never reach its epilogue's or its copies' waits.)
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        mbar_drain(bar(kTd), 0, p.hdr);
        if (*abort_flag)
            for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < 1000000;) {
            }
    }
    __syncthreads();
    cluster_meet();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// box_tiles: scale tiles of 128 rows to a copy.
bool make_pair_side(PairSide& s, const moe_fp4_t& v, int rows, int64_t K, int box_tiles) {
    s.s = v.s;
    s.rows = rows;
    s.tiles = (rows + kTile - 1) / kTile;
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 64 * (kAtom / 8)), (cuuint64_t)((rows + 127) / 128)};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 64 * kAtom)};
    const cuuint32_t box[2] = {4 * kAtom / 8, (cuuint32_t)box_tiles};
    return codes_map(&s.codes, v.q, rows, K, 128) &&
           make_map_nd(&s.scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, v.b, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

cudaError_t launch_pair_fp4(moe_fp4_t x, moe_fp4_t w, int T, int N, int K, uint16_t* out, void* ws, cudaStream_t st) {
    PairParams p{};
    if (!make_pair_side(p.x, x, T, K, 1) || !make_pair_side(p.w, w, N, K, 2)) return cudaErrorInvalidValue;
    p.out = out;
    p.hdr = static_cast<WsHeader*>(ws);
    p.ld = N;
    p.K = K;
    cudaError_t err = ensure_dynamic_smem((const void*)pair_kernel, kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * std::min(p.x.tiles * p.w.tiles, sm_count() / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pair_kernel, p);
}

}  // namespace moe
