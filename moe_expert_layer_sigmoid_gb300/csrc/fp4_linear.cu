// Projections with both operands in microscaled 4-bit floats: the tensor cores' block-scaled products
// (kind::mxf4nvf4, E2M1 x E2M1 with an E4M3 scale for each 16, fp32 accumulators in TMEM).
//
//   out[t][n] = (sum over blocks of bx bw (sum of 16 code products)) * s_x[t] * s_w[n]
// Code products and block scales meet inside the product, so codes go from memory to the tensor core as they are
// stored; the two row scales are applied once, to the finished sum.
//
// A tile is M = 128 weight rows by NT tokens, K in stages of 256 elements: 128 bytes of codes per row (TMA, 128-byte
// swizzle) and, for each 128 rows and 64 elements, 512 bytes of scales, which lie in memory in the order
// that tcgen05.cp spreads over TMEM (lane r % 32 and column r / 32 hold row r's four scales).  Four products of
// K = 64 per stage.  NT is the smallest of 16, 32, 64, 128 that holds the tokens, so that few tokens do not pay for
// many; what bounds few tokens is the weights' bytes.  They are spread over all SMs by cutting K, and the cuts' sums are
// joined in a fixed order by the last CTA of a tile to arrive.
//
// Warps: 0 copies, 1 allocates TMEM and issues the products, 2-9 the epilogue, two per quarter of TMEM's
// lanes.  The scales of a stage have TMEM columns of their own, which are free when the stage's shared memory is.
#include "fp4.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 8, kEpiWarp0 = 2;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kStageK = 256;           // elements of K per stage
constexpr int kRowBytes = kStageK / 2;  // codes of a row per stage
constexpr int kAtom = 512;             // scales of 128 rows and 64 elements
constexpr int kTmemCols = 512;

template <int NT>
struct Shape {
    static constexpr int kBlocks = (NT + 127) / 128;  // scale tiles of the tokens
    static constexpr int kA = 128 * kRowBytes, kB = NT * kRowBytes;
    static constexpr int kSfA = 4 * kAtom, kSfB = 4 * kAtom * kBlocks;
    static constexpr int kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = 216 * 1024 / kStage < 8 ? 216 * 1024 / kStage : 8;
    static constexpr int kAcc = NT <= 128 ? 2 : 1;             // accumulators
    static constexpr int kSfCols = 16 + 16 * kBlocks;          // TMEM columns of a stage's scales
    static constexpr int kSfCol0 = kAcc * NT;
    // FULL[stages], EMPTY[stages], AFULL[acc], AEMPTY[acc], TD (the products in flight at the end)
    static constexpr int kFull = 0, kEmpty = kStages, kAFull = 2 * kStages, kAEmpty = kAFull + kAcc, kTd = kAEmpty + kAcc;
    static constexpr int kBarAt = kStages * kStage;
    static constexpr int kMisc = kBarAt + 8 * (kTd + 1);
    static constexpr int kSmem = kMisc + 16 + 1024;  // + alignment slack
    static_assert(kSmem <= 227 * 1024 && kSfCol0 + kStages * kSfCols <= kTmemCols && kStage % 1024 == 0, "");
};

struct LinearParams {
    CUtensorMap tm_w, tm_x;
    const uint8_t *wb, *xb;  // block scales
    const float *ws, *xs;    // row scales
    uint16_t* out;
    WsHeader* hdr;
    int32_t* counters;  // arrivals per tile, 0 between calls
    float* parts;       // sums of a unit's part of K, [unit][NT][128]
    int T, N, K;
    int m_tiles, tiles, splits;
};

// Instruction descriptor, kind::mxf4nvf4: E2M1 A and B, unsigned E4M3 scales, fp32 D, both K-major.
__device__ __forceinline__ uint32_t idesc_fp4(int M, int N) {
    return (1u << 7)                      // A format: E2M1
           | (1u << 10)                   // B format: E2M1
           | ((uint32_t)(N >> 3) << 17)   // N / 8
           | ((uint32_t)(M >> 7) << 27);  // M / 128
}

// D (TMEM) (+)= A (shared memory) x B (shared memory) with scales in TMEM, K = 64.
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 32 rows of 16 bytes of shared memory to four TMEM columns, in each quarter of the lanes.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
    const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 |
                          (uint64_t)(128 >> 4) << 32 |  // 8 rows of 16 bytes to the next 8
                          (uint64_t)1 << 46;            // version; no swizzle
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

struct Unit {
    int m, n;      // tile of weight rows, of tokens
    int k0, k1;    // stages
};
__device__ __forceinline__ Unit unit_of(const LinearParams& p, int u) {
    const int tile = u / p.splits, s = u - tile * p.splits, all = (p.K + kStageK - 1) / kStageK;
    Unit r;
    r.n = tile / p.m_tiles;
    r.m = tile - r.n * p.m_tiles;
    r.k0 = (int)((int64_t)all * s / p.splits);
    r.k1 = (int)((int64_t)all * (s + 1) / p.splits);
    return r;
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory"); }

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p) {
    using S = Shape<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return sbase + S::kBarAt + 8 * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
    volatile int* last_here = reinterpret_cast<volatile int*>(smem + S::kMisc + 8);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(bar(S::kFull + s), 1);
            mbar_init(bar(S::kEmpty + s), 1);
        }
        for (int b = 0; b < S::kAcc; ++b) {
            mbar_init(bar(S::kAFull + b), 1);
            mbar_init(bar(S::kAEmpty + b), kEpiWarps);
        }
        mbar_init(bar(S::kTd), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&p.tm_w);
        prefetch_tmap(&p.tm_x);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int units = p.tiles * p.splits, grid = gridDim.x;
    const int atoms = p.K / 64;                      // scale atoms of a row tile
    const int x_blocks = (p.T + 127) / 128;          // row tiles of the tokens' scales

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            const uint32_t withheld = withheld_stage(p.hdr);
            uint32_t it = 0;
            bool ok = true;
            auto weights = [&](uint32_t i, const Unit& u, int ks) {
                const uint32_t at = sbase + (i % S::kStages) * S::kStage, full = bar(S::kFull + i % S::kStages);
                const int nk = min(4, atoms - 4 * ks);
                const int blocks = min(S::kBlocks, x_blocks - u.n * NT / 128);
                mbar_expect_tx(full, S::kA + S::kB + nk * kAtom * (1 + blocks));
                tma_load_2d(at, &p.tm_w, ks * kRowBytes, u.m * 128, full);
                bulk_load(at + S::kA + S::kB, p.wb + ((int64_t)u.m * atoms + 4 * ks) * kAtom, nk * kAtom, full);
            };
            auto tokens = [&](uint32_t i, const Unit& u, int ks) {
                const uint32_t at = sbase + (i % S::kStages) * S::kStage, full = bar(S::kFull + i % S::kStages);
                const int nk = min(4, atoms - 4 * ks), first = u.n * NT / 128;
                tma_load_2d(at + S::kA, &p.tm_x, ks * kRowBytes, u.n * NT, full);
                for (int b = 0; b < min(S::kBlocks, x_blocks - first); ++b)
                    bulk_load(at + S::kA + S::kB + S::kSfA + b * 4 * kAtom,
                              p.xb + ((int64_t)(first + b) * atoms + 4 * ks) * kAtom, nk * kAtom, full);
            };
            // The weights of the first stages do not wait for the kernel before this one, which makes the tokens' codes.
            uint32_t ahead = 0;
            if ((int)blockIdx.x < units) {
                const Unit u = unit_of(p, blockIdx.x);
                ahead = min(S::kStages, u.k1 - u.k0);
                for (uint32_t i = 0; i < ahead; ++i)
                    if (i + 1 != withheld) weights(i, u, u.k0 + i);
            }
            pdl_wait();
            for (int n = blockIdx.x; n < units && ok; n += grid) {
                const Unit u = unit_of(p, n);
                for (int ks = u.k0; ks < u.k1; ++ks, ++it) {
                    if (it >= ahead &&
                        !mbar_wait(bar(S::kEmpty + it % S::kStages), ((it / S::kStages) & 1) ^ 1, abort_flag, p.hdr)) {
                        ok = false;
                        break;
                    }
                    if (it + 1 == withheld) continue;  // its FULL phase never completes
                    if (it >= ahead) weights(it, u, ks);
                    tokens(it, u, ks);
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
        uint32_t it = 0, tc = 0;
        bool ok = true;
        for (int n = blockIdx.x; n < units && ok; n += grid) {
            const Unit u = unit_of(p, n);
            const int b = tc % S::kAcc;
            if (!warp_wait(bar(S::kAEmpty + b), ((tc / S::kAcc) & 1) ^ 1, abort_flag, p.hdr)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + b * NT;
            for (int ks = u.k0; ks < u.k1; ++ks, ++it) {
                const int s = it % S::kStages;
                if (!warp_wait(bar(S::kFull + s), (it / S::kStages) & 1, abort_flag, p.hdr)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t at = sbase + s * S::kStage, sf = at + S::kA + S::kB;
                    const uint32_t sfa = tmem + S::kSfCol0 + s * S::kSfCols, sfb = sfa + 16;
                    const int nk = min(4, atoms - 4 * ks);
                    const uint64_t ad = smem_desc_sw128(at), bd = smem_desc_sw128(at + S::kA);
                    for (int kk = 0; kk < nk; ++kk) {
                        copy_scales(sfa + 4 * kk, sf + kk * kAtom);
#pragma unroll
                        for (int r = 0; r < S::kBlocks; ++r)
                            copy_scales(sfb + 4 * (S::kBlocks * kk + r), sf + S::kSfA + (4 * r + kk) * kAtom);
                    }
                    for (int kk = 0; kk < nk; ++kk)  // 32 bytes = 2 address units per step
                        mma_fp4(d, ad + 2 * kk, bd + 2 * kk, idesc, sfa + 4 * kk, sfb + 4 * S::kBlocks * kk,
                                ks > u.k0 || kk > 0);
                    mma_commit(bar(S::kEmpty + s));
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) mma_commit(bar(S::kAFull + b));
            __syncwarp();
            ++tc;
        }
        // the products are done before the CTA frees TMEM
        if (elect_one()) mma_commit(bar(S::kTd));
        __syncwarp();
        mbar_drain(bar(S::kTd), 0, p.hdr);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        // After a failed wait every warp keeps walking the units without the work, so that none waits
        // at a barrier that the others left.
        constexpr int kChunk = NT < 32 ? NT : 32;
        const int q = warp & 3, part = (warp - kEpiWarp0) >> 2;
        const int m = q * 32 + lane;
        bool ok = true;
        uint32_t tc = 0;
        pdl_wait();
        for (int n = blockIdx.x; n < units; n += grid, ++tc) {
            const Unit u = unit_of(p, n);
            const int b = tc % S::kAcc, t0 = u.n * NT;
            const int64_t row = (int64_t)u.m * 128 + m;  // output channel
            const int cols = min(NT, p.T - t0);
            if (ok) ok = warp_wait(bar(S::kAFull + b), (tc / S::kAcc) & 1, abort_flag, p.hdr);
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + b * NT;
            const float sw = row < p.N ? __ldg(p.ws + row) : 0.0f;
            auto finish = [&](const float (&v)[kChunk], int c0) {
                const float mine = c0 + lane < cols && lane < kChunk ? __ldg(p.xs + t0 + c0 + lane) : 0.0f;
                // Two tokens at a time: even lanes store the first one's pair of channels, odd lanes the second one's.
#pragma unroll
                for (int j = 0; j < kChunk; j += 2) {
                    const float a = v[j] * __shfl_sync(0xFFFFFFFFu, mine, j) * sw;
                    const float c = v[j + 1] * __shfl_sync(0xFFFFFFFFu, mine, j + 1) * sw;
                    const float other = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? a : c, 1);
                    const __nv_bfloat162 o = lane & 1 ? __floats2bfloat162_rn(other, c) : __floats2bfloat162_rn(a, other);
                    const int t = c0 + j + (lane & 1);
                    if (t < cols && row < p.N)
                        *reinterpret_cast<__nv_bfloat162*>(p.out + (int64_t)(t0 + t) * p.N + (row & ~1ll)) = o;
                }
            };
            if (ok) {
                tc_fence_after();
                for (int c0 = part * kChunk; c0 < cols; c0 += 2 * kChunk) {
                    uint32_t v[kChunk];
                    if constexpr (kChunk == 16) {
                        tmem_ld_x16(acc + c0, v);
                        tmem_wait_ld16(v);
                    } else {
                        tmem_ld_x32(acc + c0, v);
                        tmem_wait_ld32(v);
                    }
                    float f[kChunk];
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) f[j] = __uint_as_float(v[j]);
                    if (p.splits == 1) {
                        finish(f, c0);
                    } else {
                        float* to = p.parts + ((int64_t)n * NT + c0) * 128 + m;
#pragma unroll
                        for (int j = 0; j < kChunk; ++j)
                            if (c0 + j < cols) to[j * 128] = f[j];
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S::kAEmpty + b));
            if (p.splits == 1) continue;
            // the last CTA of the tile to arrive adds the parts, in the order of K
            __threadfence();
            epi_sync();
            const int tile = n / p.splits;
            if (threadIdx.x == 32 * kEpiWarp0) {
                const int before = atomicAdd(p.counters + tile, 1);
                *last_here = before == p.splits - 1;
                if (*last_here) p.counters[tile] = 0;
                __threadfence();
            }
            epi_sync();
            if (*last_here) {
                for (int c0 = part * kChunk; c0 < cols; c0 += 2 * kChunk) {
                    float f[kChunk];
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) f[j] = 0.0f;
                    for (int s = 0; s < p.splits; ++s) {
                        const float* from = p.parts + ((int64_t)(tile * p.splits + s) * NT + c0) * 128 + m;
#pragma unroll
                        for (int j = 0; j < kChunk; ++j)
                            if (c0 + j < cols) f[j] += __ldcg(from + j * 128);
                    }
                    finish(f, c0);
                }
            }
            epi_sync();  // (last_here has been read)
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

bool codes_map(CUtensorMap* m, const uint8_t* q, int64_t rows, int64_t K, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
    return make_map_nd(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int NT>
cudaError_t launch(LinearParams& p, const moe_fp4_t& x, const moe_fp4_t& w, cudaStream_t st) {
    using S = Shape<NT>;
    if (!codes_map(&p.tm_w, w.q, p.N, p.K, 128) || !codes_map(&p.tm_x, x.q, p.T, p.K, NT)) return cudaErrorInvalidValue;
    cudaError_t err = ensure_dynamic_smem((const void*)linear_kernel<NT>, S::kSmem);
    if (err != cudaSuccess) return err;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    p.tiles = p.m_tiles * ((p.T + NT - 1) / NT);
    const int stages = (p.K + kStageK - 1) / kStageK;
    p.splits = std::max(1, std::min({kFp4Units / p.tiles, stages / 2, 16}));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(std::min(p.tiles * p.splits, sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<NT>, p);
}

}  // namespace

int fp4_tile_tokens(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256; }

cudaError_t launch_linear_fp4(moe_fp4_t x, moe_fp4_t w, int T, int N, int K, uint16_t* out, void* ws, const Fp4Ws& at,
                              cudaStream_t st) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    LinearParams p{};
    p.wb = w.b;
    p.xb = x.b;
    p.ws = w.s;
    p.xs = x.s;
    p.out = out;
    p.hdr = static_cast<WsHeader*>(ws);
    p.counters = reinterpret_cast<int32_t*>(base + at.counters);
    p.parts = reinterpret_cast<float*>(base + at.parts);
    p.T = T;
    p.N = N;
    p.K = K;
    p.m_tiles = (N + 127) / 128;
    switch (fp4_tile_tokens(T)) {
        case 16: return launch<16>(p, x, w, st);
        case 32: return launch<32>(p, x, w, st);
        case 64: return launch<64>(p, x, w, st);
        case 128: return launch<128>(p, x, w, st);
        default: return launch<256>(p, x, w, st);
    }
}

}  // namespace moe
