// The norms between two blocks, fused with the gate, the scale and the residual
// between them: one launch, one pass over memory.
//
// A row stays with its threads from the first load to the last store, so the two sums of
// squares cost exchanges only; the bound is DRAM bandwidth, and for a few rows the launch and two exchanges.
// Rows of at most kWarpRow elements take a warp each, longer ones a CTA.  Either walks rows, and copies the rows
// to come into shared memory meanwhile, each thread what it will itself read, so that memory is busy while
// sums are exchanged.  Sums are fp32, in an order that the row's length and the residual's type set (a thread adds the groups of 8
// or 4 elements that it loads).  Measured: 8192 rows of 4096 with a
// full gate 57 us, 5.9 TB/s (rows in registers only, a CTA each: 67); one row 2.7 us.
//
// Rows past 16384 elements (and past 8192 with an fp32 residual and a full gate, whose copies do not fit) have no ring: a CTA
// each, read in place.  Past 16384 a thread's 32 elements of residual and output do not fit the 64 registers of 1024 threads, and 132 to
// 280 bytes of them go to local memory and back: 2048 rows of 24576, bf16 without a gate 136 us, 3.0 TB/s, with a full gate
// 183, fp32 202 (16384 elements in registers and ring: 58 us, 4.6 TB/s).
#include "block_norm.cuh"

namespace moe {
namespace {

struct NormParams {
    const uint16_t* y;
    const void* residual;
    const void* gate;
    const float *w_post, *w_pre;
    void* residual_out;
    uint16_t* x;
    int T, d;
    float eps, scale;
    int ahead;  // rows on the way: 1 or 3
};

constexpr int kWarpRow = 1024;  // longest row of one warp: 32 elements to a lane

// E elements at a time, so that neighbouring lanes' 16 bytes of the residual lie together: 8 where it is bf16, 4
// where it is fp32.
template <int E>
struct Bits;
template <>
struct Bits<8> { using T = uint4; };
template <>
struct Bits<4> { using T = uint2; };

__device__ __forceinline__ void unpack(uint4 x, float (&f)[8]) {
    f[0] = bf16_lo(x.x); f[1] = bf16_hi(x.x); f[2] = bf16_lo(x.y); f[3] = bf16_hi(x.y);
    f[4] = bf16_lo(x.z); f[5] = bf16_hi(x.z); f[6] = bf16_lo(x.w); f[7] = bf16_hi(x.w);
}
__device__ __forceinline__ void unpack(uint2 x, float (&f)[4]) {
    f[0] = bf16_lo(x.x); f[1] = bf16_hi(x.x); f[2] = bf16_lo(x.y); f[3] = bf16_hi(x.y);
}
__device__ __forceinline__ void unpack(uint4 x, float (&f)[4]) {  // (fp32)
    f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y); f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
}
template <int E>
__device__ __forceinline__ void load_floats(const float* p, float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
        f[i] = a.x; f[i + 1] = a.y; f[i + 2] = a.z; f[i + 3] = a.w;
    }
}
__device__ __forceinline__ uint32_t pair(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
}
__device__ __forceinline__ void store(uint16_t* p, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pair(f[0], f[1]), pair(f[2], f[3]));
}
__device__ __forceinline__ void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// The sum over a row's threads: a warp, or the CTA (`part` takes the warps' sums: not one that the sum before took,
// which some warp may still read).
template <bool CTA>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (!CTA) return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// What a thread copies of a row into shared memory: groups of the residual, the block's output and, where it has as many
// elements, the gate.
template <typename Res, int GATE, int GROUPS>
struct Slot {
    static constexpr int kE = 16 / sizeof(Res), kHalf = 2 * kE;  // elements, and bytes of bf16, of a group
    static constexpr int kY = 16 * GROUPS, kG = kY + kHalf * GROUPS;
    static constexpr int kBytes = kG + (GATE == MOE_GATE_FULL ? kHalf * GROUPS : 0);  // of a thread
};

// ELEMS: elements of a thread.  RING: rows come through shared memory, p.ahead of them on the way; else straight from memory.
template <typename Res, int GATE, bool CTA, int ELEMS, int MAX, bool RING>
__global__ void __launch_bounds__(MAX) block_norm_kernel(const NormParams p, bool sigmoid) {
    constexpr int E = 16 / sizeof(Res), GROUPS = ELEMS / E;
    using S = Slot<Res, GATE, GROUPS>;
    using Half = typename Bits<E>::T;
    constexpr bool kKeep = RING && MAX <= 640 && ELEMS <= 16;  // the norms' weights stay in registers
    extern __shared__ __align__(16) uint8_t ring[];            // [p.ahead + 1][parts][threads of the CTA]
    __shared__ float part[2][2][32];                           // by row, by norm
    const int threads = CTA ? blockDim.x : 32, me = CTA ? threadIdx.x : threadIdx.x & 31;
    const int64_t first = CTA ? blockIdx.x : (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t stride = CTA ? gridDim.x : (int64_t)gridDim.x * 8;
    auto at = [&](int j) { return E * (me + j * threads); };
    // this thread's place for a group of `size` bytes, the j-th of those that begin `off` bytes into a thread's share
    auto slot = [&](int n, int off, int size, int j) {
        return ring + ((size_t)(n & p.ahead) * S::kBytes + off + size * j) * blockDim.x + size * threadIdx.x;
    };
    auto fetch = [&](int n) {  // the n-th row of this walk
        const int64_t t = first + n * stride;
        if (t < p.T) {
            const int64_t row = t * p.d;
#pragma unroll
            for (int j = 0; j < GROUPS; ++j) {
                if (at(j) >= p.d) continue;
                copy_async<16>(slot(n, 0, 16, j), static_cast<const Res*>(p.residual) + row + at(j));
                if (p.y) copy_async<S::kHalf>(slot(n, S::kY, S::kHalf, j), p.y + row + at(j));
                if (GATE == MOE_GATE_FULL)
                    copy_async<S::kHalf>(slot(n, S::kG, S::kHalf, j), static_cast<const uint16_t*>(p.gate) + row + at(j));
            }
        }
        copy_commit();
    };
    if (RING)
        for (int n = 0; n < p.ahead; ++n) fetch(n);
    float w_post[kKeep ? GROUPS : 1][E], w_pre[kKeep ? GROUPS : 1][E];
    if (kKeep) {
#pragma unroll
        for (int j = 0; j < GROUPS; ++j)
            if (at(j) < p.d) {
                if (p.w_post) load_floats<E>(p.w_post + at(j), w_post[j]);
                if (p.w_pre) load_floats<E>(p.w_pre + at(j), w_pre[j]);
            }
    }
    int n = 0;
    for (int64_t t = first; t < p.T; t += stride, ++n) {
        const int64_t row = t * p.d;
        if (RING) {
            fetch(n + p.ahead);
            if (p.ahead == 1) copy_wait<1>();
            else copy_wait<3>();
        }
        float r[GROUPS][E], u[GROUPS][E];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            if (at(j) >= p.d) continue;
            unpack(RING ? *reinterpret_cast<const uint4*>(slot(n, 0, 16, j))
                        : *reinterpret_cast<const uint4*>(static_cast<const Res*>(p.residual) + row + at(j)), r[j]);
            if (p.y)
                unpack(RING ? *reinterpret_cast<const Half*>(slot(n, S::kY, S::kHalf, j))
                            : *reinterpret_cast<const Half*>(p.y + row + at(j)), u[j]);
        }
        if (p.y) {
            if (p.w_post) {
#pragma unroll
                for (int j = 0; j < GROUPS; ++j)
                    if (at(j) < p.d) {
#pragma unroll
                        for (int i = 0; i < E; ++i) sum += u[j][i] * u[j][i];
                    }
                const float f = rsqrtf(row_sum<CTA>(sum, part[n & 1][0]) / p.d + p.eps);
#pragma unroll
                for (int j = 0; j < GROUPS; ++j)
                    if (at(j) < p.d) {
                        float w[E];
                        if (!kKeep) load_floats<E>(p.w_post + at(j), w);
#pragma unroll
                        for (int i = 0; i < E; ++i) u[j][i] = u[j][i] * f * (kKeep ? w_post[kKeep ? j : 0][i] : w[i]);
                    }
            }
            float token = 0.0f;
            if (GATE == MOE_GATE_TOKEN) token = __ldg(static_cast<const float*>(p.gate) + t);
#pragma unroll
            for (int j = 0; j < GROUPS; ++j) {
                if (at(j) >= p.d) continue;
                float g[E];
                if (GATE == MOE_GATE_TOKEN) {
#pragma unroll
                    for (int i = 0; i < E; ++i) g[i] = token;
                } else if (GATE == MOE_GATE_CHANNEL) {
                    load_floats<E>(static_cast<const float*>(p.gate) + at(j), g);
                } else if (GATE == MOE_GATE_FULL) {
                    unpack(RING ? *reinterpret_cast<const Half*>(slot(n, S::kG, S::kHalf, j))
                                : *reinterpret_cast<const Half*>(static_cast<const uint16_t*>(p.gate) + row + at(j)), g);
                }
                if (GATE != MOE_GATE_NONE) {
                    // (the approximate quotient, two units of fp32; __expf has 2 + 1.2 |g|: for large |g| the gate is near 0, where
                    // that is lost beside the residual, or near 1, where the exponential hardly counts)
#pragma unroll
                    for (int i = 0; i < E; ++i) u[j][i] *= sigmoid ? __fdividef(1.0f, 1.0f + __expf(-g[i])) : g[i];
                }
#pragma unroll
                for (int i = 0; i < E; ++i) r[j][i] += p.scale * u[j][i];
                store(static_cast<Res*>(p.residual_out) + row + at(j), r[j]);
            }
        }
        if (!p.w_pre) continue;
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < GROUPS; ++j)
            if (at(j) < p.d) {
#pragma unroll
                for (int i = 0; i < E; ++i) sum += r[j][i] * r[j][i];
            }
        const float f = rsqrtf(row_sum<CTA>(sum, part[n & 1][1]) / p.d + p.eps);
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            if (at(j) >= p.d) continue;
            float w[E];
            if (!kKeep) load_floats<E>(p.w_pre + at(j), w);
#pragma unroll
            for (int i = 0; i < E; ++i) r[j][i] = r[j][i] * f * (kKeep ? w_pre[kKeep ? j : 0][i] : w[i]);
            store(p.x + row + at(j), r[j]);
        }
    }
}

constexpr int64_t kRing = 220 * 1024;  // shared memory of an SM for rows on the way

template <typename Res, int GATE, bool CTA, int ELEMS, int MAX, bool RING>
cudaError_t launch_kernel(NormParams p, bool sigmoid, int threads, cudaStream_t st) {
    auto* kernel = block_norm_kernel<Res, GATE, CTA, ELEMS, MAX, RING>;
    const int64_t rows = CTA ? p.T : ((int64_t)p.T + 7) / 8, sms = sm_count();
    if (!RING) {
        kernel<<<(unsigned)rows, threads, 0, st>>>(p, sigmoid);
        return cudaGetLastError();
    }
    // More rows on the way where CTAs walk many of them and shared memory holds two CTAs; else more CTAs.
    const int64_t slot = Slot<Res, GATE, ELEMS * (int)sizeof(Res) / 16>::kBytes * threads;
    p.ahead = 8 * slot <= kRing && rows > 4 * sms ? 3 : 1;
    const int64_t smem = (p.ahead + 1) * slot;
    const cudaError_t err = ensure_dynamic_smem((const void*)kernel, smem + 1024);  // (the sums' place counts too)
    if (err != cudaSuccess) return err;
    // as many CTAs as are at work at once
    const int64_t most = sms * std::max<int64_t>(1, std::min<int64_t>(kRing / smem, 1024 / threads));
    kernel<<<(unsigned)std::min(rows, most), threads, smem, st>>>(p, sigmoid);
    return cudaGetLastError();
}

template <typename Res, int GATE>
cudaError_t launch_gate(const NormParams& p, bool sigmoid, cudaStream_t st) {
    auto threads = [&](int elems) { return (p.d + 32 * elems - 1) / (32 * elems) * 32; };
    if (p.d <= 512) return launch_kernel<Res, GATE, false, 16, 256, true>(p, sigmoid, 256, st);
    if (p.d <= kWarpRow) return launch_kernel<Res, GATE, false, 32, 256, true>(p, sigmoid, 256, st);
    // (bounds for 640 threads: at most 102 registers, so that two CTAs of up to 320 threads fit an SM; with 106, 257 rows
    // of 5000 took 5.9 us, with 102 4.3)
    if (p.d <= 8192) return launch_kernel<Res, GATE, true, 16, 640, true>(p, sigmoid, threads(16), st);
    if (p.d <= 16384) {
        // (two rows of all there is in fp32 do not fit shared memory)
        constexpr bool kFits = 2 * Slot<Res, GATE, (int)sizeof(Res)>::kBytes * 1024 <= kRing;
        return launch_kernel<Res, GATE, true, 16, 1024, kFits>(p, sigmoid, threads(16), st);
    }
    return launch_kernel<Res, GATE, true, 32, 1024, false>(p, sigmoid, threads(32), st);
}

template <typename Res>
cudaError_t launch_res(const NormParams& p, int gate, bool sigmoid, cudaStream_t st) {
    switch (gate) {
        case MOE_GATE_NONE: return launch_gate<Res, MOE_GATE_NONE>(p, sigmoid, st);
        case MOE_GATE_TOKEN: return launch_gate<Res, MOE_GATE_TOKEN>(p, sigmoid, st);
        case MOE_GATE_CHANNEL: return launch_gate<Res, MOE_GATE_CHANNEL>(p, sigmoid, st);
        case MOE_GATE_FULL: return launch_gate<Res, MOE_GATE_FULL>(p, sigmoid, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_block_norm(const uint16_t* y, const void* residual, const void* gate, const float* w_post,
                              const float* w_pre, const moe_norm_dims_t& d, void* residual_out, uint16_t* x,
                              cudaStream_t st) {
    const NormParams p{y, residual, gate, w_post, w_pre, residual_out, x, d.T, d.d, d.eps, d.scale, 1};
    const bool sigmoid = d.flags & MOE_NORM_SIGMOID;
    return d.flags & MOE_NORM_RESIDUAL_F32 ? launch_res<float>(p, d.gate, sigmoid, st)
                                           : launch_res<uint16_t>(p, d.gate, sigmoid, st);
}

}  // namespace moe
