// The norms between two blocks, fused with the gate, the scale and the residual
// between them: one launch, one pass over memory.
//
// A row stays in the registers of its threads from the first load to the last store, so the two sums of
// squares cost exchanges only; the bound is DRAM bandwidth, and for a few rows the launch and two exchanges.
// Rows of at most kWarpRow elements take a warp each, longer ones a CTA.  Sums are fp32, in an order that
// the row's length alone sets.
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
};

constexpr int kWarpRow = 1024;  // longest row of one warp: 4 pieces of 8 elements to a lane

__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    f[0] = bf16_lo(x.x); f[1] = bf16_hi(x.x); f[2] = bf16_lo(x.y); f[3] = bf16_hi(x.y);
    f[4] = bf16_lo(x.z); f[5] = bf16_hi(x.z); f[6] = bf16_lo(x.w); f[7] = bf16_hi(x.w);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ uint32_t pair(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// The sum over a row's threads: a warp, or the CTA (`part`, of which each call of a kernel has its own).
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

template <typename Res, int GATE, bool CTA, int PIECES>
__global__ void __launch_bounds__(CTA ? 1024 : 256) block_norm_kernel(const NormParams p, bool sigmoid) {
    __shared__ float part[2][32];
    const int threads = CTA ? blockDim.x : 32, me = CTA ? threadIdx.x : threadIdx.x & 31;
    const int64_t t = CTA ? blockIdx.x : (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int64_t row = t * p.d;
    const Res* residual = static_cast<const Res*>(p.residual) + row;
    float r[PIECES][8], u[PIECES][8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
        const int at = 8 * (me + j * threads);
        if (at < p.d) {
            load8(residual + at, r[j]);
            if (p.y) load8(p.y + row + at, u[j]);
        }
    }
    if (p.y) {
        if (p.w_post) {
#pragma unroll
            for (int j = 0; j < PIECES; ++j)
                if (8 * (me + j * threads) < p.d) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum += u[j][i] * u[j][i];
                }
            const float f = rsqrtf(row_sum<CTA>(sum, part[0]) / p.d + p.eps);
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                const int at = 8 * (me + j * threads);
                if (at < p.d) {
                    float w[8];
                    load8(p.w_post + at, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[j][i] = u[j][i] * f * w[i];
                }
            }
        }
        float token = 0.0f;
        if (GATE == MOE_GATE_TOKEN) token = static_cast<const float*>(p.gate)[t];
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int at = 8 * (me + j * threads);
            if (at >= p.d) continue;
            float g[8];
            if (GATE == MOE_GATE_TOKEN) {
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = token;
            } else if (GATE == MOE_GATE_CHANNEL) {
                load8(static_cast<const float*>(p.gate) + at, g);
            } else if (GATE == MOE_GATE_FULL) {
                load8(static_cast<const uint16_t*>(p.gate) + row + at, g);
            }
            if (GATE != MOE_GATE_NONE) {
#pragma unroll
                for (int i = 0; i < 8; ++i) u[j][i] *= sigmoid ? 1.0f / (1.0f + __expf(-g[i])) : g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] += p.scale * u[j][i];
            store8(static_cast<Res*>(p.residual_out) + row + at, r[j]);
        }
    }
    if (!p.w_pre) return;
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
        if (8 * (me + j * threads) < p.d) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += r[j][i] * r[j][i];
        }
    const float f = rsqrtf(row_sum<CTA>(sum, part[1]) / p.d + p.eps);
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
        const int at = 8 * (me + j * threads);
        if (at >= p.d) continue;
        float w[8];
        load8(p.w_pre + at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] * f * w[i];
        store8(p.x + row + at, r[j]);
    }
}

template <typename Res, int GATE>
cudaError_t launch_gate(const NormParams& p, bool sigmoid, cudaStream_t st) {
    const int pieces = p.d / 8;  // of a row
    if (p.d <= kWarpRow) {
        const unsigned grid = (unsigned)(((int64_t)p.T + 7) / 8);
        if (pieces <= 64) block_norm_kernel<Res, GATE, false, 2><<<grid, 256, 0, st>>>(p, sigmoid);
        else block_norm_kernel<Res, GATE, false, 4><<<grid, 256, 0, st>>>(p, sigmoid);
    } else {
        const int per = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
        const int threads = ((pieces + per - 1) / per + 31) / 32 * 32;
        if (per == 1) block_norm_kernel<Res, GATE, true, 1><<<p.T, threads, 0, st>>>(p, sigmoid);
        else if (per == 2) block_norm_kernel<Res, GATE, true, 2><<<p.T, threads, 0, st>>>(p, sigmoid);
        else block_norm_kernel<Res, GATE, true, 4><<<p.T, threads, 0, st>>>(p, sigmoid);
    }
    return cudaGetLastError();
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
    const NormParams p{y, residual, gate, w_post, w_pre, residual_out, x, d.T, d.d, d.eps, d.scale};
    const bool sigmoid = d.flags & MOE_NORM_SIGMOID;
    return d.flags & MOE_NORM_RESIDUAL_F32 ? launch_res<float>(p, d.gate, sigmoid, st)
                                           : launch_res<uint16_t>(p, d.gate, sigmoid, st);
}

}  // namespace moe
