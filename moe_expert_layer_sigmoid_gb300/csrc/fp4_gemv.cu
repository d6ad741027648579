// Projections of one or a few tokens in microscaled 4-bit floats, on the CUDA cores: one launch, which quantises
// the tokens too.
//
// A warp takes the four weight rows whose block scales lie together (rows r, r + 32, r + 64, r + 96 of a scale tile:
// 16 bytes hold their scales of 64 elements), a lane 64 elements of each at a time: 32 bytes of codes per row and those 16.
// The weights are read once and wait for nothing; meanwhile every CTA quantises the tokens for itself, a block
// of 16 to a thread, and keeps them as f16 values in shared memory.  Products of two codes are multiples of 1/4 of at most 36,
// so eight of them add up exactly in f16; a block's sum and its two scales meet in fp32.
//
// What bounds a call is the weights' bytes and the time until the first arrive: with four rows to a warp, all of a decode
// step's projection is in flight at once.
#include "fp4_dev.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kAtomBytes = 64 * 2 + 16;  // a token's 64 values in f16; the gap spreads lanes over the banks

struct GemvParams {
    const uint16_t* x;
    int64_t ldx;
    moe_fp4_t w;
    uint16_t* out;
    int N, K, parts;  // parts: warps that share four rows, each a part of K
};

// Two codes as f16 values.  (By conversion: putting the bits in place by hand takes four operations and was 5% slower.)
__device__ __forceinline__ __half2 code_pair(uint32_t byte) {
    const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1);
    return *reinterpret_cast<const __half2*>(&hr);
}

// A lane's weights of one step: 64 elements of four rows and their block scales.
struct Step {
    uint4 q[4][2];
    uint4 b;  // word i: row i's four scales
};

template <int T>
__global__ void __launch_bounds__(kThreads, 2) gemv_kernel(const GemvParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part_max[T][kWarps], sums[T][4][kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int atoms = p.K / 64;
    float* bx = reinterpret_cast<float*>(smem + T * atoms * kAtomBytes);  // [T][K / 16] the tokens' block scales
    // the warp's rows
    const int64_t group = ((int64_t)blockIdx.x * kWarps + warp) / p.parts;
    const int64_t tile = group / 32, r0 = tile * 128 + group % 32;
    const int part = warp % p.parts;
    auto load = [&](int a) {
        Step s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 32 * i;
            const uint4* q = reinterpret_cast<const uint4*>(p.w.q + r * (p.K / 2) + 32 * a);
            s.q[i][0] = s.q[i][1] = make_uint4(0, 0, 0, 0);
            if (r < p.N) {
                s.q[i][0] = __ldg(q);
                s.q[i][1] = __ldg(q + 1);
            }
        }
        s.b = __ldg(reinterpret_cast<const uint4*>(p.w.b + (tile * atoms + a) * 512 + group % 32 * 16));
        return s;
    };
    int a = part * 32 + lane;
    const bool live = r0 < p.N;
    Step now;
    if (live && a < atoms) now = load(a);

    // the tokens: largest magnitudes first, then codes as the values they stand for
    const int blocks = p.K / 16;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        float m = 0.0f;
        for (int j = threadIdx.x; j < blocks; j += kThreads) {
            float f[16];
            load16(p.x + t * p.ldx + 16 * j, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(f[i]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (lane == 0) part_max[t][warp] = m;
    }
    __syncthreads();
    float sx[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) m = fmaxf(m, part_max[t][i]);
        const RowScale row = row_scale(m);
        sx[t] = row.s;
        for (int j = threadIdx.x; j < blocks; j += kThreads) {
            float f[16];
            load16(p.x + t * p.ldx + 16 * j, f);
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(f[i]));
            uint2 c;
            const uint32_t b = quant_block<true>(f, top, row, c);
            bx[t * blocks + j] = e4m3_value(b);
            __half2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = code_pair((i < 4 ? c.x : c.y) >> (8 * (i & 3)) & 0xFFu);
            uint4* to = reinterpret_cast<uint4*>(smem + (t * atoms + j / 4) * kAtomBytes + 32 * (j & 3));
            to[0] = reinterpret_cast<const uint4*>(v)[0];
            to[1] = reinterpret_cast<const uint4*>(v)[1];
        }
    }
    __syncthreads();

    float acc[T][4] = {};
    while (live && a < atoms) {
        const int next = a + 32 * p.parts;
        Step then;
        if (next < atoms) then = load(next);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // blocks of 16
            __half2 w[4][8];
            float bw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 q = now.q[i][j / 2];
                const uint32_t lo = j & 1 ? q.z : q.x, hi = j & 1 ? q.w : q.y;
#pragma unroll
                for (int n = 0; n < 8; ++n) w[i][n] = code_pair((n < 4 ? lo : hi) >> (8 * (n & 3)) & 0xFFu);
                bw[i] = e4m3_value((i == 0 ? now.b.x : i == 1 ? now.b.y : i == 2 ? now.b.z : now.b.w) >> (8 * j) & 0xFFu);
            }
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const uint4* from = reinterpret_cast<const uint4*>(smem + (t * atoms + a) * kAtomBytes + 32 * j);
                const uint4 u[2] = {from[0], from[1]};
                const __half2* v = reinterpret_cast<const __half2*>(u);
                const float b = bx[t * blocks + 4 * a + j];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    __half2 s = __hmul2(w[i][0], v[0]);
#pragma unroll
                    for (int n = 1; n < 8; ++n) s = __hfma2(w[i][n], v[n], s);
                    const float2 f = __half22float2(s);
                    acc[t][i] += (f.x + f.y) * (b * bw[i]);
                }
            }
        }
        now = then;
        a = next;
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[t][i] += __shfl_xor_sync(0xFFFFFFFFu, acc[t][i], o);
            if (lane == 0) sums[t][i][warp] = acc[t][i];
        }
    __syncthreads();
    // one thread per output: warps' parts in order
    const int per = kWarps / p.parts;  // groups of the CTA
    if ((int)threadIdx.x < per * 4 * T) {
        const int g = threadIdx.x % per, i = threadIdx.x / per % 4, t = threadIdx.x / (per * 4);
        const int64_t gg = (int64_t)blockIdx.x * per + g, r = gg / 32 * 128 + gg % 32 + 32 * i;
        if (r < p.N) {
            float v = 0.0f;
            for (int k = 0; k < p.parts; ++k) v += sums[t][i][g * p.parts + k];
            float scale = sx[0];
#pragma unroll
            for (int n = 1; n < T; ++n) scale = t == n ? sx[n] : scale;
            p.out[(int64_t)t * p.N + r] = float_to_bf16_bits(v * scale * __ldg(p.w.s + r));
        }
    }
}

template <int T>
cudaError_t launch(const GemvParams& p, cudaStream_t st) {
    const size_t smem = (size_t)T * (p.K / 64 * kAtomBytes + p.K / 16 * 4);
    cudaError_t err = ensure_dynamic_smem((const void*)gemv_kernel<T>, smem);
    if (err != cudaSuccess) return err;
    const int64_t groups = (int64_t)((p.N + 127) / 128) * 32;
    gemv_kernel<T><<<(unsigned)((groups * p.parts + kWarps - 1) / kWarps), kThreads, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

// One token (2: 10.4 us against 9.0 for the tensor cores at N = 6144, K = 4096), and a row that fits shared memory as f16.
bool gemv_fp4_takes(int T, int K) { return T <= kGemvFp4Tokens && T * K <= 16384; }

cudaError_t launch_gemv_fp4(const uint16_t* x, int64_t ldx, moe_fp4_t w, int T, int N, int K, uint16_t* out,
                            cudaStream_t st) {
    GemvParams p{x, ldx, w, out, N, K, 1};
    // warps for every SM: rows that are too few are shared, as long as each warp has a step of 32 lanes
    const int64_t groups = (int64_t)((N + 127) / 128) * 32;
    while (p.parts < kWarps && groups * p.parts < (int64_t)sm_count() * kWarps && K / 64 >= 64 * p.parts) p.parts *= 2;
    switch (T) {
        case 1: return launch<1>(p, st);
        case 2: return launch<2>(p, st);
        case 3: return launch<3>(p, st);
        default: return launch<4>(p, st);
    }
}

}  // namespace moe
