// Projections of few tokens in microscaled 4-bit floats, on the CUDA cores: one launch, which quantises the tokens too.
//
// A warp takes the four weight rows whose block scales lie together (rows r, r + 32, r + 64, r + 96 of a scale tile:
// 16 bytes hold their scales of 64 elements), a lane 64 elements of each at a time: 32 bytes of codes per row and those 16.
// The weights are read once, a step ahead, the first without waiting for anything; meanwhile every CTA quantises the tokens for
// itself, a block of 16 to a thread, and keeps them as f16 values in shared memory.  Products of two codes are multiples of 1/4 of at most 36,
// so eight of them add up exactly in f16; a block's sum and its two scales meet in fp32.
//
// What bounds a call is the weights' bytes and the time until the first arrive: with four rows to a warp and two steps on the
// way, all of a decode step's projection is in flight at once.
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
    int N, K;
    int parts;  // warps that share four rows, each a part of K; above 1 only where a CTA's warps have one turn each
};

// Eight codes as f16 values.  (By conversion: putting the bits in place by hand takes four operations for two codes and
// was 5% slower.)
__device__ __forceinline__ void values_of_8(uint32_t c, __half2 (&v)[4]) {
    uint32_t u[4];
    asm("{\n .reg .b8 p, q, r, s;\n mov.b32 {p, q, r, s}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, p;\n cvt.rn.f16x2.e2m1x2 %1, q;\n"
        " cvt.rn.f16x2.e2m1x2 %2, r;\n cvt.rn.f16x2.e2m1x2 %3, s;\n}"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const __half2*>(&u[i]);
}
// Four E4M3 scales as fp32.
__device__ __forceinline__ void scales_of_4(uint32_t b, float (&f)[4]) {
    uint32_t u[2];
    asm("{\n .reg .b16 p, q;\n mov.b32 {p, q}, %2;\n cvt.rn.f16x2.e4m3x2 %0, p;\n cvt.rn.f16x2.e4m3x2 %1, q;\n}"
        : "=r"(u[0]), "=r"(u[1])
        : "r"(b));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
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
    const int atoms = p.K / 64, blocks = p.K / 16;
    float* bx = reinterpret_cast<float*>(smem + T * atoms * kAtomBytes);  // [T][K / 16] the tokens' block scales
    // Turns: four rows (of which `parts` warps take a part of K each), 32 lanes' atoms at a time.  CTAs take neighbouring turns,
    // so that every SM gets as many.
    const int part = warp % p.parts, teams = kWarps / p.parts;
    const int groups = (p.N + 127) / 128 * 32, stride = gridDim.x * teams;
    int group = warp / p.parts * gridDim.x + blockIdx.x, a = part * 32 + lane;
    auto load = [&](int group, int a) {
        Step s;
        const int tile = group >> 5, r0 = tile * 128 + (group & 31);
        const uint8_t* q = p.w.q + (int64_t)r0 * (p.K / 2) + 32 * a;
        const bool live = group < groups && a < atoms;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s.q[i][0] = s.q[i][1] = make_uint4(0, 0, 0, 0);
            if (live && r0 + 32 * i < p.N) {
                const uint4* from = reinterpret_cast<const uint4*>(q + (int64_t)i * 16 * p.K);
                s.q[i][0] = __ldg(from);
                s.q[i][1] = __ldg(from + 1);
            }
        }
        s.b = make_uint4(0, 0, 0, 0);
        if (live) s.b = __ldg(reinterpret_cast<const uint4*>(p.w.b + ((int64_t)tile * atoms + a) * 512 + (group & 31) * 16));
        return s;
    };
    Step now = load(group, a);

    // the tokens: their largest magnitudes first, then codes as the values they stand for
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
        float m = part_max[t][0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) m = fmaxf(m, part_max[t][i]);
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
            __half2 v[2][4];
            values_of_8(c.x, v[0]);
            values_of_8(c.y, v[1]);
            uint4* to = reinterpret_cast<uint4*>(smem + (t * atoms + j / 4) * kAtomBytes + 32 * (j & 3));
            to[0] = *reinterpret_cast<const uint4*>(v[0]);
            to[1] = *reinterpret_cast<const uint4*>(v[1]);
        }
    }
    __syncthreads();

    float acc[T][4] = {};
    while (group < groups) {
        // the next step's weights are on the way while this one's are used
        const int step = 32 * p.parts, last = a - lane + step >= atoms;  // (the same for the warp)
        const int next_group = last ? group + stride : group, next_a = last ? part * 32 + lane : a + step;
        const Step next = load(next_group, next_a);
        if (a < atoms) {
            float bw[4][4];
            scales_of_4(now.b.x, bw[0]);
            scales_of_4(now.b.y, bw[1]);
            scales_of_4(now.b.z, bw[2]);
            scales_of_4(now.b.w, bw[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // blocks of 16
                __half2 w[4][2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 q = now.q[i][j / 2];
                    values_of_8(j & 1 ? q.z : q.x, w[i][0]);
                    values_of_8(j & 1 ? q.w : q.y, w[i][1]);
                }
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const uint4* from = reinterpret_cast<const uint4*>(smem + (t * atoms + a) * kAtomBytes + 32 * j);
                    const uint4 u[2] = {from[0], from[1]};
                    const __half2* v = reinterpret_cast<const __half2*>(u);
                    const float b = bx[t * blocks + 4 * a + j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        __half2 s = __hmul2(w[i][0][0], v[0]);
#pragma unroll
                        for (int n = 1; n < 8; ++n) s = __hfma2(w[i][n / 4][n % 4], v[n], s);
                        const float2 f = __half22float2(s);
                        acc[t][i] += (f.x + f.y) * (b * bw[i][j]);
                    }
                }
            }
        }
        if (last) {
            const int64_t r = group / 32 * 128 + group % 32 + 32 * (lane & 3);
#pragma unroll
            for (int t = 0; t < T; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) acc[t][i] += __shfl_xor_sync(0xFFFFFFFFu, acc[t][i], o);
                const float v = lane == 0 ? acc[t][0] : lane == 1 ? acc[t][1] : lane == 2 ? acc[t][2] : acc[t][3];
                if (p.parts > 1) {
                    if (lane < 4) sums[t][lane][warp] = v;
                } else if (lane < 4 && r < p.N) {
                    p.out[(int64_t)t * p.N + r] = float_to_bf16_bits(v * sx[t] * __ldg(p.w.s + r));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
            }
        }
        now = next;
        group = next_group;
        a = next_a;
    }
    if (p.parts == 1) return;
    // the parts of K in order
    __syncthreads();
    const int team = threadIdx.x / 4, i = threadIdx.x % 4, mine = team * gridDim.x + blockIdx.x;
    if (team < teams && mine < groups) {
        const int64_t r = mine / 32 * 128 + mine % 32 + 32 * i;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float v = 0.0f;
            for (int k = 0; k < p.parts; ++k) v += sums[t][i][team * p.parts + k];
            if (r < p.N) p.out[(int64_t)t * p.N + r] = float_to_bf16_bits(v * sx[t] * __ldg(p.w.s + r));
        }
    }
}

template <int T>
cudaError_t launch(GemvParams p, cudaStream_t st) {
    const size_t smem = (size_t)T * (p.K / 64 * kAtomBytes + p.K / 16 * 4);
    cudaError_t err = ensure_dynamic_smem((const void*)gemv_kernel<T>, smem + 1024);
    if (err != cudaSuccess) return err;
    // Where the rows leave warps idle, several share one's K, as long as each has a step of 32 lanes.
    const int groups = (p.N + 127) / 128 * 32, warps = sm_count() * 2 * kWarps;
    while (p.parts < kWarps && groups * p.parts * 2 <= warps && p.K / 64 >= 64 * p.parts) p.parts *= 2;
    gemv_kernel<T><<<std::min(groups, sm_count() * 2), kThreads, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

// One or two tokens whose rows fit shared memory as f16, on weights small enough; a row of weights costs as much as some 1024
// more of K.  Here and by the tensor cores, quantisation included, us: one token, N = 1024, K = 4096 4.1, 6.7; N = 6144 6.0, 7.3; N = 8192
// 6.4, 7.4; N = 6144, K = 8192 8.9, 8.5; N = 16384, K = 4096 9.5, 8.7; N = 32768, K = 512 8.6, 5.6; two tokens, N = 1024, K = 4096 5.8,
// 6.8; N = 4096, K = 2048 5.4, 6.0; K = 4096 7.5, 6.8; N = 6144 8.9, 7.5; three at N = 6144 12.4, 7.4.
bool gemv_fp4_takes(int T, int N, int K) {
    return T <= 2 && T * K <= 32768 && (int64_t)N * (K + 1024) < (T == 1 ? 3 << 24 : 7 << 21);
}

cudaError_t launch_gemv_fp4(const uint16_t* x, int64_t ldx, moe_fp4_t w, int T, int N, int K, uint16_t* out,
                            cudaStream_t st) {
    const GemvParams p{x, ldx, w, out, N, K, 1};
    return T == 1 ? launch<1>(p, st) : launch<2>(p, st);
}

}  // namespace moe
