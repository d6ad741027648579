// Rows to 4-bit floats with a scale for each 16 of them, and back.
//
//   s = absmax(row) / 2688,  b = e4m3(absmax(block) / (6 s)),  code = e2m1(x / (b s))
// A row is read once, into registers.  The way there is bound by instructions as much as by bytes (a quotient per element that
// has to be the rounded one): 8191 bf16 rows of 4096 18.1 us, 4.8 TB/s (18.8 with no row in L2).  The way back by bytes: 12.8 us
// where L2 takes what is written, 16.3 with other rows each time, 5.3 TB/s.  Weights, fp32, once per load: 6144 rows of 4096
// 27.6 us, 4.2 TB/s, 4096 of 16384 93, 3.3.
// Rows past 16384 take four blocks of 16 fp32 values to a thread, which 64 registers do not hold (148 bytes to local memory
// and 248 back, fp32 880 and 672): 2048 bf16 rows of 18432 37 us, 2.6 TB/s, of 28672 49, 3.1; fp32 4096 of 18432 192, 1.8.
#include "fp4_dev.cuh"

namespace moe {
namespace {

// The larger magnitude of either half.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_abs(uint4 a, uint4 b) {
    const uint32_t m = max_abs2(max_abs2(max_abs2(a.x, a.y), max_abs2(a.z, a.w)),
                                max_abs2(max_abs2(b.x, b.y), max_abs2(b.z, b.w)));
    return fmaxf(fabsf(bf16_lo(m)), fabsf(bf16_hi(m)));
}

// blockDim.x threads (whole warps) take a row, blockDim.y rows a CTA, a thread NB blocks: all of a row is in registers
// at once.  What bounds it is instructions (some hundred for a block) as much as bytes, so that many rows get few
// threads each: what is done once per thread and row, the exchange of the largest magnitude above all, is spread over NB blocks.
template <int NB>
__global__ void __launch_bounds__(512) quant_bf16_kernel(const uint16_t* __restrict__ src, int64_t ld, int rows, int K,
                                                          Fp4Rows out) {
    __shared__ float part[16];
    pdl_trigger();  // the projection's kernel fetches weights meanwhile
    const int blocks = K / 16, lane = threadIdx.x & 31, warps = blockDim.x >> 5;  // warps of a row
    const int r = blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = r < rows;
    const uint4* from = reinterpret_cast<const uint4*>(src + r * ld) + 2 * threadIdx.x;
    uint4 x[NB][2];
    float m[NB], top = 0.0f;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
        if (live && (int)(threadIdx.x + j * blockDim.x) < blocks) {
            x[j][0] = __ldg(from + 2 * j * blockDim.x);
            x[j][1] = __ldg(from + 2 * j * blockDim.x + 1);
        }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        m[j] = max_abs(x[j][0], x[j][1]);
        top = fmaxf(top, m[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (warps > 1) {
        float* tops = part + threadIdx.y * warps;
        if (lane == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
        top = tops[0];
        for (int i = 1; i < warps; ++i) top = fmaxf(top, tops[i]);
    }
    if (!live) return;
    const RowScale q = row_scale(top);
    uint8_t* to = out.q + (int64_t)r * (K / 2) + 8 * threadIdx.x;
    uint8_t* scales = out.b + (int64_t)(r >> 7) * (K * 8) + (r & 31) * 16 + (r >> 5 & 3) * 4 + threadIdx.x / 4 * 512;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const bool mine = (int)(threadIdx.x + j * blockDim.x) < blocks;
        float f[16];
        load16(x[j], f);
        uint2 c;
        uint32_t b = quant_block<true>(f, m[j], q, c);
        if (mine) *reinterpret_cast<uint2*>(to + 8 * j * blockDim.x) = c;
        // four blocks' scales lie together
        b |= __shfl_down_sync(0xFFFFFFFFu, b, 1) << 8;
        b |= __shfl_down_sync(0xFFFFFFFFu, b, 2) << 16;
        if (mine && lane % 4 == 0) *reinterpret_cast<uint32_t*>(scales + 128 * j * blockDim.x) = b;
    }
    if (threadIdx.x == 0) out.s[r] = q.s;
}

// Weights, and rows too long for a thread a block: PER blocks to a thread, read in their place.  Once per load.
template <typename Src, int PER>
__global__ void __launch_bounds__(1024) quant_kernel(const Src* __restrict__ src, int64_t ld, int64_t rows, int K,
                                                     Fp4Rows out) {
    __shared__ float part[2][32];
    pdl_trigger();
    const int blocks = K / 16, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    int flip = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, flip ^= 1) {
        float f[PER][16], m[PER], top = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int at = threadIdx.x + j * blockDim.x;
            m[j] = 0.0f;
            if (at < blocks) {
                load16(src + r * ld + 16 * at, f[j]);
#pragma unroll
                for (int i = 0; i < 16; ++i) m[j] = fmaxf(m[j], fabsf(f[j][i]));
            }
            top = fmaxf(top, m[j]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (lane == 0) part[flip][threadIdx.x >> 5] = top;
        __syncthreads();
        top = lane < warps ? part[flip][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const RowScale q = row_scale(top);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int at = threadIdx.x + j * blockDim.x;
            if (at >= blocks) break;
            uint2 c;
            const uint32_t b = quant_block<sizeof(Src) == 2>(f[j], m[j], q, c);
            *reinterpret_cast<uint2*>(out.q + r * (K / 2) + 8 * at) = c;
            out.b[fp4_scale_at(r, at, K)] = (uint8_t)b;
        }
        if (threadIdx.x == 0) out.s[r] = q.s;
    }
}

// threads.x threads take a row, threads.y rows a CTA; a thread 8 elements at a time, so that a warp's stores are whole
// lines, several of them on the way together.
__global__ void __launch_bounds__(256) unpack_kernel(moe_fp4_t w, int64_t rows, int K, uint16_t* __restrict__ out) {
    constexpr int kBatch = 4;
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (r >= rows) return;
    const float s = __ldg(w.s + r);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(w.q + r * (K / 2));
    uint4* to = reinterpret_cast<uint4*>(out + r * K);
    for (int at = threadIdx.x; at < K / 8; at += kBatch * blockDim.x) {
        uint32_t c[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int p = at + i * blockDim.x;
            if (p < K / 8) {
                c[i] = __ldg(q + p);
                b[i] = __ldg(w.b + fp4_scale_at(r, p / 2, K));
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int p = at + i * blockDim.x;
            if (p >= K / 8) break;
            const float t = e4m3_value(b[i]) * s;
            uint32_t o[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(c[i] >> (8 * n) & 0xFFu), __NV_E2M1);
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                const __nv_bfloat162 u = __floats2bfloat162_rn(v.x * t, v.y * t);
                o[n] = *reinterpret_cast<const uint32_t*>(&u);
            }
            to[p] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

template <typename Src, int PER>
cudaError_t launch_plain(const Src* src, int64_t ld, int64_t rows, int64_t K, const Fp4Rows& out, cudaStream_t st) {
    const int x = (int)((K / 16 + 32 * PER - 1) / (32 * PER) * 32);
    const int64_t most = (int64_t)sm_count() * std::max(1, 2048 / x);
    quant_kernel<Src, PER><<<(unsigned)std::min(rows, most), x, 0, st>>>(src, ld, rows, (int)K, out);
    return cudaGetLastError();
}

template <typename Src>
cudaError_t launch_any(const Src* src, int64_t ld, int64_t rows, int64_t K, const Fp4Rows& out, cudaStream_t st) {
    return K <= 16384 ? launch_plain<Src, 1>(src, ld, rows, K, out, st)
                      : launch_plain<Src, 4>(src, ld, rows, K, out, st);
}

template <int NB>
cudaError_t launch_bf16(const uint16_t* x, int64_t ld, int64_t rows, int64_t K, const Fp4Rows& out, cudaStream_t st) {
    const int tx = (int)((K / 16 + 32 * NB - 1) / (32 * NB) * 32), ty = std::max(1, 256 / tx);
    quant_bf16_kernel<NB><<<(unsigned)((rows + ty - 1) / ty), dim3(tx, ty), 0, st>>>(x, ld, (int)rows, (int)K, out);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_fp4(const void* src, bool bf16, int64_t ld, int64_t rows, int64_t K, Fp4Rows out,
                             cudaStream_t st) {
    const int64_t sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    if (!bf16) return launch_any(static_cast<const float*>(src), ld, rows, K, out, st);
    const uint16_t* x = static_cast<const uint16_t*>(src);
    if (K > 16384) return launch_any(x, ld, rows, K, out, st);
    // Blocks to a thread, by how many blocks there are for a full house of threads (1024 on every SM).  1, 2 and 4 to a
    // thread, us: 128 rows of 4096 (0.2 full) 2.2, 2.3, 3.0; 2048 rows (3.4) 6.3, 5.5, 5.8; 8191 rows (13) 22.5, 19.2, 18.1
    const int64_t blocks = K / 16, full = rows * blocks / (sms * 1024);
    if (full >= 6 && blocks >= 128) return launch_bf16<4>(x, ld, rows, K, out, st);
    if (blocks > 512 || (full >= 1 && blocks >= 64)) return launch_bf16<2>(x, ld, rows, K, out, st);
    return launch_bf16<1>(x, ld, rows, K, out, st);
}

cudaError_t launch_unpack_fp4(moe_fp4_t w, int64_t rows, int64_t K, uint16_t* out, cudaStream_t st) {
    const int pieces = (int)(K / 8), x = pieces >= 256 ? 128 : pieces >= 64 ? 32 : 8, y = 256 / x;
    unpack_kernel<<<(unsigned)((rows + y - 1) / y), dim3(x, y), 0, st>>>(w, rows, (int)K, out);
    return cudaGetLastError();
}

}  // namespace moe
