// Attention of new tokens over the paged cache, one CTA per token and query
// head: scores of 128 keys at a time (one per thread), the running maximum and
// sum of the softmax, then each thread's own columns of the weighted values.
#include <cuda_fp8.h>

#include "kv.cuh"

namespace moe {
namespace {

template <int FMT>
__device__ __forceinline__ float element(const uint8_t* row, int i) {
    if (FMT == kKvBf16) return bf16_lo(reinterpret_cast<const uint16_t*>(row)[i]);
    if (FMT == kKvE4m3) {
        const __half_raw hr = __nv_cvt_fp8_to_halfraw(row[i], __NV_E4M3);
        return __half2float(*reinterpret_cast<const __half*>(&hr));
    }
    const int b = row[i / 2];
    return (float)((i & 1) ? (int)((uint32_t)b << 24) >> 28 : (int)((uint32_t)b << 28) >> 28);
}

template <int FMT, int D>
__global__ void __launch_bounds__(128) attn_token_kernel(const AttnArgs a) {
    const int t = blockIdx.x / a.d.H, h = blockIdx.x % a.d.H, tid = threadIdx.x;
    const int hk = h / (a.d.H / a.d.H_kv);
    int lo = 0;  // the sequence of this token
    while (lo + 1 < a.d.B && !(a.q_off[lo] <= t && t < a.q_off[lo + 1] && a.q_off[lo + 1] <= a.d.T))
        ++lo;
    const int b = lo, t0 = a.q_off[b], t1 = a.q_off[b + 1], len = a.kv_len[b];
    if (t < t0 || t >= t1 || t1 > a.d.T || len < 0 || (int64_t)len > (int64_t)a.d.max_pages * a.d.page) {
        if (tid == 0) record_error(a.hdr, kErrBadSeq);
        return;
    }
    const int pos = len - (t1 - t0) + (t - t0);
    const int first = a.d.window ? max(0, pos - a.d.window + 1) : 0;
    const KvRows kr = kv_rows(a.cache, true), vr = kv_rows(a.cache, false);
    __shared__ float q[D], w[128], red[4], vsc[128];
    __shared__ const uint8_t* vrow[128];
    for (int i = tid; i < D; i += 128)
        q[i] = bf16_lo(a.q[t * a.ldq + h * D + i]);
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int j0 = first; j0 <= pos; j0 += 128) {
        __syncthreads();
        const int j = j0 + tid;
        float s = -INFINITY;
        vrow[tid] = nullptr;
        if (j <= pos) {
            int pg = a.pages[(int64_t)b * a.d.max_pages + j / a.d.page];
            if (pg < 0 || pg >= a.d.n_pages) {
                record_error(a.hdr, kErrBadPage);
                pg = 0;
            }
            const int at = j % a.d.page;
            const int64_t si = ((int64_t)pg * a.d.H_kv + hk) * a.d.page + at;
            const uint8_t* kp = kr.row(pg, hk, at);
            float dot = 0.0f;
            for (int i = 0; i < D; ++i) dot += q[i] * element<FMT>(kp, i);
            if (FMT != kKvBf16) dot *= kr.s[si];
            s = dot * a.scale;
            vrow[tid] = vr.row(pg, hk, at);
            vsc[tid] = FMT != kKvBf16 ? vr.s[si] : 1.0f;
        }
        float mx = s;
        for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
        if (tid % 32 == 0) red[tid / 32] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float c = expf(m - mn);  // the first tile: e^-inf = 0
        const float p = expf(s - mn);
        w[tid] = p;
        m = mn;
        __syncthreads();
        o *= c;
        l *= c;
        for (int k = 0; k < 128 && vrow[k]; ++k) {
            l += w[k];
            if (tid < D) o += w[k] * vsc[k] * element<FMT>(vrow[k], tid);
        }
    }
    const int64_t row = (int64_t)t * a.d.H + h;
    if (tid < D) a.out[row * D + tid] = float_to_bf16_bits(l > 0.0f ? o / l : 0.0f);
    if (tid == 0 && a.lse) a.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)a.d.T * (unsigned)a.d.H;
    const bool wide = a.d.D == 128;
    switch (a.d.format) {
        case kKvBf16:
            if (wide) attn_token_kernel<kKvBf16, 128><<<grid, 128, 0, st>>>(a);
            else attn_token_kernel<kKvBf16, 64><<<grid, 128, 0, st>>>(a);
            break;
        case kKvE4m3:
            if (wide) attn_token_kernel<kKvE4m3, 128><<<grid, 128, 0, st>>>(a);
            else attn_token_kernel<kKvE4m3, 64><<<grid, 128, 0, st>>>(a);
            break;
        case kKvInt4:
            if (wide) attn_token_kernel<kKvInt4, 128><<<grid, 128, 0, st>>>(a);
            else attn_token_kernel<kKvInt4, 64><<<grid, 128, 0, st>>>(a);
            break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace moe
