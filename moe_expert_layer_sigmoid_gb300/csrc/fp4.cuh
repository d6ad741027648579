// Microscaled 4-bit floats: layout of the block scales, launchers.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFp4TileRows = 128;   // a scale tile: 128 rows of 4 blocks, 512 bytes
constexpr int kFp4MaxK = 65536;

inline size_t fp4_scale_bytes(int64_t rows, int64_t K) {
    return (size_t)((rows + kFp4TileRows - 1) / kFp4TileRows) * (size_t)(K / 64) * 512;
}

// Byte of the scale of row r and block j.
__host__ __device__ inline int64_t fp4_scale_at(int64_t r, int j, int K) {
    return ((r / kFp4TileRows) * (K / 64) + j / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4;
}

// Where moe_linear_fp4 keeps the quantised activations, behind the header.
struct Fp4Ws {
    size_t q, b, s, bytes;
};
inline Fp4Ws fp4_ws(int64_t T, int64_t K) {
    Fp4Ws w{};
    size_t off = sizeof(WsHeader);
    w.q = off;
    off += align256((size_t)(T * (K / 2)));
    w.b = off;
    off += align256(fp4_scale_bytes(T, K));
    w.s = off;
    off += align256(sizeof(float) * (size_t)T);
    w.bytes = off;
    return w;
}

struct Fp4Rows {
    uint8_t *q, *b;
    float* s;
};

// ld: elements from row to row of the source.
cudaError_t launch_quant_fp4(const void* src, bool bf16, int64_t ld, int64_t rows, int64_t K, Fp4Rows out,
                             cudaStream_t st);
cudaError_t launch_unpack_fp4(moe_fp4_t w, int64_t rows, int64_t K, uint16_t* out, cudaStream_t st);
// The projection of few tokens, quantisation included.
bool gemv_fp4_takes(int T, int N, int K);
cudaError_t launch_gemv_fp4(const uint16_t* x, int64_t ldx, moe_fp4_t w, int T, int N, int K, uint16_t* out,
                            cudaStream_t st);
cudaError_t launch_linear_fp4(moe_fp4_t x, moe_fp4_t w, int T, int N, int K, uint16_t* out, void* ws,
                              cudaStream_t st);
cudaError_t launch_pair_fp4(moe_fp4_t x, moe_fp4_t w, int T, int N, int K, uint16_t* out, void* ws, cudaStream_t st);

}  // namespace moe
