// Block-scaled products of 4-bit floats on the tensor cores: what the kernels of moe_linear_fp4 share.
#pragma once

#include "fp4.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace moe {

constexpr int kStageK = 256;           // elements of K per stage
constexpr int kRowBytes = kStageK / 2;  // codes of a row per stage
constexpr int kAtom = 512;             // scales of 128 rows and 64 elements

// One operand: rows of codes and their scales.
struct Side {
    CUtensorMap map;
    const uint8_t* b;
    const float* s;
    int rows, tiles;  // tiles of 128 (M) or NT rows
};

// Instruction descriptor, kind::mxf4nvf4: E2M1 A and B, unsigned E4M3 scales, fp32 D, both K-major.
__device__ __forceinline__ uint32_t idesc_fp4(int M, int N) {
    return (1u << 7)                      // A format: E2M1
           | (1u << 10)                   // B format: E2M1
           | ((uint32_t)(N >> 3) << 17)   // N / 8
           | ((uint32_t)(M >> 7) << 27);  // M / 128
}

// D (TMEM) (+)= A (shared memory) x B (shared memory) with scales in TMEM, K = 64; CTAS 2: by a pair of CTAs, each with
// half of the rows of either operand.
template <int CTAS>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// Scales in shared memory: 32 rows of 16 bytes.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 |
           (uint64_t)(128 >> 4) << 32 |  // 8 rows of 16 bytes to the next 8
           (uint64_t)1 << 46;            // version; no swizzle
}
// They go to four TMEM columns, in each quarter of the lanes; CTAS 2: in each CTA of a pair from its own shared memory.
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same without handing anything over: before a cluster's barriers are used, and before its CTAs leave.  (With release it
// waits for the outputs' stores.)
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// The address of one's own shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// One step of a transposition among lanes: with the lane whose number differs in bit BIT, a's half from the lane with
// the bit clear stays or goes to the other's b.
template <int BIT>
__device__ __forceinline__ void trade(uint4& a, uint4& b, int lane) {
    const bool up = lane & BIT;
    const uint4 send = up ? a : b, keep = up ? b : a;
    uint4 got;
    got.x = __shfl_xor_sync(0xFFFFFFFFu, send.x, BIT);
    got.y = __shfl_xor_sync(0xFFFFFFFFu, send.y, BIT);
    got.z = __shfl_xor_sync(0xFFFFFFFFu, send.z, BIT);
    got.w = __shfl_xor_sync(0xFFFFFFFFu, send.w, BIT);
    a = up ? got : keep;
    b = up ? keep : got;
}

// A lane's 32 packed outputs of its row, the warp's 32 rows below each other: four lanes trade pieces of 16 bytes, so that a store
// writes whole sectors (a lane's own 16 bytes at a time cost twice the writes in L2).  `to`: where piece
// lane % 4 of row lane / 4 * 4 belongs; from there on `rows` rows and `cols` columns are inside.
__device__ __forceinline__ void store_run(uint4 (&x)[4], uint16_t* to, int64_t ld, int rows, int cols, int lane) {
    trade<1>(x[0], x[1], lane);
    trade<1>(x[2], x[3], lane);
    trade<2>(x[0], x[2], lane);
    trade<2>(x[1], x[3], lane);
    // x[i] is now piece lane % 4 of row lane / 4 * 4 + i
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < rows && cols > 0) *reinterpret_cast<uint4*>(to + i * ld) = x[i];
}

inline bool codes_map(CUtensorMap* m, const uint8_t* q, int64_t rows, int64_t K, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
    return make_map_nd(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

inline bool make_side(Side& s, const moe_fp4_t& v, int rows, int K, int tile) {
    s.b = v.b;
    s.s = v.s;
    s.rows = rows;
    s.tiles = (rows + tile - 1) / tile;
    return codes_map(&s.map, v.q, rows, K, tile);
}

}  // namespace moe
