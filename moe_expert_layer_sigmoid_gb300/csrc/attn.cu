// Attention of new tokens over the paged cache: workspace layout and the
// choice of kernel.
#include "attn.cuh"

namespace moe {
namespace {

// Sequences of at most this many rows (new tokens x query heads per key/value
// head) run on the warp-level kernel, longer ones on the tcgen05 kernel: that one's
// tiles have 128 rows, full or not, the other reads the keys from L2 and turns their
// codes into operands again for every 16.  Measured, whole calls of D = 128 and up to 8
// thousand keys, 8 key/value heads, in us (warp-level / tcgen05):
//                        32 rows       48 rows       64 rows       80 rows
//   16 sequences, bf16   64.1 / 62.3   77.7 / 62.8  114.4 / 62.8  131.2 / 62.8
//                 E4M3   53.6 / 84.5   80.1 / 84.2  100.3 / 84.8
//                 int4                 74.3 / 77.4   94.4 / 78.0  113.6 / 77.5
//   8 sequences, bf16                  50.9 / 48.7
//                E4M3                                60.9 / 57.0
//   4 sequences, bf16                  40.3 / 43.7   45.5 / 44.3
//                E4M3                                47.3 / 48.4
//   2 sequences, bf16    29.1 / 38.5   31.1 / 38.7
//                E4M3                                35.2 / 44.0
// (D = 64, 16 sequences: bf16 41.3 / 47.6 at 32, 52.4 / 47.9 at 48; E4M3 50.1 / 59.1 at 48,
// 63.7 / 60.0 at 64.)  A call of few sequences and heads leaves SMs to the extra units.
// bf16 rows of 32 stay on the warp-level kernel for D = 64, where it gains 13%, and lose 3%
// with D = 128.
int64_t few_rows(const moe_kv_dims_t& d) {
    if (4 * (int64_t)d.B * d.H_kv <= sm_count()) return 64;
    return d.format == kKvBf16 ? 32 : 48;
}

// Which kernels a call needs, from what the host knows of its sequences.  A
// sequence's rows are only known on the device, so with both launched each
// kernel takes its own; a single one takes all.
struct Kernels {
    bool rows, tiles;
    bool eight;  // units of eight rows on the warp-level kernel
};
Kernels kernels_for(const moe_kv_dims_t& d) {
    const int64_t G = d.H / d.H_kv;
    int64_t most = d.max_new > 0 ? std::min(d.max_new, d.T) : d.T;
    if (most * G <= few_rows(d)) return {true, false, most * G <= 8};
    if (d.B == 1) return {false, true, false};
    return {true, true, G <= 8};
}

// Workspace: the header, the arrival counters of the joins (at a place that no
// size moves, zero between calls; one set for each kernel), the partial results.
constexpr size_t kCountersAt = sizeof(WsHeader);
size_t counters_bytes() { return align256(sizeof(unsigned) * 4 * (size_t)sm_count()); }
size_t part_at() { return kCountersAt + 2 * counters_bytes(); }

}  // namespace

size_t attn_workspace_bytes(const moe_kv_dims_t& d) {
    const Kernels k = kernels_for(d);
    return part_at() + (k.rows ? align256(attn_rows_part_bytes(d)) : 0) +
           (k.tiles ? align256(attn_tiles_part_bytes(d)) : 0);
}

bool make_kv_map(CUtensorMap* m, const void* base, const AttnArgs& a, int box_bytes, int box_rows) {
    const bool wide = a.d.format == kKvBf16;
    const int size = wide ? 2 : 1;
    const cuuint64_t dims[4] = {(cuuint64_t)kv_row_bytes(a.d.format, a.d.D) / size, (cuuint64_t)a.d.page,
                                (cuuint64_t)a.d.H_kv, (cuuint64_t)a.d.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)a.cache.slot_stride, (cuuint64_t)a.cache.head_stride,
                                   (cuuint64_t)a.cache.page_stride};
    const cuuint32_t box[4] = {(cuuint32_t)(box_bytes / size), (cuuint32_t)box_rows, 1, 1};
    return make_map_nd(m, wide ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 4,
                       dims, strides, box,
                       box_bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                       : box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                         : CU_TENSOR_MAP_SWIZZLE_32B);
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st) {
    const Kernels k = kernels_for(a.d);
    uint8_t* ws = reinterpret_cast<uint8_t*>(a.hdr);
    const int64_t most = (int64_t)1 << 62;
    size_t at = part_at();
    cudaError_t e = cudaSuccess;
    if (k.tiles) {
        e = launch_attn_tiles(a, k.rows ? few_rows(a.d) : 0, most, reinterpret_cast<float*>(ws + at),
                              reinterpret_cast<unsigned*>(ws + kCountersAt + counters_bytes()), st);
        at += align256(attn_tiles_part_bytes(a.d));
    }
    if (k.rows && e == cudaSuccess)
        e = launch_attn_rows(a, 0, k.tiles ? few_rows(a.d) : most, k.eight, k.tiles, reinterpret_cast<float*>(ws + at),
                             reinterpret_cast<unsigned*>(ws + kCountersAt), st);
    return e;
}

}  // namespace moe
