// Attention of new tokens over the paged cache: workspace layout and the
// choice of kernel.
#include "attn.cuh"

namespace moe {
namespace {

// Sequences of at most this many rows (new tokens x query heads per key/value
// head) run on the warp-level kernel, longer ones on the tcgen05 kernel: that one's
// tiles have 128 rows, full or not, the other reads keys from L2 again for every 16.  Measured,
// E4M3, 16 sequences of up to 6.8 thousand keys: with 16 to 48 rows each 73 us against
// 95 us, with up to 128 rows 120 us against 97 us.
constexpr int64_t kFewRows = 64;

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
    if (most * G <= kFewRows) return {true, false, most * G <= 8};
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
        e = launch_attn_tiles(a, k.rows ? kFewRows : 0, most, reinterpret_cast<float*>(ws + at),
                              reinterpret_cast<unsigned*>(ws + kCountersAt + counters_bytes()), st);
        at += align256(attn_tiles_part_bytes(a.d));
    }
    if (k.rows && e == cudaSuccess)
        e = launch_attn_rows(a, 0, k.tiles ? kFewRows : most, k.eight, k.tiles, reinterpret_cast<float*>(ws + at),
                             reinterpret_cast<unsigned*>(ws + kCountersAt), st);
    return e;
}

}  // namespace moe
