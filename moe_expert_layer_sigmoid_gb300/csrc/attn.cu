// Attention of new tokens over the paged cache: workspace layout and the
// choice of kernel.
#include "attn.cuh"

namespace moe {
namespace {

// Workspace: the header, the arrival counters of the joins (at a place that no
// size moves, zero between calls), the partial results.
constexpr size_t kCountersAt = sizeof(WsHeader);
size_t part_at() { return kCountersAt + align256(sizeof(unsigned) * 2 * (size_t)sm_count()); }

}  // namespace

size_t attn_workspace_bytes(const moe_kv_dims_t& d) { return part_at() + align256(attn_rows_part_bytes(d)); }

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
    uint8_t* ws = reinterpret_cast<uint8_t*>(a.hdr);
    return launch_attn_rows(a, 0, (int64_t)1 << 62, reinterpret_cast<float*>(ws + part_at()),
                            reinterpret_cast<unsigned*>(ws + kCountersAt), st);
}

}  // namespace moe
