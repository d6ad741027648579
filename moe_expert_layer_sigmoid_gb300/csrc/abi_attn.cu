// extern "C" entry points of the paged key/value cache and its attention:
// argument validation on the host, then one launcher each on the caller's
// stream; nothing here allocates or synchronises.
#include <cmath>

#include "attn.cuh"

using namespace moe;

namespace moe {

moe_status_t check_kv_dims(const moe_kv_dims_t* d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->T < 0 || d->B < 0 || d->H <= 0 || d->H_kv <= 0 || d->D <= 0 || d->page <= 0 ||
        d->n_pages <= 0 || d->max_pages <= 0 || d->max_new < 0 || d->window < 0 || d->flags != 0)
        return MOE_ERR_INVALID_ARG;
    if (d->H % d->H_kv) return MOE_ERR_INVALID_ARG;
    if (d->D != 64 && d->D != 128) return MOE_ERR_UNSUPPORTED;
    if (d->page < 16 || d->page > 256 || (d->page & (d->page - 1))) return MOE_ERR_UNSUPPORTED;
    if (d->format < MOE_KV_BF16 || d->format > MOE_KV_INT4) return MOE_ERR_UNSUPPORTED;
    if (d->H / d->H_kv > 128 || d->B > 8192) return MOE_ERR_UNSUPPORTED;
    const int64_t lim = (int64_t)1 << 31;
    if ((int64_t)d->n_pages * d->page >= lim || (int64_t)d->max_pages * d->page >= lim ||
        (int64_t)d->T * d->H >= lim)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool kv_ok(const moe_kv_t* c, const moe_kv_dims_t& d) {
    if (!c || !act_ok(c->k) || !act_ok(c->v)) return false;
    for (const int64_t s : {c->page_stride, c->head_stride, c->slot_stride})
        if (s <= 0 || s % 16 || s >= (int64_t)1 << 40) return false;
    if (d.format == MOE_KV_BF16) return true;
    return act_ok(c->ks) && act_ok(c->vs);
}

// Rows of `width` elements, ld elements apart, read with 16-byte loads.
bool rows_ok(const void* p, int64_t ld, int32_t T, int64_t width) {
    return act_ok(p) && ld % 8 == 0 && (T <= 1 || (ld >= width && ld < (int64_t)1 << 31));
}

moe_status_t check_ws(const void* ws, size_t ws_bytes, size_t need) {
    return !ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 256 ? MOE_ERR_WORKSPACE
                                                                           : MOE_OK;
}

}  // namespace moe

extern "C" {

size_t moe_attn_workspace_bytes(const moe_kv_dims_t* dims) {
    if (check_kv_dims(dims) != MOE_OK) return 0;
    return attn_workspace_bytes(*dims);
}

moe_status_t moe_kv_write(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                          const int32_t* slots, const moe_kv_dims_t* dims, const moe_kv_t* cache,
                          void* ws, size_t ws_bytes, void* stream) {
    moe_status_t st = check_kv_dims(dims);
    if (st != MOE_OK) return st;
    if ((st = check_ws(ws, ws_bytes, sizeof(WsHeader))) != MOE_OK) return st;
    if (dims->T == 0) return MOE_OK;
    const int64_t width = (int64_t)dims->H_kv * dims->D;
    if (!rows_ok(k, ldk, dims->T, width) || !rows_ok(v, ldv, dims->T, width) || !slots ||
        !kv_ok(cache, *dims))
        return MOE_ERR_INVALID_ARG;
    return map_err(launch_kv_write(k, ldk, v, ldv, slots, *dims, *cache, static_cast<WsHeader*>(ws),
                                   static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_kv_read(const int32_t* slots, const moe_kv_dims_t* dims, const moe_kv_t* cache,
                         uint16_t* k, uint16_t* v, void* ws, size_t ws_bytes, void* stream) {
    moe_status_t st = check_kv_dims(dims);
    if (st != MOE_OK) return st;
    if ((st = check_ws(ws, ws_bytes, sizeof(WsHeader))) != MOE_OK) return st;
    if (dims->T == 0) return MOE_OK;
    if (!slots || !act_ok(k) || !act_ok(v) || !kv_ok(cache, *dims)) return MOE_ERR_INVALID_ARG;
    return map_err(launch_kv_read(slots, *dims, *cache, k, v, static_cast<WsHeader*>(ws),
                                  static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_attn_paged(const uint16_t* q, int64_t ldq, const int32_t* q_off,
                            const int32_t* kv_len, const int32_t* pages,
                            const moe_kv_dims_t* dims, const moe_kv_t* cache, float scale,
                            uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    moe_status_t st = check_kv_dims(dims);
    if (st != MOE_OK) return st;
    if ((st = check_ws(ws, ws_bytes, moe_attn_workspace_bytes(dims))) != MOE_OK) return st;
    if (dims->T == 0) return MOE_OK;
    if (dims->B == 0 || !rows_ok(q, ldq, dims->T, (int64_t)dims->H * dims->D) || !q_off ||
        !kv_len || !pages || !kv_ok(cache, *dims) || !std::isfinite(scale * kLog2e) || !act_ok(out) ||
        reinterpret_cast<uintptr_t>(lse) % 4)
        return MOE_ERR_INVALID_ARG;
    const AttnArgs a{q,      ldq,   q_off, kv_len, pages, *dims,
                     *cache, scale, out,   lse,    static_cast<WsHeader*>(ws)};
    return map_err(launch_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
