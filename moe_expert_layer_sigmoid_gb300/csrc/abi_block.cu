// extern "C" entry points of what stands around the attention and the experts:
// page planning, rotary positions, the norms between blocks, 4-bit floats.
// Argument validation on the host, then the launches on the caller's stream; nothing here allocates or
// synchronises.
#include <cmath>

#include "block_norm.cuh"
#include "fp4.cuh"
#include "rope.cuh"

namespace moe {
cudaError_t launch_kv_plan(const int32_t* new_len, const moe_kv_dims_t& d, const moe_kv_pages_t& st,
                           int32_t* q_off, int32_t* pos, int32_t* slots, WsHeader* hdr, cudaStream_t stream);
}

using namespace moe;

namespace {

bool aligned4(const void* p) { return p && reinterpret_cast<uintptr_t>(p) % 4 == 0; }
bool act_ok_or_null(const void* p) { return !p || act_ok(p); }

moe_status_t check_rope_config(const moe_rope_config_t* g) {
    if (!g || !std::isfinite(g->base) || !(g->base > 1.0) ||
        !std::isfinite((float)g->magnitude) || !((float)g->magnitude > 0.0f) || g->rot <= 0 || g->scaling < MOE_ROPE_NONE || g->scaling > MOE_ROPE_BAND)
        return MOE_ERR_INVALID_ARG;
    if (g->scaling != MOE_ROPE_NONE && !(std::isfinite(g->factor) && g->factor >= 1.0)) return MOE_ERR_INVALID_ARG;
    if (g->scaling >= MOE_ROPE_RAMP &&
        !(std::isfinite(g->orig_len) && g->orig_len > 0.0 && std::isfinite(g->hi) && g->lo > 0.0 && g->hi > g->lo))
        return MOE_ERR_INVALID_ARG;
    return g->rot % 16 || g->rot > 256 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t check_rope(const moe_rope_t* r, int32_t D) {
    if (!r || !act_ok(r->table) || !act_ok_or_null(r->q_norm) || !act_ok_or_null(r->k_norm) || r->n_pos < 0 ||
        r->rot <= 0 || r->rot > D || (r->flags & ~(MOE_ROPE_PAIRS | MOE_ROPE_INVERSE)) ||
        !(std::isfinite(r->eps) && r->eps >= 0.0f))
        return MOE_ERR_INVALID_ARG;
    return r->rot % 16 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t check_fp4(int64_t rows, int64_t K) {
    if (rows < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (K % 64 || K > kFp4MaxK || rows >= ((int64_t)1 << 31) - 128) return MOE_ERR_UNSUPPORTED;
    return rows * K >= (int64_t)1 << 40 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t check_linear(int32_t T, int32_t N, int32_t K) {
    if (T < 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_fp4(N, K);
    if (st != MOE_OK) return st;
    return N % 8 || N >= 1 << 24 || T >= 1 << 24 || (int64_t)T * N >= (int64_t)1 << 40 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t quant(const void* src, bool bf16, int64_t rows, int64_t K, uint8_t* q, uint8_t* b, float* s,
                   void* stream) {
    const moe_status_t st = check_fp4(rows, K);
    if (st != MOE_OK || rows == 0) return st;
    if (!act_ok(src) || !act_ok(q) || !act_ok(b) || !aligned4(s)) return MOE_ERR_INVALID_ARG;
    return map_err(launch_quant_fp4(src, bf16, K, rows, K, Fp4Rows{q, b, s}, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

moe_status_t moe_kv_plan(const int32_t* new_len, const moe_kv_dims_t* dims, const moe_kv_pages_t* state,
                         int32_t* q_off, int32_t* pos, int32_t* slots, void* ws, size_t ws_bytes,
                         void* stream) {
    moe_status_t st = check_kv_dims(dims);
    if (st != MOE_OK) return st;
    if ((st = check_ws(ws, ws_bytes, sizeof(WsHeader))) != MOE_OK) return st;
    if (!state || !aligned4(state->free_pages) || !aligned4(state->n_free) || !aligned4(q_off))
        return MOE_ERR_INVALID_ARG;
    if (dims->T > 0 && (!aligned4(pos) || !aligned4(slots))) return MOE_ERR_INVALID_ARG;
    if (dims->B > 0 && (!aligned4(new_len) || !aligned4(state->kv_len) || !aligned4(state->first) ||
                        !aligned4(state->pages)))
        return MOE_ERR_INVALID_ARG;
    return map_err(launch_kv_plan(new_len, *dims, *state, q_off, pos, slots, static_cast<WsHeader*>(ws),
                                  static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_rope_table(const moe_rope_config_t* config, int32_t pos0, int32_t n_pos, float* table,
                            void* stream) {
    const moe_status_t st = check_rope_config(config);
    if (st != MOE_OK) return st;
    if (pos0 < 0 || n_pos < 0 || (int64_t)pos0 + n_pos > (int64_t)1 << 31) return MOE_ERR_INVALID_ARG;
    if ((int64_t)n_pos * config->rot >= (int64_t)1 << 40) return MOE_ERR_UNSUPPORTED;
    if (n_pos == 0) return MOE_OK;
    if (!act_ok(table)) return MOE_ERR_INVALID_ARG;
    return map_err(launch_rope_table(*config, pos0, n_pos, table, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_rope_rows(const uint16_t* x, int64_t ldx, const int32_t* pos, int32_t T, int32_t H,
                           int32_t D, const moe_rope_t* rope, uint16_t* out, int64_t ldo, void* ws,
                           size_t ws_bytes, void* stream) {
    if (T < 0 || H <= 0 || D <= 0) return MOE_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || (int64_t)T * H >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
    moe_status_t st = check_rope(rope, D);
    if (st != MOE_OK) return st;
    if ((st = check_ws(ws, ws_bytes, sizeof(WsHeader))) != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const int64_t width = (int64_t)H * D;
    if (!rows_ok(x, ldx, T, width) || !rows_ok(out, ldo, T, width) || !aligned4(pos) ||
        (x == out && T > 1 && ldx != ldo))
        return MOE_ERR_INVALID_ARG;
    return map_err(launch_rope_rows(x, ldx, pos, T, H, D, *rope, out, ldo, static_cast<WsHeader*>(ws),
                                    static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_rope_kv_write(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                               const uint16_t* v, int64_t ldv, const int32_t* pos,
                               const int32_t* slots, const moe_rope_t* rope,
                               const moe_kv_dims_t* dims, const moe_kv_t* cache, uint16_t* q_out,
                               int64_t ldo, void* ws, size_t ws_bytes, void* stream) {
    moe_status_t st = check_kv_dims(dims);
    if (st != MOE_OK) return st;
    if ((st = check_rope(rope, dims->D)) != MOE_OK) return st;
    if ((st = check_ws(ws, ws_bytes, sizeof(WsHeader))) != MOE_OK) return st;
    if (dims->T == 0) return MOE_OK;
    const int64_t wide = (int64_t)dims->H * dims->D, narrow = (int64_t)dims->H_kv * dims->D;
    if (!rows_ok(q, ldq, dims->T, wide) || !rows_ok(k, ldk, dims->T, narrow) || !rows_ok(v, ldv, dims->T, narrow) ||
        !rows_ok(q_out, ldo, dims->T, wide) || !aligned4(pos) || !aligned4(slots) || !kv_ok(cache, *dims) ||
        (q == q_out && dims->T > 1 && ldq != ldo))
        return MOE_ERR_INVALID_ARG;
    const RopeWriteArgs a{q, k, v, ldq, ldk, ldv, ldo, pos, slots, *rope, *dims, *cache, q_out,
                          static_cast<WsHeader*>(ws)};
    return map_err(launch_rope_kv_write(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_block_norm(const uint16_t* y, const void* residual, const void* gate,
                            const float* w_post, const float* w_pre, const moe_norm_dims_t* dims,
                            void* residual_out, uint16_t* x, void* stream) {
    if (!dims || dims->T < 0 || dims->d <= 0 || dims->gate < MOE_GATE_NONE || dims->gate > MOE_GATE_FULL ||
        (dims->flags & ~(MOE_NORM_SIGMOID | MOE_NORM_RESIDUAL_F32)) ||
        !(std::isfinite(dims->eps) && dims->eps >= 0.0f) || !std::isfinite(dims->scale))
        return MOE_ERR_INVALID_ARG;
    if (dims->d % 8 || dims->d > 32768) return MOE_ERR_UNSUPPORTED;
    if (dims->T == 0) return MOE_OK;
    if ((gate != nullptr) != (dims->gate != MOE_GATE_NONE) || (w_pre != nullptr) != (x != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (!y && (gate || w_post || !w_pre)) return MOE_ERR_INVALID_ARG;
    if (!act_ok_or_null(y) || !act_ok(residual) || !act_ok_or_null(w_post) || !act_ok_or_null(w_pre) ||
        !act_ok_or_null(x) || (y && !act_ok(residual_out)) ||
        (gate && !(dims->gate == MOE_GATE_TOKEN ? aligned4(gate) : act_ok(gate))))
        return MOE_ERR_INVALID_ARG;
    return map_err(launch_block_norm(y, residual, gate, w_post, w_pre, *dims, residual_out, x,
                                     static_cast<cudaStream_t>(stream)));
}

size_t moe_fp4_scale_bytes(int64_t rows, int64_t K) {
    return check_fp4(rows, K) == MOE_OK ? fp4_scale_bytes(rows, K) : 0;
}

moe_status_t moe_pack_fp4(const float* w, int64_t rows, int64_t K, uint8_t* q, uint8_t* b, float* s,
                          void* stream) {
    return quant(w, false, rows, K, q, b, s, stream);
}

moe_status_t moe_quant_rows_fp4(const uint16_t* x, int64_t rows, int64_t K, uint8_t* q, uint8_t* b,
                                float* s, void* stream) {
    return quant(x, true, rows, K, q, b, s, stream);
}

moe_status_t moe_unpack_fp4(moe_fp4_t w, int64_t rows, int64_t K, uint16_t* out, void* stream) {
    const moe_status_t st = check_fp4(rows, K);
    if (st != MOE_OK || rows == 0) return st;
    if (!act_ok(w.q) || !act_ok(w.b) || !aligned4(w.s) || !act_ok(out)) return MOE_ERR_INVALID_ARG;
    return map_err(launch_unpack_fp4(w, rows, K, out, static_cast<cudaStream_t>(stream)));
}

size_t moe_linear_fp4_workspace_bytes(int32_t T, int32_t N, int32_t K) {
    return check_linear(T, N, K) == MOE_OK ? fp4_ws(T, K).bytes : 0;
}

moe_status_t moe_linear_fp4(const uint16_t* x, int64_t ldx, int32_t T, int32_t N, int32_t K,
                            moe_fp4_t w, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
    moe_status_t st = check_linear(T, N, K);
    if (st != MOE_OK) return st;
    const Fp4Ws at = fp4_ws(T, K);
    if ((st = check_ws(ws, ws_bytes, at.bytes)) != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!rows_ok(x, ldx, T, K) || !act_ok(w.q) || !act_ok(w.b) || !aligned4(w.s) || !act_ok(out))
        return MOE_ERR_INVALID_ARG;
    if (gemv_fp4_takes(T, N, K))
        return map_err(launch_gemv_fp4(x, ldx, w, T, N, K, out, static_cast<cudaStream_t>(stream)));
    uint8_t* base = static_cast<uint8_t*>(ws);
    const Fp4Rows xq{base + at.q, base + at.b, reinterpret_cast<float*>(base + at.s)};
    const cudaStream_t stm = static_cast<cudaStream_t>(stream);
    const cudaError_t err = launch_quant_fp4(x, true, ldx, T, K, xq, stm);
    if (err != cudaSuccess) return map_err(err);
    return map_err(launch_linear_fp4(moe_fp4_t{xq.q, xq.b, xq.s}, w, T, N, K, out, ws, stm));
}

}  // extern "C"
