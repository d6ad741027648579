"""Python binding of libmoe.so, the GB300 routed MoE FFN layer.

Argument marshalling only: every function here checks tensor shapes, dtypes
and devices, passes raw pointers and the current CUDA stream to the C ABI
declared in include/moe.h, and raises MoeError on a non-OK status.  All
arithmetic runs in the library's CUDA kernels; there is no other path.  If
libmoe.so has not been built, importing works but every call raises.

PyTorch supplies device memory and streams.  bf16 / fp16 tensors are passed
as their bit patterns.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_CHECK = 5

MOE_KV_BF16 = 0
MOE_KV_E4M3 = 1
MOE_KV_INT4 = 2

MOE_ROPE_NONE = 0
MOE_ROPE_LINEAR = 1
MOE_ROPE_RAMP = 2
MOE_ROPE_BAND = 3

MOE_ROPE_PAIRS = 0x1
MOE_ROPE_INVERSE = 0x2

MOE_GATE_NONE = 0
MOE_GATE_TOKEN = 1
MOE_GATE_CHANNEL = 2
MOE_GATE_FULL = 3

MOE_NORM_SIGMOID = 0x1
MOE_NORM_RESIDUAL_F32 = 0x2

MOE_FLAG_FORCE_GEMV = 0x1
MOE_FLAG_FORCE_GROUPED = 0x2
MOE_FLAG_NO_SCHED = 0x4
MOE_FLAG_DECODE_MMA = 0x8

# every extern "C" symbol include/moe.h declares
EXPORTS = (
    "moe_status_string", "moe_pack_w4", "moe_workspace_bytes", "moe_router_topk",
    "moe_build_descriptors", "moe_gateup_swiglu_w4a16", "moe_down_w4a16", "moe_combine_shared",
    "moe_layer_workspace_bytes", "moe_layer_forward", "moe_layer_forward_host",
    "moe_check_device_status", "moe_router_topk_noalloc", "moe_pack_w4_bytes",
    "moe_combine_shared_residual", "moe_layer_forward_residual", "moe_import_q4_blocks",
    "moe_down_combine_w4a16", "moe_pack_w8", "moe_quant_rows_fp8",
    "moe_layer_workspace_bytes_w8a8", "moe_layer_forward_w8a8", "moe_gateup_swiglu_w8a8",
    "moe_down_w8a8", "moe_debug_set_waits", "moe_kv_write", "moe_kv_read",
    "moe_attn_workspace_bytes", "moe_attn_paged", "moe_kv_plan", "moe_rope_table", "moe_rope_rows",
    "moe_rope_kv_write", "moe_block_norm", "moe_fp4_scale_bytes", "moe_pack_fp4", "moe_quant_rows_fp4",
    "moe_unpack_fp4", "moe_linear_fp4_workspace_bytes", "moe_linear_fp4",
)


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class Dims(ctypes.Structure):
    """moe_dims_t."""
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("F", ctypes.c_int32), ("F_s", ctypes.c_int32),
                ("group", ctypes.c_int32), ("flags", ctypes.c_uint32)]

    def replace(self, **kw) -> "Dims":
        vals = {f: getattr(self, f) for f, _ in self._fields_}
        vals.update(kw)
        return Dims(**vals)


class W4(ctypes.Structure):
    """moe_w4_t: packed int4 bytes and fp16 scales (device pointers)."""
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p)]


class W8(ctypes.Structure):
    """moe_w8_t: E4M3 codes and fp32 row scales (device pointers)."""
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p)]


class KvDims(ctypes.Structure):
    """moe_kv_dims_t."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "B", "H", "H_kv", "D", "page", "n_pages", "max_pages", "max_new", "window",
                 "format")] + [("flags", ctypes.c_uint32)]

    def replace(self, **kw) -> "KvDims":
        vals = {f: getattr(self, f) for f, _ in self._fields_}
        vals.update(kw)
        return KvDims(**vals)


class Kv(ctypes.Structure):
    """moe_kv_t: a cache pool's codes, row scales (device pointers) and strides in bytes.
    kv_cache makes one and records its shape for the calls' checks."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_void_p),
                ("vs", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64)]
    shape = dev = None


class KvPages(ctypes.Structure):
    """moe_kv_pages_t: the state of a pool's pages (device pointers).  kv_pages makes one and
    records its sizes for the calls' checks."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("kv_len", "first", "pages", "free_pages", "n_free")]
    sizes = dev = None


class RopeConfig(ctypes.Structure):
    """moe_rope_config_t: which angles a rotary table holds."""
    _fields_ = [(n, ctypes.c_double) for n in ("base", "factor", "orig_len", "lo", "hi", "magnitude")] + \
               [("rot", ctypes.c_int32), ("scaling", ctypes.c_int32)]


class Rope(ctypes.Structure):
    """moe_rope_t: how rows are turned (device pointers).  rope makes one and records the width of
    its norms for the calls' checks."""
    _fields_ = [("table", ctypes.c_void_p), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("n_pos", ctypes.c_int32), ("rot", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("eps", ctypes.c_float)]
    D = dev = None


class NormDims(ctypes.Structure):
    """moe_norm_dims_t."""
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("eps", ctypes.c_float), ("scale", ctypes.c_float)]


class Fp4(ctypes.Structure):
    """moe_fp4_t: 4-bit codes, block scales and row scales (device pointers).  fp4 makes one and
    records its shape for the calls' checks."""
    _fields_ = [("q", ctypes.c_void_p), ("b", ctypes.c_void_p), ("s", ctypes.c_void_p)]
    shape = dev = None


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmoe.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(Dims)
    KD, KC, f32 = ctypes.POINTER(KvDims), ctypes.POINTER(Kv), ctypes.c_float
    R = ctypes.POINTER(Rope)
    sigs = {
        "moe_status_string": ([i32], ctypes.c_char_p),
        "moe_pack_w4": ([p, i64, i64, i32, p, p, p], i32),
        "moe_workspace_bytes": ([D], sz),
        "moe_layer_workspace_bytes": ([D], sz),
        "moe_router_topk": ([p, p, p, D, p, p, p, p, sz, p], i32),
        "moe_build_descriptors": ([p, D, p, p, p, p, p, p, sz, p], i32),
        "moe_gateup_swiglu_w4a16": ([p, D, p, p, p, W4, W4, p, p, sz, p], i32),
        "moe_down_w4a16": ([p, D, p, p, W4, W4, p, p, sz, p], i32),
        "moe_down_combine_w4a16": ([p, D, p, p, p, p, W4, W4, p, p, p, sz, p], i32),
        "moe_pack_w8": ([p, i64, i64, p, p, p], i32),
        "moe_quant_rows_fp8": ([p, i64, i64, p, p, p], i32),
        "moe_layer_workspace_bytes_w8a8": ([D], sz),
        "moe_layer_forward_w8a8": ([p, p, p, D, W8, W8, W8, W8, p, p, sz, p], i32),
        "moe_gateup_swiglu_w8a8": ([p, D, p, W8, W8, p, p, sz, p], i32),
        "moe_down_w8a8": ([p, D, W8, W8, p, p, sz, p], i32),
        "moe_debug_set_waits": ([p, sz, ctypes.c_uint64, i32, p], i32),
        "moe_pack_w4_bytes": ([i64, i64, i32, ctypes.POINTER(sz)], sz),
        "moe_import_q4_blocks": ([p, i64, i64, i32, p, p, p, p], i32),
        "moe_combine_shared": ([p, p, p, D, p, p], i32),
        "moe_combine_shared_residual": ([p, p, p, D, p, p, p], i32),
        "moe_layer_forward_residual": ([p, p, p, D, W4, W4, W4, W4, p, p, p, sz, p], i32),
        "moe_layer_forward": ([p, p, p, D, W4, W4, W4, W4, p, p, sz, p], i32),
        "moe_layer_forward_host": ([p, p, p, D, W4, W4, W4, W4, p, p, sz, p], i32),
        "moe_check_device_status": ([p, sz, p], i32),
        "moe_router_topk_noalloc": ([p, p, p, D, p, p, p, p], i32),
        "moe_kv_write": ([p, i64, p, i64, p, KD, KC, p, sz, p], i32),
        "moe_kv_read": ([p, KD, KC, p, p, p, sz, p], i32),
        "moe_attn_workspace_bytes": ([KD], sz),
        "moe_attn_paged": ([p, i64, p, p, p, KD, KC, f32, p, p, p, sz, p], i32),
        "moe_kv_plan": ([p, KD, ctypes.POINTER(KvPages), p, p, p, p, sz, p], i32),
        "moe_rope_table": ([ctypes.POINTER(RopeConfig), i32, i32, p, p], i32),
        "moe_rope_rows": ([p, i64, p, i32, i32, i32, R, p, i64, p, sz, p], i32),
        "moe_rope_kv_write": ([p, i64, p, i64, p, i64, p, p, R, KD, KC, p, i64, p, sz, p], i32),
        "moe_block_norm": ([p, p, p, p, p, ctypes.POINTER(NormDims), p, p, p], i32),
        "moe_fp4_scale_bytes": ([i64, i64], sz),
        "moe_pack_fp4": ([p, i64, i64, p, p, p, p], i32),
        "moe_quant_rows_fp4": ([p, i64, i64, p, p, p, p], i32),
        "moe_unpack_fp4": ([Fp4, i64, i64, p, p], i32),
        "moe_linear_fp4_workspace_bytes": ([i32, i32, i32], sz),
        "moe_linear_fp4": ([p, i64, i32, i32, i32, Fp4, p, p, sz, p], i32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t):
    if t is None:
        return None
    return t.data_ptr()


# 16-bit float patterns may travel as int16 or as the matching torch dtype
_BITS16 = (torch.int16, torch.bfloat16, torch.float16)
_ALIASES = {torch.int16: _BITS16}


def _dev(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype and t.dtype not in _ALIASES.get(dtype, (dtype,)):
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    """The raw stream: the current device's current one, or that of a torch stream.  (Read without
    building a torch.cuda.Stream, which takes 3 us on the GB300's host cores, against 0.3 us.)"""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _made_for(stream):
    """Outputs that a call makes itself belong to its stream, as its kernel does: their memory is free there, and what fills
    them comes first."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def w4(q: torch.Tensor, s: torch.Tensor) -> W4:
    return W4(_dev(q, torch.uint8, "q"), _dev(s, torch.int16, "s"))


def w8(q: torch.Tensor, s: torch.Tensor) -> W8:
    return W8(_dev(q, torch.uint8, "q"), _dev(s, torch.float32, "s"))


# ------------------------------------------------------------------ entry points

def moe_pack_w4(w: torch.Tensor, group: int, q: torch.Tensor | None = None,
                s: torch.Tensor | None = None, stream=None):
    """fp32 [rows][K] -> (q uint8 [rows][K/2], s fp16 bits as int16 [rows][K/group])."""
    rows, K = w.shape
    with _made_for(stream):
        if q is None:
            q = torch.empty((rows, K // 2), dtype=torch.uint8, device=w.device)
        if s is None:
            s = torch.empty((rows, K // group), dtype=torch.int16, device=w.device)
    _check(lib().moe_pack_w4(_dev(w, torch.float32, "w"), rows, K, group,
                             _dev(q, torch.uint8, "q"), _dev(s, torch.int16, "s"),
                             _stream(stream)), "moe_pack_w4")
    return q, s


def moe_pack_w8(w: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                stream=None):
    """fp32 [rows][K] -> (E4M3 codes uint8 [rows][K], fp32 row scales [rows])."""
    rows, K = w.shape
    with _made_for(stream):
        if q is None:
            q = torch.empty((rows, K), dtype=torch.uint8, device=w.device)
        if s is None:
            s = torch.empty(rows, dtype=torch.float32, device=w.device)
    _check(lib().moe_pack_w8(_dev(w, torch.float32, "w"), rows, K, _dev(q, torch.uint8, "q"),
                             _dev(s, torch.float32, "s"), _stream(stream)), "moe_pack_w8")
    return q, s


def moe_quant_rows_fp8(x: torch.Tensor, q: torch.Tensor | None = None,
                       a: torch.Tensor | None = None, stream=None):
    """bf16 rows (int16 bits) [rows][K] -> (E4M3 codes uint8 [rows][K], fp32 scales [rows])."""
    rows, K = x.shape
    if q is None or a is None:
        with _made_for(stream):
            if q is None:
                q = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
            if a is None:
                a = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().moe_quant_rows_fp8(_dev(x, torch.int16, "x"), rows, K, _dev(q, torch.uint8, "q"),
                                    _dev(a, torch.float32, "a"), _stream(stream)),
           "moe_quant_rows_fp8")
    return q, a


def moe_layer_workspace_bytes_w8a8(dims: Dims) -> int:
    return lib().moe_layer_workspace_bytes_w8a8(ctypes.byref(dims))


def moe_layer_forward_w8a8(x, W_r, bias, dims: Dims, Wgu: W8, Wd: W8, Wgu_s: W8, Wd_s: W8, out,
                           ws, stream=None):
    _check(lib().moe_layer_forward_w8a8(
        _dev(x, torch.int16, "x"), _dev(W_r, torch.float32, "W_r"), _dev(bias, torch.float32, "bias"),
        ctypes.byref(dims), Wgu, Wd, Wgu_s, Wd_s, _dev(out, torch.int16, "out"), _ptr(ws),
        ws.numel(), _stream(stream)), "moe_layer_forward_w8a8")


def moe_gateup_swiglu_w8a8(x, dims: Dims, perm, Wgu: W8, Wgu_s: W8, H, ws, stream=None):
    _check(lib().moe_gateup_swiglu_w8a8(
        _dev(x, torch.int16, "x"), ctypes.byref(dims), _dev(perm, torch.int32, "perm"), Wgu, Wgu_s,
        _dev(H, torch.int16, "H"), _ptr(ws), ws.numel(), _stream(stream)), "moe_gateup_swiglu_w8a8")


def moe_down_w8a8(H, dims: Dims, Wd: W8, Wd_s: W8, Y, ws, stream=None):
    _check(lib().moe_down_w8a8(
        _dev(H, torch.int16, "H"), ctypes.byref(dims), Wd, Wd_s, _dev(Y, torch.float32, "Y"),
        _ptr(ws), ws.numel(), _stream(stream)), "moe_down_w8a8")


def moe_debug_set_waits(ws, wait_ns: int, withhold_stage: int, stream=None):
    """Test hook: the bounded waits' limit and a withheld pipeline stage (see moe.h)."""
    _check(lib().moe_debug_set_waits(_ptr(ws), ws.numel(), wait_ns, withhold_stage,
                                     _stream(stream)), "moe_debug_set_waits")


def moe_import_q4_blocks(blocks: torch.Tensor, K: int, group: int, w_scratch=None,
                         q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                         stream=None):
    """GGUF-style Q4 blocks uint8 [rows][K/32*18] -> (q uint8 [rows][K/2], s fp16 bits as
    int16 [rows][K/group], w_scratch fp32 [rows][K] holding the decoded weights)."""
    rows = blocks.shape[0]
    if blocks.dim() != 2 or blocks.shape[1] != (K // 32) * 18:
        raise ValueError("blocks must be [rows][K/32*18] bytes")
    dev = blocks.device
    with _made_for(stream):
        if w_scratch is None:
            w_scratch = torch.empty((rows, K), dtype=torch.float32, device=dev)
        if q is None:
            q = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
        if s is None:
            s = torch.empty((rows, K // group), dtype=torch.int16, device=dev)
    _check(lib().moe_import_q4_blocks(
        _dev(blocks, torch.uint8, "blocks"), rows, K, group,
        _dev(w_scratch, torch.float32, "w_scratch"), _dev(q, torch.uint8, "q"),
        _dev(s, torch.int16, "s"), _stream(stream)), "moe_import_q4_blocks")
    return q, s, w_scratch


def moe_workspace_bytes(dims: Dims) -> int:
    return lib().moe_workspace_bytes(ctypes.byref(dims))


def moe_layer_workspace_bytes(dims: Dims) -> int:
    return lib().moe_layer_workspace_bytes(ctypes.byref(dims))


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zero-initialised workspace buffer (256-byte aligned by the allocator)."""
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


def moe_router_topk(x, W_r, bias, dims: Dims, topk_idx, topk_w, margin, ws, stream=None):
    _check(lib().moe_router_topk(
        _dev(x, torch.int16, "x"), _dev(W_r, torch.float32, "W_r"),
        _dev(bias, torch.float32, "bias"), ctypes.byref(dims),
        _dev(topk_idx, torch.int32, "topk_idx"), _dev(topk_w, torch.float32, "topk_w"),
        None if margin is None else _dev(margin, torch.float32, "margin"),
        _ptr(ws), ws.numel(), _stream(stream)), "moe_router_topk")


def moe_router_topk_noalloc(x, W_r, bias, dims: Dims, topk_idx, topk_w, margin, stream=None):
    """The router without a workspace: its scratch is a fixed device array inside the
    library (see include/moe.h for the size limit and the sharing rules)."""
    _check(lib().moe_router_topk_noalloc(
        _dev(x, torch.int16, "x"), _dev(W_r, torch.float32, "W_r"),
        _dev(bias, torch.float32, "bias"), ctypes.byref(dims),
        _dev(topk_idx, torch.int32, "topk_idx"), _dev(topk_w, torch.float32, "topk_w"),
        None if margin is None else _dev(margin, torch.float32, "margin"), _stream(stream)),
        "moe_router_topk_noalloc")


def moe_build_descriptors(topk_idx, dims: Dims, counts, offsets, perm, pos, sched, ws,
                          stream=None):
    _check(lib().moe_build_descriptors(
        _dev(topk_idx, torch.int32, "topk_idx"), ctypes.byref(dims),
        _dev(counts, torch.int32, "counts"), _dev(offsets, torch.int32, "offsets"),
        _dev(perm, torch.int32, "perm"), _dev(pos, torch.int32, "pos"),
        _dev(sched, torch.int32, "sched"), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_build_descriptors")


def moe_gateup_swiglu_w4a16(x, dims: Dims, offsets, perm, sched, Wgu: W4, Wgu_s: W4, H, ws,
                            stream=None):
    _check(lib().moe_gateup_swiglu_w4a16(
        _dev(x, torch.int16, "x"), ctypes.byref(dims), _dev(offsets, torch.int32, "offsets"),
        _dev(perm, torch.int32, "perm"), _dev(sched, torch.int32, "sched"), Wgu, Wgu_s,
        _dev(H, torch.int16, "H"), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_gateup_swiglu_w4a16")


def moe_down_w4a16(H, dims: Dims, offsets, sched, Wd: W4, Wd_s: W4, Y, ws, stream=None):
    _check(lib().moe_down_w4a16(
        _dev(H, torch.int16, "H"), ctypes.byref(dims), _dev(offsets, torch.int32, "offsets"),
        _dev(sched, torch.int32, "sched"), Wd, Wd_s, _dev(Y, torch.float32, "Y"), _ptr(ws),
        ws.numel(), _stream(stream)), "moe_down_w4a16")


def moe_down_combine_w4a16(H, dims: Dims, offsets, sched, topk_w, pos, Wd: W4, Wd_s: W4,
                           residual, out, ws, stream=None):
    """Down projection with the weighted combine (and an optional residual) fused in;
    ws is a layer-sized workspace (it holds Y)."""
    _check(lib().moe_down_combine_w4a16(
        _dev(H, torch.int16, "H"), ctypes.byref(dims), _dev(offsets, torch.int32, "offsets"),
        _dev(sched, torch.int32, "sched"), _dev(topk_w, torch.float32, "topk_w"),
        _dev(pos, torch.int32, "pos"), Wd, Wd_s,
        None if residual is None else _dev(residual, torch.int16, "residual"),
        _dev(out, torch.int16, "out"), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_down_combine_w4a16")


def moe_combine_shared(Y, topk_w, pos, dims: Dims, out, stream=None):
    _check(lib().moe_combine_shared(
        _dev(Y, torch.float32, "Y"), _dev(topk_w, torch.float32, "topk_w"),
        _dev(pos, torch.int32, "pos"), ctypes.byref(dims), _dev(out, torch.int16, "out"),
        _stream(stream)), "moe_combine_shared")


def moe_combine_shared_residual(Y, topk_w, pos, dims: Dims, residual, out, stream=None):
    """out = bf16(residual + (routed + shared)); out may be residual itself."""
    _check(lib().moe_combine_shared_residual(
        _dev(Y, torch.float32, "Y"), _dev(topk_w, torch.float32, "topk_w"),
        _dev(pos, torch.int32, "pos"), ctypes.byref(dims), _dev(residual, torch.int16, "residual"),
        _dev(out, torch.int16, "out"), _stream(stream)), "moe_combine_shared_residual")


def moe_layer_forward_residual(x, W_r, bias, dims: Dims, Wgu: W4, Wd: W4, Wgu_s: W4, Wd_s: W4,
                               residual, out, ws, stream=None):
    """The layer with the residual add in its last kernel; out may be residual itself."""
    _check(lib().moe_layer_forward_residual(
        _dev(x, torch.int16, "x"), _dev(W_r, torch.float32, "W_r"),
        _dev(bias, torch.float32, "bias"), ctypes.byref(dims), Wgu, Wd, Wgu_s, Wd_s,
        _dev(residual, torch.int16, "residual"), _dev(out, torch.int16, "out"), _ptr(ws),
        ws.numel(), _stream(stream)), "moe_layer_forward_residual")


def moe_pack_w4_bytes(rows: int, K: int, group: int) -> tuple[int, int]:
    """(packed bytes, scale bytes) of moe_pack_w4's output; (0, 0) for arguments it
    rejects."""
    sb = ctypes.c_size_t(0)
    qb = lib().moe_pack_w4_bytes(rows, K, group, ctypes.byref(sb))
    return int(qb), int(sb.value)


def moe_layer_forward(x, W_r, bias, dims: Dims, Wgu: W4, Wd: W4, Wgu_s: W4, Wd_s: W4, out, ws,
                      stream=None):
    _check(lib().moe_layer_forward(
        _dev(x, torch.int16, "x"), _dev(W_r, torch.float32, "W_r"),
        _dev(bias, torch.float32, "bias"), ctypes.byref(dims), Wgu, Wd, Wgu_s, Wd_s,
        _dev(out, torch.int16, "out"), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_layer_forward")


def moe_layer_forward_host(x_host, W_r, bias, dims: Dims, Wgu: W4, Wd: W4, Wgu_s: W4, Wd_s: W4,
                           out_host, ws, stream=None):
    """x_host / out_host: pinned CPU int16 tensors [T][d].  Asynchronous."""
    for t, n in ((x_host, "x_host"), (out_host, "out_host")):
        if t.is_cuda or t.dtype != torch.int16 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous CPU int16 tensor")
    _check(lib().moe_layer_forward_host(
        x_host.data_ptr(), _dev(W_r, torch.float32, "W_r"), _dev(bias, torch.float32, "bias"),
        ctypes.byref(dims), Wgu, Wd, Wgu_s, Wd_s, out_host.data_ptr(), _ptr(ws), ws.numel(),
        _stream(stream)), "moe_layer_forward_host")


def moe_check_device_status(ws, stream=None) -> int:
    """Synchronises the stream; returns the status (MOE_ERR_DEVICE_CHECK if a device check
    tripped since the last call) without raising."""
    return lib().moe_check_device_status(_ptr(ws), ws.numel(), _stream(stream))


# ------------------------------------------------------- the paged cache and its attention

_KV_DTYPES = {MOE_KV_BF16: (torch.bfloat16, torch.int16), MOE_KV_E4M3: (torch.uint8,),
              MOE_KV_INT4: (torch.uint8,)}


def kv_cache(k: torch.Tensor, v: torch.Tensor, ks: torch.Tensor | None = None,
             vs: torch.Tensor | None = None) -> Kv:
    """A cache pool from its tensors: k and v [n_pages][H_kv][page][row], bf16 rows of D values
    or uint8 rows of D (E4M3) or D/2 (int4) bytes.  The first three dimensions may have any
    strides that are multiples of 16 bytes, the same for k and v; the rows are contiguous.
    ks and vs: fp32 [n_pages][H_kv][page], contiguous; for uint8 rows only.  The tensors must
    outlive the handle."""
    if not (k.is_cuda and v.is_cuda):
        raise ValueError("k and v must be CUDA tensors")
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must be 4-dimensional, of one shape and type")
    if k.dtype not in (torch.bfloat16, torch.int16, torch.uint8):
        raise ValueError(f"k and v must be bf16 or uint8, got {k.dtype}")
    if k.stride(3) != 1 or v.stride(3) != 1:
        raise ValueError("the rows of k and v must be contiguous")
    size = k.element_size()
    row = k.shape[3] * size

    def strides(t):  # a dimension of one element has no stride of its own
        return [t.stride(i) * size if t.shape[i] > 1 else row for i in range(3)]

    if strides(k) != strides(v):
        raise ValueError("k and v must have the same strides")
    quantised = k.dtype == torch.uint8
    if quantised != (ks is not None) or quantised != (vs is not None):
        raise ValueError("ks and vs belong to uint8 rows, both of them")
    for t, n in ((ks, "ks"), (vs, "vs")):
        if t is not None and tuple(t.shape) != tuple(k.shape[:3]):
            raise ValueError(f"{n} must be [n_pages][H_kv][page]")
    if any(t is not None and t.get_device() != k.get_device() for t in (v, ks, vs)):
        raise ValueError("the cache's tensors must be on one device")
    c = Kv(k.data_ptr(), v.data_ptr(), _dev(ks, torch.float32, "ks") if quantised else None,
           _dev(vs, torch.float32, "vs") if quantised else None, *strides(k))
    c.shape, c.dtype, c.dev = tuple(k.shape), k.dtype, k.get_device()
    return c


def _kv_check(dims: KvDims, cache: Kv, H_kv: int, D: int):
    if cache.shape is None:  # made from raw pointers
        return
    fmt = dims.format
    if (cache.shape != (dims.n_pages, H_kv, dims.page, D // 2 if fmt == MOE_KV_INT4 else D) or
            (fmt in _KV_DTYPES and cache.dtype not in _KV_DTYPES[fmt])):
        raise ValueError("the cache's shape or type is not that of dims")


def _rows(t: torch.Tensor, T: int, H: int, D: int, name: str):
    """Pointer and token stride of bf16 [T][H][D] whose tokens may lie apart."""
    if not t.is_cuda or t.dtype not in _BITS16:
        raise ValueError(f"{name} must be a bf16 CUDA tensor")
    ld, head, one = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.shape != (T, H, D) or one != 1 or (head != D and H > 1):
        raise ValueError(f"{name} must be [T][H][D] with contiguous tokens, got {tuple(t.shape)}")
    return t.data_ptr(), ld if T > 1 else H * D


def _ints(t: torch.Tensor, n: int, name: str):
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    return _dev(t, torch.int32, name)


def moe_attn_workspace_bytes(dims: KvDims) -> int:
    return lib().moe_attn_workspace_bytes(ctypes.byref(dims))


def moe_kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, dims: KvDims, cache: Kv, ws,
                 stream=None):
    """New keys and values bf16 [T][H_kv][D] (tokens may lie apart) into the cache's slots
    int32 [T]; a negative slot is not written."""
    T, H, D = dims.T, dims.H_kv, dims.D
    _kv_check(dims, cache, H, D)
    kp, ldk = _rows(k, T, H, D, "k")
    vp, ldv = _rows(v, T, H, D, "v")
    status = (_lib or lib()).moe_kv_write(
        kp, ldk, vp, ldv, _ints(slots, T, "slots"), ctypes.byref(dims), ctypes.byref(cache),
        ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        raise MoeError(status, "moe_kv_write")


def moe_kv_read(slots: torch.Tensor, dims: KvDims, cache: Kv, k: torch.Tensor, v: torch.Tensor, ws,
                stream=None):
    """The slots int32 [T] back as bf16 rows k, v [T][H_kv][D]; a negative slot gives zeros."""
    T, H, D = dims.T, dims.H_kv, dims.D
    _kv_check(dims, cache, H, D)
    n = T * H * D
    if k.numel() != n or v.numel() != n:
        raise ValueError("k and v must be [T][H_kv][D]")
    status = (_lib or lib()).moe_kv_read(
        _ints(slots, T, "slots"), ctypes.byref(dims), ctypes.byref(cache), _dev(k, torch.int16, "k"),
        _dev(v, torch.int16, "v"), ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        raise MoeError(status, "moe_kv_read")


def moe_attn_paged(q: torch.Tensor, q_off: torch.Tensor, kv_len: torch.Tensor, pages: torch.Tensor,
                   dims: KvDims, cache: Kv, scale: float, out: torch.Tensor,
                   lse: torch.Tensor | None, ws, stream=None):
    """Attention of the new tokens q bf16 [T][H][D] (tokens may lie apart) over the cache, which
    holds their keys and values: out bf16 [T][H][D], lse fp32 [T][H] or None.  q_off int32
    [B+1], kv_len int32 [B], pages int32 [B][max_pages]; ws is not the layer's.  See include/moe.h."""
    T, B, H, D = dims.T, dims.B, dims.H, dims.D
    _kv_check(dims, cache, dims.H_kv, D)
    qp, ldq = _rows(q, T, H, D, "q")
    if out.numel() != T * H * D or (lse is not None and lse.numel() != T * H):
        raise ValueError("out must be [T][H][D] and lse [T][H]")
    status = (_lib or lib()).moe_attn_paged(
        qp, ldq, _ints(q_off, B + 1, "q_off"), _ints(kv_len, B, "kv_len"),
        _ints(pages, B * dims.max_pages, "pages"), ctypes.byref(dims), ctypes.byref(cache), scale,
        _dev(out, torch.int16, "out"), None if lse is None else _dev(lse, torch.float32, "lse"),
        ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        raise MoeError(status, "moe_attn_paged")


# ------------------------------------- page planning, rotary positions, block norms, 4-bit floats

_current_device = torch._C._cuda_getDevice
_I32_END = 1 << 31
_BF16, _F32, _I32, _U8 = (torch.bfloat16, torch.int16), (torch.float32,), (torch.int32,), (torch.uint8,)


def _flat(t, n: int, dtypes, dev: int, name: str):
    """Pointer of a contiguous tensor of n values on the current device, whose stream the calls go to; None
    stays None.  (One test on the way through: these calls take a few microseconds, most of them here.)"""
    if t is None:
        return None
    if t.get_device() == dev and t.numel() == n and t.dtype in dtypes and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {dtypes[0]}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    raise ValueError(f"{name} must be contiguous")


def _heads(t, shape, dev: int, name: str):
    """Pointer and token stride of bf16 [T][H][D] on the current device whose tokens may lie apart."""
    if t.get_device() == dev and t.dtype in _BF16 and t.shape == shape:
        ld, head, one = t.stride()
        T, H, D = shape
        if one == 1 and (head == D or H == 1):
            return t.data_ptr(), ld if T > 1 else H * D
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.dtype not in _BF16:
        raise ValueError(f"{name} must be {_BF16[0]}, got {t.dtype}")
    raise ValueError(f"{name} must be [T][H][D] with contiguous tokens, got {tuple(t.shape)}")


def _space(ws, dev: int):
    """Pointer and bytes of a workspace (of any type: its bytes count)."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor on the current device")
    return ws.data_ptr(), ws.nbytes


def _here(handle, dev: int, name: str):
    """A handle's tensors are on the current device, as the call's others (one made from raw pointers has no device)."""
    if handle.dev != dev and handle.dev is not None:
        raise ValueError(f"the tensors of {name} must be on the current device")


def kv_pages(kv_len: torch.Tensor, first: torch.Tensor, pages: torch.Tensor, free_pages: torch.Tensor,
             n_free: torch.Tensor) -> KvPages:
    """The state that moe_kv_plan keeps, from its int32 tensors: kv_len and first [B], pages
    [B][max_pages], free_pages [n_pages], n_free [1].  The handle keeps them alive."""
    B = kv_len.numel()
    if pages.dim() != 2 or pages.shape[0] != B:
        raise ValueError("pages must be [B][max_pages]")
    dev = _current_device()
    st = KvPages(_flat(kv_len, B, _I32, dev, "kv_len"), _flat(first, B, _I32, dev, "first"),
                 _flat(pages, pages.numel(), _I32, dev, "pages"),
                 _flat(free_pages, free_pages.numel(), _I32, dev, "free_pages"), _flat(n_free, 1, _I32, dev, "n_free"))
    st.sizes, st.dev = (B, pages.shape[1], free_pages.numel()), dev
    st.tensors = (kv_len, first, pages, free_pages, n_free)
    return st


def moe_kv_plan(new_len: torch.Tensor, dims: KvDims, state: KvPages, q_off: torch.Tensor, pos: torch.Tensor,
                slots: torch.Tensor, ws, stream=None):
    """One step of a batch planned: new_len int32 [B] tokens more (or, negative, fewer) per sequence; the
    state's lengths and pages follow, and q_off int32 [B+1], pos and slots int32 [T] name the new
    tokens.  See include/moe.h."""
    T, B = dims.T, dims.B
    if state.sizes is not None and state.sizes != (B, dims.max_pages, dims.n_pages):
        raise ValueError("the state's sizes are not those of dims")
    dev = _current_device()
    _here(state, dev, "state")
    status = (_lib or lib()).moe_kv_plan(
        _flat(new_len, B, _I32, dev, "new_len"), dims, state, _flat(q_off, B + 1, _I32, dev, "q_off"),
        _flat(pos, T, _I32, dev, "pos"), _flat(slots, T, _I32, dev, "slots"), *_space(ws, dev), _stream(stream))
    if status:
        raise MoeError(status, "moe_kv_plan")


def moe_rope_table(config: RopeConfig, pos0: int, table: torch.Tensor, stream=None):
    """The rotary table fp32 [n_pos][rot] of positions pos0 on: cosines, then sines."""
    if table.dim() != 2 or table.shape[1] != config.rot:
        raise ValueError("table must be [n_pos][rot]")
    if not -_I32_END <= pos0 < _I32_END:  # (it would be cut to another position)
        raise ValueError(f"pos0 must be a position below 2^31, got {pos0}")
    status = (_lib or lib()).moe_rope_table(config, pos0, table.shape[0],
                                            _flat(table, table.numel(), _F32, _current_device(), "table"),
                                            _stream(stream))
    if status:
        raise MoeError(status, "moe_rope_table")


def rope(table: torch.Tensor, flags: int = 0, q_norm: torch.Tensor | None = None,
         k_norm: torch.Tensor | None = None, eps: float = 0.0) -> Rope:
    """How rows are turned: a table fp32 [n_pos][rot], MOE_ROPE_* flags, and the weights fp32 [D] of the
    heads' norms, if any.  The handle keeps them alive."""
    if table.dim() != 2:
        raise ValueError("table must be [n_pos][rot]")
    widths = {t.numel() for t in (q_norm, k_norm) if t is not None}
    if len(widths) > 1:
        raise ValueError("q_norm and k_norm must be [D]")
    D, dev = widths.pop() if widths else None, _current_device()
    r = Rope(_flat(table, table.numel(), _F32, dev, "table"), _flat(q_norm, D, _F32, dev, "q_norm"),
             _flat(k_norm, D, _F32, dev, "k_norm"), table.shape[0], table.shape[1], flags, eps)
    r.D, r.dev = D, dev
    r.tensors = (table, q_norm, k_norm)
    return r


def _rope_check(rope: Rope, D: int, dev: int):
    _here(rope, dev, "rope")
    if rope.D is not None and rope.D != D:
        raise ValueError(f"the norms must be [D] with D = {D}")


def moe_rope_rows(x: torch.Tensor, pos: torch.Tensor, rope: Rope, out: torch.Tensor, ws, stream=None):
    """Rows bf16 [T][H][D] (tokens may lie apart), normalised by q_norm where rope has it, turned to their
    positions int32 [T].  out may be x."""
    if x.dim() != 3:
        raise ValueError("x must be [T][H][D]")
    T, H, D = x.shape
    dev = _current_device()
    _rope_check(rope, D, dev)
    status = (_lib or lib()).moe_rope_rows(
        *_heads(x, (T, H, D), dev, "x"), _flat(pos, T, _I32, dev, "pos"), T, H, D, rope,
        *_heads(out, (T, H, D), dev, "out"), *_space(ws, dev), _stream(stream))
    if status:
        raise MoeError(status, "moe_rope_rows")


def moe_rope_kv_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, slots: torch.Tensor,
                      rope: Rope, dims: KvDims, cache: Kv, q_out: torch.Tensor, ws, stream=None):
    """New queries bf16 [T][H][D] turned into q_out (which may be q), new keys [T][H_kv][D] turned and
    written into the cache's slots with the values (tokens of each may lie apart)."""
    T, H, D = dims.T, dims.H, dims.D
    _kv_check(dims, cache, dims.H_kv, D)
    dev, wide, narrow = _current_device(), (T, H, D), (T, dims.H_kv, D)
    _here(cache, dev, "cache")
    _rope_check(rope, D, dev)
    status = (_lib or lib()).moe_rope_kv_write(
        *_heads(q, wide, dev, "q"), *_heads(k, narrow, dev, "k"), *_heads(v, narrow, dev, "v"),
        _flat(pos, T, _I32, dev, "pos"), _flat(slots, T, _I32, dev, "slots"), rope, dims, cache,
        *_heads(q_out, wide, dev, "q_out"), *_space(ws, dev), _stream(stream))
    if status:
        raise MoeError(status, "moe_rope_kv_write")


def moe_block_norm(y: torch.Tensor | None, residual: torch.Tensor, gate: torch.Tensor | None,
                   w_post: torch.Tensor | None, w_pre: torch.Tensor | None, dims: NormDims,
                   residual_out: torch.Tensor | None, x: torch.Tensor | None, stream=None):
    """residual_out = residual + scale * gate * norm(y) and x = norm(residual_out), each part where it
    is given: y, x bf16 [T][d], residual bf16 or fp32 (MOE_NORM_RESIDUAL_F32), the norms' weights fp32 [d],
    the gate by dims.gate.  residual_out may be residual and x may be y.  See include/moe.h."""
    T, d, kind, dev = dims.T, dims.d, dims.gate, _current_device()
    n, res = T * d, _F32 if dims.flags & MOE_NORM_RESIDUAL_F32 else _BF16
    if gate is not None:
        gate = _flat(gate, T if kind == MOE_GATE_TOKEN else d if kind == MOE_GATE_CHANNEL else n,
                     _F32 if kind in (MOE_GATE_TOKEN, MOE_GATE_CHANNEL) else _BF16, dev, "gate")
    status = (_lib or lib()).moe_block_norm(
        _flat(y, n, _BF16, dev, "y"), _flat(residual, n, res, dev, "residual"), gate,
        _flat(w_post, d, _F32, dev, "w_post"), _flat(w_pre, d, _F32, dev, "w_pre"), dims,
        _flat(residual_out, n, res, dev, "residual_out"), _flat(x, n, _BF16, dev, "x"), _stream(stream))
    if status:
        raise MoeError(status, "moe_block_norm")


def moe_fp4_scale_bytes(rows: int, K: int) -> int:
    if max(rows, K) >= _I32_END:
        return 0
    return lib().moe_fp4_scale_bytes(rows, K)


def fp4(q: torch.Tensor, b: torch.Tensor, s: torch.Tensor) -> Fp4:
    """Rows in 4-bit floats: q uint8 [rows][K/2], b uint8 block scales in their tiles, s fp32 [rows].  The
    handle keeps them alive."""
    if q.dim() != 2 or s.numel() != q.shape[0] or b.numel() != moe_fp4_scale_bytes(q.shape[0], 2 * q.shape[1]):
        raise ValueError("q must be [rows][K/2], s [rows] and b moe_fp4_scale_bytes(rows, K) bytes")
    dev = _current_device()
    w = Fp4(_flat(q, q.numel(), _U8, dev, "q"), _flat(b, b.numel(), _U8, dev, "b"), _flat(s, s.numel(), _F32, dev, "s"))
    w.shape, w.dev, w.tensors = (q.shape[0], 2 * q.shape[1]), dev, (q, b, s)
    return w


def _fp4_out(x: torch.Tensor, q, b, s, stream):
    if x.dim() != 2:
        raise ValueError("rows must be [rows][K]")
    rows, K = x.shape
    n = moe_fp4_scale_bytes(rows, K)
    if q is None or b is None or s is None:
        with _made_for(stream):
            if q is None:
                q = torch.empty((rows, K // 2), dtype=torch.uint8, device=x.device)
            if b is None:  # (zeros: the tiles' bytes past the last row are not written)
                b = torch.zeros(n, dtype=torch.uint8, device=x.device)
            if s is None:
                s = torch.empty(rows, dtype=torch.float32, device=x.device)
    dev = _current_device()
    return rows, K, q, b, s, (_flat(q, rows * (K // 2), _U8, dev, "q"), _flat(b, n, _U8, dev, "b"),
                              _flat(s, rows, _F32, dev, "s"))


def moe_pack_fp4(w: torch.Tensor, q: torch.Tensor | None = None, b: torch.Tensor | None = None,
                 s: torch.Tensor | None = None, stream=None):
    """fp32 [rows][K] -> (codes uint8 [rows][K/2], block scales uint8, row scales fp32 [rows])."""
    rows, K, q, b, s, to = _fp4_out(w, q, b, s, stream)
    _check((_lib or lib()).moe_pack_fp4(_flat(w, rows * K, _F32, _current_device(), "w"), rows, K, *to, _stream(stream)),
           "moe_pack_fp4")
    return q, b, s


def moe_quant_rows_fp4(x: torch.Tensor, q: torch.Tensor | None = None, b: torch.Tensor | None = None,
                       s: torch.Tensor | None = None, stream=None):
    """bf16 [rows][K] -> (codes uint8 [rows][K/2], block scales uint8, row scales fp32 [rows])."""
    rows, K, q, b, s, to = _fp4_out(x, q, b, s, stream)
    _check((_lib or lib()).moe_quant_rows_fp4(_flat(x, rows * K, _BF16, _current_device(), "x"), rows, K, *to,
                                              _stream(stream)), "moe_quant_rows_fp4")
    return q, b, s


def moe_unpack_fp4(q: torch.Tensor, b: torch.Tensor, s: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """What rows in 4-bit floats stand for, bf16 [rows][K]."""
    w = fp4(q, b, s)
    rows, K = w.shape
    if out is None:
        with _made_for(stream):
            out = torch.empty((rows, K), dtype=torch.bfloat16, device=q.device)
    _check((_lib or lib()).moe_unpack_fp4(w, rows, K, _flat(out, rows * K, _BF16, _current_device(), "out"),
                                          _stream(stream)), "moe_unpack_fp4")
    return out


def moe_linear_fp4_workspace_bytes(T: int, N: int, K: int) -> int:
    if max(T, N, K) >= _I32_END:
        return 0
    return lib().moe_linear_fp4_workspace_bytes(T, N, K)


def moe_linear_fp4(x: torch.Tensor, w: Fp4, out: torch.Tensor, ws, stream=None):
    """out bf16 [T][N] = the projection of x bf16 [T][K] (tokens may lie apart), quantised to 4-bit floats,
    by weights w of moe_pack_fp4."""
    if w.shape is None:
        raise ValueError("w must come from fp4()")
    N, K = w.shape
    dev = _current_device()
    _here(w, dev, "w")
    if x.dim() != 2 or x.get_device() != dev or x.dtype not in _BF16:
        raise ValueError("x must be a bf16 CUDA tensor [T][K] on the current device")
    (T, width), (ld, one) = x.shape, x.stride()
    if width != K or one != 1:
        raise ValueError(f"x must be [T][{K}] with contiguous tokens, got {tuple(x.shape)}")
    status = (_lib or lib()).moe_linear_fp4(
        x.data_ptr(), ld if T > 1 else K, T, N, K, w, _flat(out, T * N, _BF16, dev, "out"), *_space(ws, dev),
        _stream(stream))
    if status:
        raise MoeError(status, "moe_linear_fp4")
