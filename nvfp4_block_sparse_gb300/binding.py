"""ctypes binding of libqsa.so: the C entry points of include/qsa.h under the
same names, taking torch CUDA tensors.  Argument marshalling only -- every
step runs in the library's CUDA kernels; there is no CPU fallback, and a
missing library raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

QSA_OK = 0
QSA_ERR_INVALID_ARG = 1
QSA_ERR_UNSUPPORTED = 2
QSA_ERR_CUDA = 3
QSA_ERR_WORKSPACE = 4
QSA_ERR_DEVICE_TIMEOUT = 5

# Every symbol include/qsa.h declares.
EXPORTS = (
    "qsa_status_string",
    "qsa_index_scores",
    "qsa_select_topk",
    "qsa_sparse_decode_workspace_bytes",
    "qsa_sparse_decode_workspace_bytes_ex",
    "qsa_workspace_init",
    "qsa_sparse_decode",
    "qsa_sparse_decode_ex",
    "qsa_sparse_decode_noalloc",
    "qsa_sparse_decode_noalloc_status",
    "qsa_debug_set_wait_ns",
    "qsa_debug_bounds_status",
    "qsa_workspace_status",
    "qsa_store_kv_tokens",
    "qsa_select_sparse_decode",
    "qsa_select_sparse_decode_fused",
    "qsa_rollback_state_bytes",
    "qsa_rollback_gather",
    "qsa_rollback_restore",
    "qsa_sparse_prefill_workspace_bytes",
    "qsa_sparse_prefill",
    "qsa_rope_init",
    "qsa_rope_rows",
    "qsa_qk_norm_rope",
    "qsa_store_kv_tokens_rope",
    "qsa_load_kv_tokens",
    "qsa_dense_attention_workspace_bytes",
    "qsa_dense_attention",
    "qsa_rope_axes_init",
    "qsa_rope_axes_rows",
    "qsa_store_kv_tokens_fp8",
    "qsa_load_kv_tokens_fp8",
    "qsa_dense_attention_fp8_workspace_bytes",
    "qsa_dense_attention_fp8",
    "qsa_prompt_attention_workspace_bytes",
    "qsa_prompt_attention",
)

ROPE_LAYOUTS = {"sections": 0, "interleaved": 1, "spectra": 2}
ROPE_SCALINGS = {"none": 0, "linear": 1, "yarn": 2, "wavelength": 3}


class QsaError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__("%s failed: %s (status %d)" % (fn, msg, status))
        self.status = status


class qsa_geom_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "rows_per_req", "num_q_heads", "num_kv_heads", "head_dim",
        "index_dim", "page_size", "max_blocks", "num_pages")]


class qsa_rope_config_t(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("scaling", ctypes.c_int)] + [
        (n, ctypes.c_double) for n in ("theta", "factor", "original_context", "low", "high",
                                       "attention_factor")]


class qsa_rope_t(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("amplitude", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 128)]


class qsa_rope_axes_t(ctypes.Structure):
    _fields_ = [("rope", qsa_rope_t), ("axes", ctypes.c_int), ("axis", ctypes.c_uint8 * 128)]


class qsa_norm_rope_t(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("weight_plus_one", ctypes.c_int), ("eps", ctypes.c_float)]


_lib = None
_vp = ctypes.c_void_p


def bounds_checked() -> bool:
    """True when QSA_BOUNDS_CHECKED=1 selects the bounds-checked library."""
    return os.environ.get("QSA_BOUNDS_CHECKED", "") == "1"


def library_path() -> str:
    return _build.BOUNDS_LIB if bounds_checked() else _build.LIB


def load(build_if_missing: bool = False):
    """Loads libqsa.so, or libqsa_bounds.so under QSA_BOUNDS_CHECKED=1
    (building first only when asked)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise ImportError("%s is not built (run __graft_entry__.build() or "
                              "python -m nvfp4_block_sparse_gb300.build)" % os.path.basename(path))
        _build.build()
    lib = ctypes.CDLL(path)
    G = ctypes.POINTER(qsa_geom_t)
    st = ctypes.c_int
    lib.qsa_status_string.restype = ctypes.c_char_p
    lib.qsa_status_string.argtypes = [st]
    lib.qsa_index_scores.restype = st
    lib.qsa_index_scores.argtypes = [G, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.qsa_select_topk.restype = st
    lib.qsa_select_topk.argtypes = [G, _vp, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]
    lib.qsa_sparse_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.qsa_sparse_decode_workspace_bytes.argtypes = [G, ctypes.c_int]
    lib.qsa_sparse_decode_workspace_bytes_ex.restype = ctypes.c_size_t
    lib.qsa_sparse_decode_workspace_bytes_ex.argtypes = [G, ctypes.c_int, ctypes.c_int]
    lib.qsa_workspace_init.restype = st
    lib.qsa_workspace_init.argtypes = [_vp, ctypes.c_size_t, _vp]
    dec = [G, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, ctypes.c_float, ctypes.c_float,
           _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t]
    lib.qsa_sparse_decode.restype = st
    lib.qsa_sparse_decode.argtypes = dec + [_vp]
    lib.qsa_sparse_decode_ex.restype = st
    lib.qsa_sparse_decode_ex.argtypes = dec + [ctypes.c_int, _vp]
    lib.qsa_select_sparse_decode_fused.restype = ctypes.c_int
    lib.qsa_select_sparse_decode_fused.argtypes = [G]
    lib.qsa_select_sparse_decode.restype = st
    lib.qsa_select_sparse_decode.argtypes = [G, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                                             ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                             _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                                             ctypes.c_size_t, ctypes.c_int, _vp]
    lib.qsa_sparse_decode_noalloc.restype = st
    lib.qsa_sparse_decode_noalloc.argtypes = [G, _vp, _vp, _vp, _vp, _vp, ctypes.c_float,
                                              ctypes.c_float, ctypes.c_float, _vp, _vp, _vp,
                                              ctypes.c_int, _vp, _vp, _vp]
    lib.qsa_store_kv_tokens.restype = st
    lib.qsa_store_kv_tokens.argtypes = [G, _vp, _vp, _vp, ctypes.c_float, ctypes.c_float, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.qsa_rollback_state_bytes.restype = ctypes.c_size_t
    lib.qsa_rollback_state_bytes.argtypes = [G]
    lib.qsa_rollback_gather.restype = st
    lib.qsa_rollback_gather.argtypes = [G] + [_vp] * 9
    lib.qsa_rollback_restore.restype = st
    lib.qsa_rollback_restore.argtypes = [G] + [_vp] * 10
    lib.qsa_sparse_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.qsa_sparse_prefill_workspace_bytes.argtypes = [G, ctypes.c_int]
    lib.qsa_sparse_prefill.restype = st
    lib.qsa_sparse_prefill.argtypes = dec + [_vp]
    f32, i64 = ctypes.c_float, ctypes.c_int64
    NR = ctypes.POINTER(qsa_norm_rope_t)
    lib.qsa_rope_init.restype = st
    lib.qsa_rope_init.argtypes = [ctypes.POINTER(qsa_rope_config_t), ctypes.POINTER(qsa_rope_t)]
    lib.qsa_rope_rows.restype = st
    lib.qsa_rope_rows.argtypes = [G, ctypes.POINTER(qsa_rope_t)] + [_vp] * 4
    lib.qsa_qk_norm_rope.restype = st
    lib.qsa_qk_norm_rope.argtypes = [G, NR, _vp, i64, _vp, i64] + [_vp] * 6
    lib.qsa_store_kv_tokens_rope.restype = st
    lib.qsa_store_kv_tokens_rope.argtypes = ([G, NR, _vp, i64, _vp, i64, _vp, i64] + [_vp] * 4 +
                                             [f32, f32] + [_vp] * 9)
    lib.qsa_load_kv_tokens.restype = st
    lib.qsa_load_kv_tokens.argtypes = [G] + [_vp] * 6 + [f32, f32] + [_vp] * 3
    AX = ctypes.POINTER(qsa_rope_axes_t)
    lib.qsa_rope_axes_init.restype = st
    lib.qsa_rope_axes_init.argtypes = [ctypes.POINTER(qsa_rope_config_t), ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int), ctypes.c_int, AX]
    lib.qsa_rope_axes_rows.restype = st
    lib.qsa_rope_axes_rows.argtypes = [AX, _vp, i64, _vp, _vp]
    lib.qsa_store_kv_tokens_fp8.restype = st
    lib.qsa_store_kv_tokens_fp8.argtypes = [G, _vp, i64, _vp, i64, _vp, i64] + [_vp] * 7
    lib.qsa_load_kv_tokens_fp8.restype = st
    lib.qsa_load_kv_tokens_fp8.argtypes = [G, _vp, i64] + [_vp] * 9
    lib.qsa_prompt_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.qsa_prompt_attention_workspace_bytes.argtypes = [G, i64]
    lib.qsa_prompt_attention.restype = st
    lib.qsa_prompt_attention.argtypes = ([G, _vp, i64, _vp, i64, _vp, i64, _vp, i64, f32, ctypes.c_int] +
                                         [_vp] * 4 + [ctypes.c_size_t, _vp])
    lib.qsa_dense_attention_fp8_workspace_bytes.restype = ctypes.c_size_t
    lib.qsa_dense_attention_fp8_workspace_bytes.argtypes = [G]
    lib.qsa_dense_attention_fp8.restype = st
    lib.qsa_dense_attention_fp8.argtypes = ([G] + [_vp] * 5 + [f32, _vp, _vp, ctypes.c_int] +
                                            [_vp] * 4 + [ctypes.c_size_t, _vp])
    lib.qsa_dense_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.qsa_dense_attention_workspace_bytes.argtypes = [G]
    lib.qsa_dense_attention.restype = st
    lib.qsa_dense_attention.argtypes = ([G] + [_vp] * 5 + [f32] * 3 + [_vp, _vp, ctypes.c_int] +
                                        [_vp] * 4 + [ctypes.c_size_t, _vp])
    lib.qsa_sparse_decode_noalloc_status.restype = st
    lib.qsa_sparse_decode_noalloc_status.argtypes = [ctypes.POINTER(ctypes.c_int), _vp]
    lib.qsa_debug_set_wait_ns.restype = None
    lib.qsa_debug_set_wait_ns.argtypes = [ctypes.c_ulonglong]
    lib.qsa_debug_bounds_status.restype = ctypes.c_int
    lib.qsa_debug_bounds_status.argtypes = []
    lib.qsa_workspace_status.restype = st
    lib.qsa_workspace_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int), _vp]
    _lib = lib
    return lib


def make_geom(**kw) -> qsa_geom_t:
    return qsa_geom_t(*[int(kw[n]) for n, _ in qsa_geom_t._fields_])


def _geom(geom) -> qsa_geom_t:
    return geom if isinstance(geom, qsa_geom_t) else make_geom(**geom)


def _check(fn: str, status: int):
    if status != QSA_OK:
        raise QsaError(fn, status, load().qsa_status_string(status).decode())


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def qsa_status_string(status: int) -> str:
    return load().qsa_status_string(int(status)).decode()


def qsa_index_scores(geom, iq, ik_pool, page_table, seqlens, scores, stream=None):
    g = _geom(geom)
    _check("qsa_index_scores", load().qsa_index_scores(
        ctypes.byref(g), _ptr(iq, torch.int8, "iq"), _ptr(ik_pool, torch.int8, "ik_pool"),
        _ptr(page_table, torch.int32, "page_table"), _ptr(seqlens, torch.int32, "seqlens"),
        _ptr(scores, torch.int32, "scores"), _stream(stream)))


def qsa_store_kv_tokens(geom, k_new, v_new, ik_new, k_scale, v_scale, page_table, seqlens,
                        k_pool, k_sf, v_pool, v_sf, ik_pool, stream=None):
    g = _geom(geom)
    _check("qsa_store_kv_tokens", load().qsa_store_kv_tokens(
        ctypes.byref(g), _ptr(k_new, torch.bfloat16, "k_new"), _ptr(v_new, torch.bfloat16, "v_new"),
        _ptr(ik_new, torch.int8, "ik_new"), float(k_scale), float(v_scale),
        _ptr(page_table, torch.int32, "page_table"), _ptr(seqlens, torch.int32, "seqlens"),
        _ptr(k_pool, torch.uint8, "k_pool"), _ptr(k_sf, torch.uint8, "k_sf"),
        _ptr(v_pool, torch.uint8, "v_pool"), _ptr(v_sf, torch.uint8, "v_sf"),
        _ptr(ik_pool, torch.int8, "ik_pool"), _stream(stream)))


def qsa_rollback_state_bytes(geom) -> int:
    g = _geom(geom)
    return int(load().qsa_rollback_state_bytes(ctypes.byref(g)))


def qsa_rollback_gather(geom, page_table, seqlens, k_pool, k_sf, v_pool, v_sf, ik_pool, saved,
                        stream=None):
    g = _geom(geom)
    _check("qsa_rollback_gather", load().qsa_rollback_gather(
        ctypes.byref(g), _ptr(page_table, torch.int32, "page_table"),
        _ptr(seqlens, torch.int32, "seqlens"), _ptr(k_pool, torch.uint8, "k_pool"),
        _ptr(k_sf, torch.uint8, "k_sf"), _ptr(v_pool, torch.uint8, "v_pool"),
        _ptr(v_sf, torch.uint8, "v_sf"), _ptr(ik_pool, torch.int8, "ik_pool"),
        _ptr(saved, torch.uint8, "saved"), _stream(stream)))


def qsa_rollback_restore(geom, page_table, seqlens, rejected, saved, k_pool, k_sf, v_pool, v_sf,
                         ik_pool, stream=None):
    g = _geom(geom)
    _check("qsa_rollback_restore", load().qsa_rollback_restore(
        ctypes.byref(g), _ptr(page_table, torch.int32, "page_table"),
        _ptr(seqlens, torch.int32, "seqlens"), _ptr(rejected, torch.int32, "rejected"),
        _ptr(saved, torch.uint8, "saved"), _ptr(k_pool, torch.uint8, "k_pool"),
        _ptr(k_sf, torch.uint8, "k_sf"), _ptr(v_pool, torch.uint8, "v_pool"),
        _ptr(v_sf, torch.uint8, "v_sf"), _ptr(ik_pool, torch.int8, "ik_pool"), _stream(stream)))


def qsa_select_sparse_decode_fused(geom) -> bool:
    g = _geom(geom)
    return bool(load().qsa_select_sparse_decode_fused(ctypes.byref(g)))


def qsa_select_sparse_decode(geom, scores, window, q, k_pool, k_sf, v_pool, v_sf, k_scale,
                             v_scale, sm_scale, page_table, seqlens, k, sel, nsel, out, lse,
                             workspace, num_splits=0, stream=None):
    g = _geom(geom)
    _check("qsa_select_sparse_decode", load().qsa_select_sparse_decode(
        ctypes.byref(g), _ptr(scores, torch.int32, "scores"), int(window),
        _ptr(q, torch.bfloat16, "q"), _ptr(k_pool, torch.uint8, "k_pool"),
        _ptr(k_sf, torch.uint8, "k_sf"), _ptr(v_pool, torch.uint8, "v_pool"),
        _ptr(v_sf, torch.uint8, "v_sf"), float(k_scale), float(v_scale), float(sm_scale),
        _ptr(page_table, torch.int32, "page_table"), _ptr(seqlens, torch.int32, "seqlens"),
        int(k), _ptr(sel, torch.int32, "sel"), _ptr(nsel, torch.int32, "nsel"),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), int(num_splits),
        _stream(stream)))


def qsa_select_topk(geom, scores, seqlens, k, window, sel, nsel, stream=None):
    g = _geom(geom)
    _check("qsa_select_topk", load().qsa_select_topk(
        ctypes.byref(g), _ptr(scores, torch.int32, "scores"),
        _ptr(seqlens, torch.int32, "seqlens"), int(k), int(window),
        _ptr(sel, torch.int32, "sel"), _ptr(nsel, torch.int32, "nsel"), _stream(stream)))


def qsa_sparse_decode_workspace_bytes(geom, k) -> int:
    return int(load().qsa_sparse_decode_workspace_bytes(ctypes.byref(_geom(geom)), int(k)))


def qsa_sparse_decode_workspace_bytes_ex(geom, k, num_splits) -> int:
    return int(load().qsa_sparse_decode_workspace_bytes_ex(ctypes.byref(_geom(geom)), int(k),
                                                            int(num_splits)))


def qsa_workspace_init(workspace, stream=None):
    _check("qsa_workspace_init", load().qsa_workspace_init(
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)))


def _decode_args(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale, page_table,
                 seqlens, sel, k, out, lse, workspace):
    g = _geom(geom)
    return [ctypes.byref(g), _ptr(q, torch.bfloat16, "q"), _ptr(k_pool, torch.uint8, "k_pool"),
            _ptr(k_sf, torch.uint8, "k_sf"), _ptr(v_pool, torch.uint8, "v_pool"),
            _ptr(v_sf, torch.uint8, "v_sf"), float(k_scale), float(v_scale), float(sm_scale),
            _ptr(page_table, torch.int32, "page_table"), _ptr(seqlens, torch.int32, "seqlens"),
            _ptr(sel, torch.int32, "sel"), int(k), _ptr(out, torch.bfloat16, "out"),
            _ptr(lse, torch.float32, "lse"), _ptr(workspace, torch.uint8, "workspace"),
            workspace.numel()], g


def qsa_sparse_decode(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale,
                      page_table, seqlens, sel, k, out, lse, workspace, stream=None):
    args, _g = _decode_args(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale,
                            page_table, seqlens, sel, k, out, lse, workspace)
    _check("qsa_sparse_decode", load().qsa_sparse_decode(*args, _stream(stream)))


def qsa_sparse_decode_ex(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale,
                         page_table, seqlens, sel, k, out, lse, workspace, num_splits,
                         stream=None):
    args, _g = _decode_args(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale,
                            page_table, seqlens, sel, k, out, lse, workspace)
    _check("qsa_sparse_decode_ex",
           load().qsa_sparse_decode_ex(*args, int(num_splits), _stream(stream)))


def qsa_sparse_prefill_workspace_bytes(geom, k) -> int:
    g = _geom(geom)
    return int(load().qsa_sparse_prefill_workspace_bytes(ctypes.byref(g), int(k)))


def qsa_sparse_prefill(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale,
                       page_table, seqlens, sel, k, out, lse, workspace, stream=None):
    args, _g = _decode_args(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale,
                            page_table, seqlens, sel, k, out, lse, workspace)
    _check("qsa_sparse_prefill", load().qsa_sparse_prefill(*args, _stream(stream)))


def qsa_sparse_decode_noalloc(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale,
                              page_table, seqlens, sel, k, out, lse, stream=None):
    """qsa_sparse_decode without a workspace, for callers that cannot
    allocate device memory: the library's built-in scratch array is used
    instead (shared by every call on the device, so overlapping calls race)."""
    g = _geom(geom)
    _check("qsa_sparse_decode_noalloc", load().qsa_sparse_decode_noalloc(
        ctypes.byref(g), _ptr(q, torch.bfloat16, "q"), _ptr(k_pool, torch.uint8, "k_pool"),
        _ptr(k_sf, torch.uint8, "k_sf"), _ptr(v_pool, torch.uint8, "v_pool"),
        _ptr(v_sf, torch.uint8, "v_sf"), float(k_scale), float(v_scale), float(sm_scale),
        _ptr(page_table, torch.int32, "page_table"), _ptr(seqlens, torch.int32, "seqlens"),
        _ptr(sel, torch.int32, "sel"), int(k), _ptr(out, torch.bfloat16, "out"),
        _ptr(lse, torch.float32, "lse"), _stream(stream)))


def qsa_sparse_decode_noalloc_status(stream=None) -> int:
    """Reads and clears the built-in scratch array's status word on the
    current device: 0, or the code of a bounded device wait that gave up in a
    qsa_sparse_decode_noalloc call since the previous query."""
    code = ctypes.c_int(0)
    st = load().qsa_sparse_decode_noalloc_status(ctypes.byref(code), _stream(stream))
    if st not in (QSA_OK, QSA_ERR_DEVICE_TIMEOUT):
        _check("qsa_sparse_decode_noalloc_status", st)
    return int(code.value)


def qsa_debug_bounds_status() -> int:
    """First failed bounds-check code since the last call (clearing them), 0
    when every check held, -1 when the loaded library has no checks."""
    return int(load().qsa_debug_bounds_status())


def qsa_debug_set_wait_ns(ns: int) -> None:
    """Diagnostics: bound of the head_dim-128 decode kernel's copy waits in ns
    (0 restores the 2 s default)."""
    load().qsa_debug_set_wait_ns(int(ns))


def qsa_workspace_status(workspace, stream=None) -> int:
    code = ctypes.c_int(0)
    st = load().qsa_workspace_status(_ptr(workspace, torch.uint8, "workspace"),
                                     ctypes.byref(code), _stream(stream))
    if st not in (QSA_OK, QSA_ERR_DEVICE_TIMEOUT):
        _check("qsa_workspace_status", st)
    return int(code.value)


# ---------------------------------------------------------------------------
# The calls below check every tensor's type, size, layout and device, make that
# device current for the launch, and default to its current stream.  A decode
# step makes one such call per layer, so the checks cost what they must: one
# pass of tensor queries, and the reason for a refusal only when there is one.
# ---------------------------------------------------------------------------

_BF16, _F32, _I32, _U8, _I8 = (torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int8)


def _refuse(t, dtype, name, numel, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on device %d, other tensors on %d" % (name, t.get_device(), dev))
    if t.numel() < numel:
        raise ValueError("%s has %d elements, needs %d" % (name, t.numel(), numel))
    raise ValueError("%s must be contiguous" % name)


def _device(t, name):
    """The CUDA device of a call's first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    return dev


def _at(t, dtype, name, numel, dev):
    """Pointer of a contiguous tensor of at least ``numel`` elements on device ``dev``."""
    try:
        if (t.dtype is dtype and t.get_device() == dev and t.numel() >= numel
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, name, numel, dev)


def _rows_at(t, heads, dims, name, rows, dev):
    """Pointer and row stride of [rows, heads, dims] bf16 rows whose heads are behind one another."""
    try:
        (n, h, d), (row, head, one) = t.shape, t.stride()
        if (t.dtype is _BF16 and t.get_device() == dev and n >= rows and h == heads and d == dims
                and one == 1 and (head == dims or heads == 1)):
            return t.data_ptr(), row if rows > 1 else heads * dims
    except (AttributeError, ValueError):
        pass
    _device(t, name)
    if t.dtype is not _BF16 or t.get_device() != dev:
        _refuse(t, _BF16, name, 0, dev)
    if t.dim() != 3 or t.shape[0] < rows or t.shape[1] != heads or t.shape[2] != dims:
        raise ValueError("%s must be [%d, %d, %d], got %s" % (name, rows, heads, dims, list(t.shape)))
    raise ValueError("%s must have its heads behind one another" % name)


def _launch(fn, dev, stream, args):
    """One library call on device ``dev``, on ``stream`` or the device's current one."""
    here = torch._C._cuda_getDevice()
    if dev != here:
        with torch.cuda.device(dev):
            return _launch(fn, dev, stream, args)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    st = fn(*args, raw)
    if st:
        _check(fn.__name__, st)


def _rope_config(rotary_dim, theta, scaling, factor, original_context, beta_fast, beta_slow,
                 low_freq, high_freq, attention_factor):
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(ROPE_SCALINGS))
    low, high = (beta_slow, beta_fast) if scaling == "yarn" else (low_freq, high_freq)
    return qsa_rope_config_t(int(rotary_dim), ROPE_SCALINGS[scaling], float(theta), float(factor),
                             float(original_context), float(low), float(high),
                             float(attention_factor))


def make_rope(rotary_dim, theta, scaling="none", factor=1.0, original_context=0.0, beta_fast=32.0,
              beta_slow=1.0, low_freq=1.0, high_freq=4.0, attention_factor=0.0) -> qsa_rope_t:
    """A rotation plan (qsa_rope_init): ``scaling`` is "none", "linear", "yarn" (beta_fast,
    beta_slow: turns within original_context) or "wavelength" (low_freq, high_freq likewise)."""
    cfg = _rope_config(rotary_dim, theta, scaling, factor, original_context, beta_fast, beta_slow,
                       low_freq, high_freq, attention_factor)
    rope = qsa_rope_t()
    _check("qsa_rope_init", load().qsa_rope_init(ctypes.byref(cfg), ctypes.byref(rope)))
    return rope


def make_rope_axes(pairs, theta, layout="sections", scaling="none", factor=1.0, original_context=0.0,
                   beta_fast=32.0, beta_slow=1.0, low_freq=1.0, high_freq=4.0,
                   attention_factor=0.0) -> qsa_rope_axes_t:
    """A rotation plan of several position axes (qsa_rope_axes_init): ``pairs`` of each axis,
    together rotary_dim / 2; ``layout`` is "sections", "interleaved" or "spectra"; the rest as
    make_rope."""
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be one of %s" % ", ".join(ROPE_LAYOUTS))
    pairs = [int(n) for n in pairs]
    cfg = _rope_config(2 * sum(pairs), theta, scaling, factor, original_context, beta_fast, beta_slow,
                       low_freq, high_freq, attention_factor)
    plan = qsa_rope_axes_t()
    _check("qsa_rope_axes_init", load().qsa_rope_axes_init(
        ctypes.byref(cfg), len(pairs), (ctypes.c_int * max(len(pairs), 1))(*pairs), ROPE_LAYOUTS[layout],
        ctypes.byref(plan)))
    return plan


def make_norm_rope(rotary_dim, interleaved=False, eps=1e-6, weight_plus_one=False) -> qsa_norm_rope_t:
    return qsa_norm_rope_t(int(rotary_dim), int(bool(interleaved)), int(bool(weight_plus_one)),
                           float(eps))


def qsa_rope_rows(geom, rope, seqlens, cs, positions=None, stream=None):
    """The step's rotation rows: cs fp32 [T, rotary_dim / 2, 2] from the lengths, or from
    ``positions`` int32 [T] (then ``seqlens`` may be None)."""
    g = _geom(geom)
    B, T = g.batch, g.batch * g.rows_per_req
    dev = _device(cs, "cs")
    _launch(load().qsa_rope_rows, dev, stream, (
        ctypes.byref(g), ctypes.byref(rope),
        None if seqlens is None else _at(seqlens, _I32, "seqlens", B, dev),
        None if positions is None else _at(positions, _I32, "positions", T, dev),
        _at(cs, _F32, "cs", T * rope.rotary_dim, dev)))


def qsa_rope_axes_rows(plan, positions, cs, stream=None):
    """Rotation rows of ``positions`` int32 [axes, T]: cs fp32 [T, rotary_dim / 2, 2]."""
    dev = _device(cs, "cs")
    if not isinstance(positions, torch.Tensor) or positions.dim() != 2 or positions.shape[0] != plan.axes:
        raise ValueError("positions must be int32 [%d, T]" % plan.axes)
    T = positions.shape[1]
    args = (ctypes.byref(plan), _at(positions, _I32, "positions", plan.axes * T, dev), T,
            _at(cs, _F32, "cs", T * plan.rope.rotary_dim, dev))
    if T:
        _launch(load().qsa_rope_axes_rows, dev, stream, args)


def qsa_qk_norm_rope(geom, norm_rope, q, k, q_weight, k_weight, cs, q_out, k_out, stream=None):
    """Norm of every query and key head with its rotation; q [T, Hq, D] and k [T, Hkv, D] may be
    views into one projection's rows; weights may be None (no norm), q and q_out too."""
    g = _geom(geom)
    T, Hq, Hkv, D = g.batch * g.rows_per_req, g.num_q_heads, g.num_kv_heads, g.head_dim
    dev = _device(k, "k")
    qp, qs = (None, 0) if q is None else _rows_at(q, Hq, D, "q", T, dev)
    kp, ks = _rows_at(k, Hkv, D, "k", T, dev)
    _launch(load().qsa_qk_norm_rope, dev, stream, (
        ctypes.byref(g), ctypes.byref(norm_rope), qp, qs, kp, ks,
        None if q_weight is None else _at(q_weight, _BF16, "q_weight", D, dev),
        None if k_weight is None else _at(k_weight, _BF16, "k_weight", D, dev),
        None if cs is None else _at(cs, _F32, "cs", T * norm_rope.rotary_dim, dev),
        None if q_out is None else _at(q_out, _BF16, "q_out", T * Hq * D, dev),
        _at(k_out, _BF16, "k_out", T * Hkv * D, dev)))


def qsa_store_kv_tokens_rope(geom, norm_rope, q, k, v, ik_new, q_weight, k_weight, cs, k_scale,
                             v_scale, page_table, seqlens, q_out, k_pool, k_sf, v_pool, v_sf,
                             ik_pool, stream=None):
    """qsa_qk_norm_rope and qsa_store_kv_tokens in one launch; v [T, Hkv, D] as k; q and q_out may
    be None."""
    g = _geom(geom)
    B, T, Hq, Hkv, D = (g.batch, g.batch * g.rows_per_req, g.num_q_heads, g.num_kv_heads,
                        g.head_dim)
    slots = g.num_pages * g.page_size
    n = slots * Hkv * D
    dev = _device(k, "k")
    qp, qs = (None, 0) if q is None else _rows_at(q, Hq, D, "q", T, dev)
    kp, ks = _rows_at(k, Hkv, D, "k", T, dev)
    vp, vs = _rows_at(v, Hkv, D, "v", T, dev)
    _launch(load().qsa_store_kv_tokens_rope, dev, stream, (
        ctypes.byref(g), ctypes.byref(norm_rope), qp, qs, kp, ks, vp, vs,
        _at(ik_new, _I8, "ik_new", T * 64, dev),
        None if q_weight is None else _at(q_weight, _BF16, "q_weight", D, dev),
        None if k_weight is None else _at(k_weight, _BF16, "k_weight", D, dev),
        None if cs is None else _at(cs, _F32, "cs", T * norm_rope.rotary_dim, dev),
        k_scale, v_scale, _at(page_table, _I32, "page_table", B * g.max_blocks, dev),
        _at(seqlens, _I32, "seqlens", B, dev),
        None if q_out is None else _at(q_out, _BF16, "q_out", T * Hq * D, dev),
        _at(k_pool, _U8, "k_pool", n // 2, dev), _at(k_sf, _U8, "k_sf", n // 16, dev),
        _at(v_pool, _U8, "v_pool", n // 2, dev), _at(v_sf, _U8, "v_sf", n // 16, dev),
        _at(ik_pool, _I8, "ik_pool", slots * 64, dev)))


def qsa_load_kv_tokens(geom, page_table, seqlens, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale,
                       k_out, v_out, stream=None):
    """The R newest rows of each request's cache as bf16 [T, Hkv, D]."""
    g = _geom(geom)
    B, m = g.batch, g.batch * g.rows_per_req * g.num_kv_heads * g.head_dim
    n = g.num_pages * g.page_size * g.num_kv_heads * g.head_dim
    dev = _device(k_out, "k_out")
    _launch(load().qsa_load_kv_tokens, dev, stream, (
        ctypes.byref(g), _at(page_table, _I32, "page_table", B * g.max_blocks, dev),
        _at(seqlens, _I32, "seqlens", B, dev),
        _at(k_pool, _U8, "k_pool", n // 2, dev), _at(k_sf, _U8, "k_sf", n // 16, dev),
        _at(v_pool, _U8, "v_pool", n // 2, dev), _at(v_sf, _U8, "v_sf", n // 16, dev),
        k_scale, v_scale, _at(k_out, _BF16, "k_out", m, dev), _at(v_out, _BF16, "v_out", m, dev)))


def _pools8(g, k_pool, k_exp, v_pool, v_exp, dev):
    n = g.num_pages * g.page_size * g.num_kv_heads
    return (_at(k_pool, _U8, "k_pool", n * g.head_dim, dev), _at(k_exp, _U8, "k_exp", n // 16, dev),
            _at(v_pool, _U8, "v_pool", n * g.head_dim, dev), _at(v_exp, _U8, "v_exp", n // 16, dev))


def qsa_store_kv_tokens_fp8(geom, k, v, page_table, seqlens, k_pool, k_exp, v_pool, v_exp,
                            cu_rows=None, stream=None):
    """Appends the requests' newest rows k, v [T, Hkv, D] (views into one projection's rows, say) to
    the 8-bit cache; with ``cu_rows`` int32 [B + 1] request b's are rows cu_rows[b]..cu_rows[b + 1] - 1."""
    g = _geom(geom)
    B, Hkv, D = g.batch, g.num_kv_heads, g.head_dim
    dev = _device(k, "k")
    T = B * g.rows_per_req if cu_rows is None else k.shape[0]
    kp, ks = _rows_at(k, Hkv, D, "k", T, dev)
    vp, vs = _rows_at(v, Hkv, D, "v", T, dev)
    args = (ctypes.byref(g), kp, ks, vp, vs,
            None if cu_rows is None else _at(cu_rows, _I32, "cu_rows", B + 1, dev), T,
            _at(page_table, _I32, "page_table", B * g.max_blocks, dev), _at(seqlens, _I32, "seqlens", B, dev),
            *_pools8(g, k_pool, k_exp, v_pool, v_exp, dev))
    if T:
        _launch(load().qsa_store_kv_tokens_fp8, dev, stream, args)


def qsa_load_kv_tokens_fp8(geom, page_table, seqlens, k_pool, k_exp, v_pool, v_exp, k_out, v_out,
                           cu_rows=None, stream=None):
    """The requests' newest rows of the 8-bit cache as bf16 [T, Hkv, D], rows as in
    qsa_store_kv_tokens_fp8."""
    g = _geom(geom)
    B = g.batch
    dev = _device(k_out, "k_out")
    T = B * g.rows_per_req if cu_rows is None else k_out.shape[0]
    m = T * g.num_kv_heads * g.head_dim
    args = (ctypes.byref(g), None if cu_rows is None else _at(cu_rows, _I32, "cu_rows", B + 1, dev), T,
            _at(page_table, _I32, "page_table", B * g.max_blocks, dev), _at(seqlens, _I32, "seqlens", B, dev),
            *_pools8(g, k_pool, k_exp, v_pool, v_exp, dev),
            _at(k_out, _BF16, "k_out", m, dev), _at(v_out, _BF16, "v_out", m, dev))
    if T:
        _launch(load().qsa_load_kv_tokens_fp8, dev, stream, args)


def qsa_dense_attention_workspace_bytes(geom) -> int:
    return int(load().qsa_dense_attention_workspace_bytes(ctypes.byref(_geom(geom))))


def qsa_dense_attention(geom, q, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale, sm_scale, page_table,
                        seqlens, out, lse, workspace, window=0, sinks=None, stream=None):
    """Dense attention of every row over its request's cached tokens (the newest ``window`` of
    them unless 0), with an optional sink logit per query head."""
    g = _geom(geom)
    B, m, D = g.batch, g.batch * g.rows_per_req * g.num_q_heads, g.head_dim
    n = g.num_pages * g.page_size * g.num_kv_heads * D
    dev = _device(q, "q")
    _launch(load().qsa_dense_attention, dev, stream, (
        ctypes.byref(g), _at(q, _BF16, "q", m * D, dev),
        _at(k_pool, _U8, "k_pool", n // 2, dev), _at(k_sf, _U8, "k_sf", n // 16, dev),
        _at(v_pool, _U8, "v_pool", n // 2, dev), _at(v_sf, _U8, "v_sf", n // 16, dev),
        k_scale, v_scale, sm_scale, _at(page_table, _I32, "page_table", B * g.max_blocks, dev),
        _at(seqlens, _I32, "seqlens", B, dev), window,
        None if sinks is None else _at(sinks, _F32, "sinks", g.num_q_heads, dev),
        _at(out, _BF16, "out", m * D, dev), _at(lse, _F32, "lse", m, dev),
        _at(workspace, _U8, "workspace", 0, dev), workspace.numel()))


def qsa_dense_attention_fp8_workspace_bytes(geom) -> int:
    return int(load().qsa_dense_attention_fp8_workspace_bytes(ctypes.byref(_geom(geom))))


def qsa_dense_attention_fp8(geom, q, k_pool, k_exp, v_pool, v_exp, sm_scale, page_table, seqlens, out,
                            lse, workspace, window=0, sinks=None, stream=None):
    """qsa_dense_attention over the 8-bit cache."""
    g = _geom(geom)
    B, m, D = g.batch, g.batch * g.rows_per_req * g.num_q_heads, g.head_dim
    dev = _device(q, "q")
    _launch(load().qsa_dense_attention_fp8, dev, stream, (
        ctypes.byref(g), _at(q, _BF16, "q", m * D, dev), *_pools8(g, k_pool, k_exp, v_pool, v_exp, dev),
        sm_scale, _at(page_table, _I32, "page_table", B * g.max_blocks, dev),
        _at(seqlens, _I32, "seqlens", B, dev), window,
        None if sinks is None else _at(sinks, _F32, "sinks", g.num_q_heads, dev),
        _at(out, _BF16, "out", m * D, dev), _at(lse, _F32, "lse", m, dev),
        _at(workspace, _U8, "workspace", 0, dev), workspace.numel()))


def qsa_prompt_attention_workspace_bytes(geom, total_rows) -> int:
    return int(load().qsa_prompt_attention_workspace_bytes(ctypes.byref(_geom(geom)), int(total_rows)))


def qsa_prompt_attention(geom, q, k, v, cu_seqlens, sm_scale, out, lse, workspace, window=0, sinks=None,
                         stream=None):
    """Causal attention of packed sequences: q [T, Hq, D], k and v [T, Hkv, D] (views into one
    projection's rows, say), sequence b in rows cu_seqlens[b]..cu_seqlens[b + 1] - 1 (int32 [B + 1])."""
    g = _geom(geom)
    Hq, Hkv, D = g.num_q_heads, g.num_kv_heads, g.head_dim
    dev = _device(q, "q")
    T = q.shape[0]
    qp, qs = _rows_at(q, Hq, D, "q", T, dev)
    kp, ks = _rows_at(k, Hkv, D, "k", T, dev)
    vp, vs = _rows_at(v, Hkv, D, "v", T, dev)
    args = (ctypes.byref(g), qp, qs, kp, ks, vp, vs, _at(cu_seqlens, _I32, "cu_seqlens", g.batch + 1, dev), T,
            sm_scale, window, None if sinks is None else _at(sinks, _F32, "sinks", Hq, dev),
            _at(out, _BF16, "out", T * Hq * D, dev), _at(lse, _F32, "lse", T * Hq, dev),
            _at(workspace, _U8, "workspace", 0, dev), workspace.numel())
    if T:
        _launch(load().qsa_prompt_attention, dev, stream, args)
