"""Python binding of libkvr (include/kvr.h): argument marshalling only.

Every function has the C entry point's name and order of arguments; torch
tensors are passed by their data pointers, streams by their CUDA handle.
Import fails loudly when libkvr.so has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvr.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m selective_kv_cache_gb300.build` "
        "(or __graft_entry__.build()); the refresh has no CPU fallback")
lib = C.CDLL(LIB_PATH)

KVR_OK, KVR_EINVAL, KVR_ERANGE, KVR_ENOMEM, KVR_ECUDA, KVR_ETIMEOUT, KVR_EDEVICE, KVR_ESTATE, KVR_EUNSUPPORTED = range(9)
STATUS_NAMES = ["OK", "EINVAL", "ERANGE", "ENOMEM", "ECUDA", "ETIMEOUT", "EDEVICE", "ESTATE", "EUNSUPPORTED"]
KVR_F32, KVR_BF16, KVR_INT4 = 0, 1, 2   # KVR_INT4: page format only
KVR_SINK_STATIC = 0x1
KVR_COMMIT_META = 0x1
KVR_SPLICE_LOCAL = 0x1
KVR_SPLICE_SINK = 0x2
KVR_MOD_Q, KVR_MOD_K, KVR_MOD_V, KVR_MOD_O, KVR_MOD_MLP = range(5)
KERNELS = ["select", "gather", "rmsnorm", "gemm_qkv", "epi_qkv", "attention", "gemm_o", "epi_o",
           "gemm_gate_up", "epi_gate_up", "gemm_down", "epi_down", "commit"]
KVR_K_COUNT = len(KERNELS)

EXPORTS = ["kvr_create_cache", "kvr_destroy_cache", "kvr_select", "kvr_workspace_bytes",
           "kvr_refresh_layer", "kvr_refresh", "kvr_attend", "kvr_sync_status", "kvr_last_error",
           "kvr_read_selection", "kvr_read_meta", "kvr_profile_enable", "kvr_profile_read",
           "kvr_refresh_layer_noalloc", "kvr_refresh_interval_wise", "kvr_reselect", "kvr_lora_merge",
           "kvr_shift", "kvr_splice", "kvr_cache_info", "kvr_restart_layer", "kvr_policy_sensitivity",
           "kvr_policy_create", "kvr_policy_destroy", "kvr_policy_plan", "kvr_policy_commit", "kvr_policy_versions",
           "kvr_sur_workspace_bytes", "kvr_sur_select", "kvr_sur_status", "kvr_refresh_range",
           "kvr_wait_check", "kvr_paged_append", "kvr_paged_read", "kvr_paged_workspace_bytes", "kvr_paged_attend",
           "kvr_paged_status"]


class kvr_model_desc(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("d_model", C.c_int32), ("n_q_heads", C.c_int32),
                ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("ffn_dim", C.c_int32),
                ("rope_theta", C.c_double), ("rms_eps", C.c_float), ("dtype", C.c_int32),
                ("has_qkv_bias", C.c_int32), ("has_qk_norm", C.c_int32)]


class kvr_layer_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("w_qkv", "b_qkv", "w_o", "w_gate_up", "w_down", "norm1", "norm2",
                                          "q_norm", "k_norm")]


class kvr_pages(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("format", "n_kv_heads", "head_dim", "page_size", "group", "n_pages", "batch",
                                         "max_pages")] + \
               [(n, C.c_int64) for n in ("page_stride", "head_stride", "slot_stride")] + \
               [(n, C.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "page_table", "kv_len", "err")]


class kvr_score_opts(C.Structure):
    _fields_ = [(n, C.c_float) for n in ("scale", "softcap", "alpha", "beta")] + \
               [(n, C.c_void_p) for n in ("local_bits", "sink_bits", "slopes", "key_begin", "key_end")]


class KvrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.kvr_last_error().decode()
        super().__init__(f"{where}: {STATUS_NAMES[status] if 0 <= status < 9 else status}: {msg}")


P = C.c_void_p
I32 = C.c_int32
lib.kvr_create_cache.argtypes = [C.POINTER(kvr_model_desc), I32, I32, P, P, I32, I32, P, P, C.c_float, C.c_float,
                                 C.c_uint32, P, C.POINTER(P)]
lib.kvr_destroy_cache.argtypes = [P]
lib.kvr_select.argtypes = [P, P, P, I32, P, P, I32, P, P, P, P, P]
lib.kvr_workspace_bytes.argtypes = [P, I32]
lib.kvr_workspace_bytes.restype = C.c_size_t
lib.kvr_refresh_layer.argtypes = [P, I32, C.POINTER(kvr_layer_weights), P, P, C.c_size_t, C.c_uint32, P]
lib.kvr_refresh_layer_noalloc.argtypes = [P, I32, C.POINTER(kvr_layer_weights), P, C.c_uint32, P]
lib.kvr_refresh_interval_wise.argtypes = [P, P, P, I32, P, P, I32, P, C.POINTER(kvr_layer_weights), I32, I32, P, P,
                                          C.c_size_t, C.c_uint32, P, P]
lib.kvr_reselect.argtypes = [P, P, P, P, P, P, P, P, P]
lib.kvr_refresh_range.argtypes = [P, C.POINTER(kvr_layer_weights), I32, I32, P, P, P, P, I32, P, P, P, P, P,
                                  C.c_size_t, C.c_uint32, P]
lib.kvr_lora_merge.argtypes = [P, P, I32, I32, I32, I32, P, P, I32, C.c_float, I32, P]
lib.kvr_shift.argtypes = [P, I32, I32, P]
lib.kvr_splice.argtypes = [P, I32, I32, I32, P, P, I32, C.c_uint32, P]
lib.kvr_cache_info.argtypes = [P, P, P]
lib.kvr_restart_layer.argtypes = [I32, I32, I32]
lib.kvr_policy_sensitivity.argtypes = [I32, I32, P, P, P, P]
lib.kvr_policy_create.argtypes = [I32, C.c_int64, I32, P, P, P, C.POINTER(P)]
lib.kvr_policy_destroy.argtypes = [P]
lib.kvr_policy_plan.argtypes = [P, P, I32, I32, P, P, P, P]
lib.kvr_policy_commit.argtypes = [P, P, I32, I32, C.c_int64, P]
lib.kvr_policy_versions.argtypes = [P, P]
lib.kvr_sur_workspace_bytes.argtypes = [I32, I32, I32, I32]
lib.kvr_sur_workspace_bytes.restype = C.c_size_t
lib.kvr_sur_select.argtypes = [P, I32, I32, I32, P, I32, I32, P, I32, P, I32, I32, P, C.c_size_t, P, P, P, P]
lib.kvr_sur_status.argtypes = [P, P]
lib.kvr_refresh.argtypes = [P, C.POINTER(kvr_layer_weights), I32, I32, P, P, C.c_size_t, C.c_uint32, P]
lib.kvr_attend.argtypes = [P, I32, P, P, P, C.c_size_t, P]
lib.kvr_sync_status.argtypes = [P, P]
lib.kvr_wait_check.argtypes = [P, C.c_int64, P]
lib.kvr_last_error.restype = C.c_char_p
lib.kvr_restart_layer.restype = C.c_int32
lib.kvr_read_selection.argtypes = [P, I32, P, I32, P, I32, P, P, P, P, I32, P, P, P]
lib.kvr_read_meta.argtypes = [P, P, P]
lib.kvr_profile_enable.argtypes = [P, I32]
lib.kvr_profile_read.argtypes = [P, P, P, I32]
I64 = C.c_int64
lib.kvr_paged_append.argtypes = [P, I32, P, P, P, I64, P, I64, P, I32, P, I64, P, I32, P]
lib.kvr_paged_read.argtypes = [P, I32, P, P, P, I64, P, I64, P]
lib.kvr_paged_workspace_bytes.argtypes = [P, I32, I32, I32]
lib.kvr_paged_workspace_bytes.restype = C.c_size_t
lib.kvr_paged_attend.argtypes = [P, P, I32, I32, I32, P, P, P, I64, P, I64, P, C.c_size_t, P]
lib.kvr_paged_status.argtypes = [P, P]
for _f in EXPORTS:
    if _f not in ("kvr_workspace_bytes", "kvr_last_error", "kvr_restart_layer", "kvr_sur_workspace_bytes",
                  "kvr_paged_workspace_bytes"):
        getattr(lib, _f).restype = C.c_int


def _check(status: int, where: str):
    if status != KVR_OK:
        raise KvrError(status, where)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def model_desc(shape) -> kvr_model_desc:
    """kvr_model_desc from any object with the shape attributes."""
    return kvr_model_desc(shape.n_layers, shape.d_model, shape.n_q_heads, shape.n_kv_heads, shape.head_dim,
                          shape.ffn_dim, float(shape.rope_theta), float(shape.rms_eps),
                          KVR_BF16 if shape.dtype == "bf16" else KVR_F32, int(bool(shape.qkv_bias)),
                          int(bool(getattr(shape, "qk_norm", False))))


def layer_weights(L) -> kvr_layer_weights:
    """kvr_layer_weights from a dict of device tensors (keys as the struct)."""
    return kvr_layer_weights(*[_ptr(L.get(k)) for k in ("w_qkv", "b_qkv", "w_o", "w_gate_up", "w_down",
                                                         "norm1", "norm2", "q_norm", "k_norm")])


def layer_weights_array(layers: Sequence[dict]):
    arr = (kvr_layer_weights * len(layers))()
    for i, L in enumerate(layers):
        arr[i] = layer_weights(L)
    return arr


def kvr_create_cache(desc: kvr_model_desc, batch: int, capacity: int, k_base, v_base, n_tokens: int,
                     suffix_start: int, local_bits=None, sink_bits=None, alpha: float = 0.0, beta: float = 0.0,
                     flags: int = 0, stream=None) -> int:
    """Returns the cache handle (an int).  local_bits / sink_bits: uint32 numpy
    arrays [batch, ceil(capacity/32)] (host) or None."""
    out = P()
    lb = None if local_bits is None else local_bits.ctypes.data
    sb = None if sink_bits is None else sink_bits.ctypes.data
    _check(lib.kvr_create_cache(C.byref(desc), batch, capacity, _ptr(k_base), _ptr(v_base), n_tokens, suffix_start,
                                lb, sb, alpha, beta, flags, _stream(stream), C.byref(out)), "kvr_create_cache")
    return out.value


def kvr_destroy_cache(c: int):
    _check(lib.kvr_destroy_cache(c), "kvr_destroy_cache")


def kvr_select(c: int, positions, counts, budget_percent: int = -1, token_ids=None, embed_table=None,
               vocab: int = 0, hidden_src=None, hidden_out=None, stream=None):
    """positions, counts: host int32 numpy arrays (or pinned int32 tensors).
    Returns (n_rows, n_intervals)."""
    n_rows = I32()
    n_iv = I32()
    pp = positions.ctypes.data if hasattr(positions, "ctypes") else _ptr(positions)
    cp = counts.ctypes.data if hasattr(counts, "ctypes") else _ptr(counts)
    _check(lib.kvr_select(c, pp, cp, budget_percent, _ptr(token_ids), _ptr(embed_table), vocab, _ptr(hidden_src),
                          _ptr(hidden_out), C.byref(n_rows), C.byref(n_iv), _stream(stream)), "kvr_select")
    return n_rows.value, n_iv.value


def kvr_workspace_bytes(c: int, max_rows: int = 0) -> int:
    return lib.kvr_workspace_bytes(c, max_rows)


def kvr_refresh_layer(c: int, layer: int, weights: kvr_layer_weights, hidden_inout, workspace, ws_bytes: int,
                      flags: int = 0, stream=None):
    _check(lib.kvr_refresh_layer(c, layer, C.byref(weights), _ptr(hidden_inout), _ptr(workspace), ws_bytes, flags,
                                 _stream(stream)), "kvr_refresh_layer")


def kvr_refresh_layer_noalloc(c: int, layer: int, weights: kvr_layer_weights, hidden_inout, flags: int = 0,
                              stream=None):
    """kvr_refresh_layer with the library's fixed 64 MiB device scratch instead of
    a caller workspace (nothing is allocated)."""
    _check(lib.kvr_refresh_layer_noalloc(c, layer, C.byref(weights), _ptr(hidden_inout), flags, _stream(stream)),
           "kvr_refresh_layer_noalloc")


def kvr_refresh(c: int, weights_array, layer_begin: int, layer_end: int, hidden_inout, workspace, ws_bytes: int,
                flags: int = 0, stream=None):
    _check(lib.kvr_refresh(c, weights_array, layer_begin, layer_end, _ptr(hidden_inout), _ptr(workspace), ws_bytes,
                           flags, _stream(stream)), "kvr_refresh")


def kvr_refresh_interval_wise(c: int, positions, counts, budget_percent: int = -1, token_ids=None, embed_table=None,
                              vocab: int = 0, hidden_src=None, weights_array=None, layer_begin: int = 0,
                              layer_end: int = 0, hidden_out=None, workspace=None, ws_bytes: int = 0,
                              flags: int = KVR_COMMIT_META, stream=None) -> int:
    """Returns the number of intervals."""
    n_iv = I32()
    pp = positions.ctypes.data if hasattr(positions, "ctypes") else _ptr(positions)
    cp = counts.ctypes.data if hasattr(counts, "ctypes") else _ptr(counts)
    _check(lib.kvr_refresh_interval_wise(c, pp, cp, budget_percent, _ptr(token_ids), _ptr(embed_table), vocab,
                                         _ptr(hidden_src), weights_array, layer_begin, layer_end, _ptr(hidden_out),
                                         _ptr(workspace), ws_bytes, flags, C.byref(n_iv), _stream(stream)),
           "kvr_refresh_interval_wise")
    return n_iv.value


def kvr_reselect(c: int, positions, counts, carry_rows, fill_rows, hidden_out, stream=None):
    n_rows = I32()
    n_iv = I32()
    pp = positions.ctypes.data if hasattr(positions, "ctypes") else _ptr(positions)
    cp = counts.ctypes.data if hasattr(counts, "ctypes") else _ptr(counts)
    _check(lib.kvr_reselect(c, pp, cp, _ptr(carry_rows), _ptr(fill_rows), _ptr(hidden_out), C.byref(n_rows),
                            C.byref(n_iv), _stream(stream)), "kvr_reselect")
    return n_rows.value, n_iv.value


def kvr_refresh_range(c: int, weights_array, range_begin: int, range_end: int, positions, counts, token_ids=None,
                      embed_table=None, vocab: int = 0, hidden_src=None, boundary=None, hidden_sel=None,
                      hidden_full=None, workspace=None, ws_bytes: int = 0, flags: int = KVR_COMMIT_META, stream=None):
    pp = positions.ctypes.data if hasattr(positions, "ctypes") else _ptr(positions)
    cp = counts.ctypes.data if hasattr(counts, "ctypes") else _ptr(counts)
    _check(lib.kvr_refresh_range(c, weights_array, range_begin, range_end, pp, cp, _ptr(token_ids),
                                 _ptr(embed_table), vocab, _ptr(hidden_src), _ptr(boundary), _ptr(hidden_sel),
                                 _ptr(hidden_full), _ptr(workspace), ws_bytes, flags, _stream(stream)),
           "kvr_refresh_range")


def kvr_wait_check(c: int, cycles: int, stream=None):
    _check(lib.kvr_wait_check(c, cycles, _stream(stream)), "kvr_wait_check")


def kvr_lora_merge(w, w_out, n_out: int, K: int, row_begin: int, row_count: int, a, b, rank: int, scale: float,
                   dtype: int, stream=None):
    _check(lib.kvr_lora_merge(_ptr(w), _ptr(w_out), n_out, K, row_begin, row_count, _ptr(a), _ptr(b), rank, scale,
                              dtype, _stream(stream)), "kvr_lora_merge")


def kvr_shift(c: int, start: int, d: int, stream=None):
    _check(lib.kvr_shift(c, start, d, _stream(stream)), "kvr_shift")


def kvr_splice(c: int, seq: int, dst_pos: int, n: int, k_src, v_src, src_pos: int = 0, flags: int = 0,
               stream=None):
    _check(lib.kvr_splice(c, seq, dst_pos, n, _ptr(k_src), _ptr(v_src), src_pos, flags, _stream(stream)),
           "kvr_splice")


def kvr_cache_info(c: int):
    """(n_tokens, suffix_start) of the cache now."""
    n = C.c_int32()
    s = C.c_int32()
    _check(lib.kvr_cache_info(c, C.byref(n), C.byref(s)), "kvr_cache_info")
    return n.value, s.value


def kvr_attend(c: int, layer: int, q, out, workspace=None, ws_bytes: int = 0, stream=None):
    _check(lib.kvr_attend(c, layer, _ptr(q), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)), "kvr_attend")


def kvr_sync_status(c: int, stream=None):
    _check(lib.kvr_sync_status(c, _stream(stream)), "kvr_sync_status")


def kvr_last_error() -> str:
    return lib.kvr_last_error().decode()


def kvr_read_selection(c: int, seq: int, count: int, n_intervals: int, words: int, max_tiles: int = 4096):
    """Host copies of the device-built selection of sequence `seq`."""
    import numpy as np
    U = np.zeros(max(count, 1), np.int32)
    iv = np.zeros((max(n_intervals, 1), 2), np.int32)
    sel = np.zeros(words, np.uint32)
    eloc = np.zeros(words, np.uint32)
    esnk = np.zeros(words, np.uint32)
    plan = np.zeros((max_tiles, 6), np.int32)
    nt, rpt, kpt = I32(), I32(), I32()
    _check(lib.kvr_read_selection(c, seq, U.ctypes.data, count, iv.ctypes.data, n_intervals, sel.ctypes.data,
                                  eloc.ctypes.data, esnk.ctypes.data, plan.ctypes.data, max_tiles, C.byref(nt),
                                  C.byref(rpt), C.byref(kpt)), "kvr_read_selection")
    return dict(U=U[:count], intervals=iv[:n_intervals], sel=sel, eloc=eloc, esnk=esnk, plan=plan[:nt.value],
                rows_per_tile=rpt.value, keys_per_tile=kpt.value)


def kvr_read_meta(c: int, batch: int, words: int):
    import numpy as np
    local = np.zeros((batch, words), np.uint32)
    sink = np.zeros((batch, words), np.uint32)
    _check(lib.kvr_read_meta(c, local.ctypes.data, sink.ctypes.data), "kvr_read_meta")
    return local, sink


def kvr_profile_enable(c: int, enable: bool = True):
    _check(lib.kvr_profile_enable(c, int(enable)), "kvr_profile_enable")


def kvr_profile_read(c: int):
    """{kernel name: (launches, total ms)} since the last read."""
    ms = (C.c_double * KVR_K_COUNT)()
    n = (C.c_int64 * KVR_K_COUNT)()
    _check(lib.kvr_profile_read(c, ms, n, KVR_K_COUNT), "kvr_profile_read")
    return {KERNELS[i]: (int(n[i]), float(ms[i])) for i in range(KVR_K_COUNT)}

# ---------------------------------------------------------------- layer-range policy
def kvr_restart_layer(module: int, s: int, n_layers: int) -> int:
    return int(lib.kvr_restart_layer(module, s, n_layers))


def kvr_policy_sensitivity(n_layers: int, restart, window, drift):
    import numpy as np
    r = np.ascontiguousarray(restart, dtype=np.int32)
    w = np.ascontiguousarray(window, dtype=np.int32)
    d = np.ascontiguousarray(drift, dtype=np.float64)
    out = np.zeros(n_layers, np.float64)
    _check(lib.kvr_policy_sensitivity(n_layers, len(r), r.ctypes.data, w.ctypes.data, d.ctypes.data,
                                      out.ctypes.data), "kvr_policy_sensitivity")
    return out


def kvr_policy_create(n_layers: int, theta0, sensitivity, stream=None) -> int:
    """theta0: flat device tensor (bf16 or fp32); sensitivity: n_layers floats."""
    import numpy as np
    s = np.ascontiguousarray(sensitivity, dtype=np.float64)
    out = P()
    dt = KVR_BF16 if theta0.dtype == torch.bfloat16 else KVR_F32
    _check(lib.kvr_policy_create(n_layers, theta0.numel(), dt, _ptr(theta0), s.ctypes.data, _stream(stream),
                                 C.byref(out)), "kvr_policy_create")
    return out.value


def kvr_policy_destroy(p: int):
    _check(lib.kvr_policy_destroy(p), "kvr_policy_destroy")


def kvr_policy_plan(p: int, n_layers: int, theta_t, module: int, update_layer: int, stream=None):
    """Returns (drift [n_layers], risk [n_layers], (begin, end))."""
    import numpy as np
    d = np.zeros(n_layers, np.float64)
    q = np.zeros(n_layers, np.float64)
    rng = np.zeros(2, np.int32)
    _check(lib.kvr_policy_plan(p, _ptr(theta_t), module, update_layer, d.ctypes.data, q.ctypes.data,
                               rng.ctypes.data, _stream(stream)), "kvr_policy_plan")
    return d, q, (int(rng[0]), int(rng[1]))


def kvr_policy_commit(p: int, theta_t, begin: int, end: int, version: int, stream=None):
    _check(lib.kvr_policy_commit(p, _ptr(theta_t), begin, end, version, _stream(stream)), "kvr_policy_commit")


def kvr_policy_versions(p: int, n_layers: int):
    import numpy as np
    v = np.zeros(n_layers, np.int64)
    _check(lib.kvr_policy_versions(p, v.ctypes.data), "kvr_policy_versions")
    return v


# ---------------------------------------------------------------- Semantic-Unit Refresh selection
def kvr_sur_workspace_bytes(S: int, Q: int, d: int, n_units: int) -> int:
    return int(lib.kvr_sur_workspace_bytes(S, Q, d, n_units))


def kvr_sur_select(embed, suffix_ids, query_ids, unit_bounds, budget_percent: int, suffix_start: int, workspace,
                   positions_out, scores_out=None, stream=None) -> int:
    """Device tensors: embed [vocab, d], suffix_ids [S], query_ids [Q],
    unit_bounds [n_units + 1] (int32), workspace (uint8), positions_out int32
    (room for the allowance).  Returns B, the number of positions written."""
    n = I32()
    dt = KVR_BF16 if embed.dtype == torch.bfloat16 else KVR_F32
    _check(lib.kvr_sur_select(_ptr(embed), embed.shape[0], embed.shape[1], dt, _ptr(suffix_ids), suffix_ids.numel(),
                              suffix_start, _ptr(query_ids), query_ids.numel(), _ptr(unit_bounds),
                              unit_bounds.numel() - 1, budget_percent, _ptr(workspace), workspace.numel(),
                              _ptr(positions_out), C.byref(n), _ptr(scores_out), _stream(stream)), "kvr_sur_select")
    return n.value


def kvr_sur_status(workspace, stream=None):
    _check(lib.kvr_sur_status(_ptr(workspace), _stream(stream)), "kvr_sur_status")


# ---------------------------------------------------------------- paged cache
_PAGE_FORMATS = {"f32": KVR_F32, "bf16": KVR_BF16, "int4": KVR_INT4}
_ROW_DTYPES = {KVR_F32: torch.float32, KVR_BF16: torch.bfloat16, KVR_INT4: torch.bfloat16}


def _want(t, what: str, dtype, dims: int = 0, device=None):
    """The binding's own check of a tensor argument: a wrong dtype, a host
    tensor or one of another device would reach the kernels as a bare pointer."""
    if t.dtype != dtype or not t.is_cuda or (dims and t.dim() != dims) or (device is not None and t.device != device):
        raise ValueError(f"{what}: need a {dims or 'n'}-d {dtype} tensor on {device or 'the GPU'}, got a "
                         f"{t.dim()}-d {t.dtype} tensor on {t.device}")
    return t


def _int_array(t, what: str, n: Optional[int] = None, device=None):
    _want(t, what, torch.int32, device=device)
    if not t.is_contiguous() or (n is not None and t.numel() < n):
        raise ValueError(f"{what}: need a contiguous int32 tensor of at least {n} elements")
    return t


def pages(fmt: str, k, v, page_table, kv_len, err, n_kv_heads: int, page_size: int, layout: str = "hnd",
          k_scale=None, v_scale=None, group: int = 0, strides=None, n_pages: Optional[int] = None) -> kvr_pages:
    """kvr_pages of device tensors.  fmt: "f32", "bf16" or "int4".  k, v:
    [n_pages, n_kv_heads, page_size, head_dim] ("hnd") or [n_pages, page_size,
    n_kv_heads, head_dim] ("nhd"), contiguous; int4: uint8 of 64 bytes a row
    and fp16 k_scale, v_scale [..., 128 / group, 2].  page_table: int32
    [batch, max_pages]; kv_len: int32 [batch]; err: int32 [4], zeroed.
    strides (page, head, slot, in rows) with n_pages describe another layout
    of the same buffers, e.g. a kvr_cache's.  The tensors are kept alive by
    the struct."""
    f = _PAGE_FORMATS[fmt]
    dt = torch.uint8 if f == KVR_INT4 else _ROW_DTYPES[f]
    dev = _want(k, "k", dt).device
    _want(v, "v", dt, device=dev)
    if not k.is_contiguous() or not v.is_contiguous() or k.shape != v.shape:
        raise ValueError("k and v: need contiguous tensors of one shape")
    head_dim = 128 if f == KVR_INT4 else k.shape[-1]
    if f == KVR_INT4 and k.shape[-1] != 64:
        raise ValueError("k and v: 4-bit rows are 64 bytes")
    if strides is None:
        want = (n_kv_heads, page_size) if layout == "hnd" else (page_size, n_kv_heads)
        if layout not in ("hnd", "nhd") or k.dim() != 4 or tuple(k.shape[1:3]) != want:
            raise ValueError(f"k and v: shape {tuple(k.shape)} is not the {layout} layout of {n_kv_heads} heads and "
                             f"{page_size} slots")
        strides = (n_kv_heads * page_size, page_size, 1) if layout == "hnd" else (n_kv_heads * page_size, 1, n_kv_heads)
        n_pages = k.shape[0]
    elif n_pages is None or n_pages < 1 or (n_pages - 1) * strides[0] + (n_kv_heads - 1) * strides[1] + (
            page_size - 1) * strides[2] >= k.numel() // k.shape[-1]:
        raise ValueError("strides: the last page's rows lie outside k and v")
    if f == KVR_INT4:
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if not _want(t, what, torch.float16, device=dev).is_contiguous() or group not in (32, 64, 128) or \
                    t.numel() * group != k.numel() * 4:
                raise ValueError(f"{what}: need contiguous (scale, offset) pairs of every {group} dims of k and v")
    if page_table.dim() != 2:
        raise ValueError("page_table: need [batch, max_pages]")
    batch, max_pages = page_table.shape
    _int_array(page_table, "page_table", device=dev)
    _int_array(kv_len, "kv_len", batch, device=dev)
    _int_array(err, "err", 4, device=dev)
    p = kvr_pages(f, n_kv_heads, head_dim, page_size, group, n_pages, batch, max_pages, *strides, _ptr(k), _ptr(v),
                  _ptr(k_scale), _ptr(v_scale), _ptr(page_table), _ptr(kv_len), _ptr(err))
    p.tensors = (k, v, k_scale, v_scale, page_table, kv_len, err)
    p.device = dev
    p.row_dtype = _ROW_DTYPES[f]
    p.addr = C.addressof(p)
    return p


def score_opts(scale: float = 0.0, softcap: float = 0.0, alpha: float = 0.0, beta: float = 0.0, local_bits=None,
               sink_bits=None, slopes=None, key_begin=None, key_end=None) -> kvr_score_opts:
    """kvr_score_opts of device tensors (kept alive by the struct).  The bit
    masks are int32 tensors of the same words."""
    for t, what in ((local_bits, "local_bits"), (sink_bits, "sink_bits"), (key_begin, "key_begin"),
                    (key_end, "key_end")):
        if t is not None:
            _int_array(t, what)
    if slopes is not None and not _want(slopes, "slopes", torch.float32).is_contiguous():
        raise ValueError("slopes: need a contiguous tensor")
    o = kvr_score_opts(scale, softcap, alpha, beta, _ptr(local_bits), _ptr(sink_bits), _ptr(slopes), _ptr(key_begin),
                       _ptr(key_end))
    o.tensors = (local_bits, sink_bits, slopes, key_begin, key_end)
    o.given = [(what, None, None) if t is None else (what, t.numel(), t.device) for t, what in
               zip(o.tensors, ("local_bits", "sink_bits", "slopes", "key_begin", "key_end"))]
    o.addr = C.addressof(o)
    return o


def _packed_rows(p: kvr_pages, t, what: str, n: int):
    """(pointer, row stride in elements, heads) of a [rows, heads, head_dim] operand."""
    dh = p.head_dim
    try:
        rows, heads, d = t.shape
        s0, s1, s2 = t.stride()
    except ValueError:
        rows = -1
    if rows < n or d != dh or s2 != 1 or (s1 != dh and heads > 1) or (s0 < heads * dh and rows > 1) or \
            t.dtype is not p.row_dtype or t.device != p.device:
        raise ValueError(f"{what}: need [{n}, heads, {dh}] of {p.row_dtype} on {p.device}, a row's heads contiguous; "
                         f"got {tuple(t.shape)} strides {t.stride()} of {t.dtype} on {t.device}")
    # the stride of a single row is whatever torch says; the library wants a full one
    return t.data_ptr(), s0 if s0 > heads * dh else heads * dh, heads


def _rows(p: kvr_pages, cu_rows, positions):
    """(n_rows, the two pointers)"""
    if positions.dtype is not torch.int32 or not positions.is_contiguous() or positions.device != p.device:
        _int_array(positions, "positions", None, p.device)
    if cu_rows.dtype is not torch.int32 or not cu_rows.is_contiguous() or cu_rows.device != p.device or \
            cu_rows.numel() <= p.batch:
        _int_array(cu_rows, "cu_rows", p.batch + 1, p.device)
    return positions.numel(), cu_rows.data_ptr(), positions.data_ptr()


def _paged_stream(p: kvr_pages, stream) -> int:
    # a launch goes to the current device, whichever device the pointers are of
    if torch._C._cuda_getDevice() != p.device.index:
        raise ValueError(f"pages on {p.device}: make it the current device")
    return torch._C._cuda_getCurrentRawStream(p.device.index) if stream is None else _stream(stream)


def kvr_paged_append(p: kvr_pages, cu_rows, positions, k_rows, v_rows, rope=None, q_rows=None, q_out=None,
                     stream=None):
    """k_rows, v_rows: [n_rows, n_kv_heads, head_dim]; rope: fp32 [rope_len,
    head_dim / 2, 2] (cos, sin) or None; q_rows, q_out: [n_rows, n_q_heads,
    head_dim] (q_out packed) or None."""
    n, cu, pos = _rows(p, cu_rows, positions)
    kp, ks, kh = _packed_rows(p, k_rows, "k_rows", n)
    vp, vs, vh = _packed_rows(p, v_rows, "v_rows", n)
    if kh != p.n_kv_heads or vh != p.n_kv_heads:
        raise ValueError(f"k_rows, v_rows: need {p.n_kv_heads} heads")
    qp, qs, qo, hq = None, 0, None, 0
    if q_rows is not None and q_out is not None:
        qp, qs, hq = _packed_rows(p, q_rows, "q_rows", n)
        qo, _, ho = _packed_rows(p, q_out, "q_out", n)
        if ho != hq or not q_out.is_contiguous():
            raise ValueError("q_out: need a packed tensor of q_rows' heads")
    elif q_rows is not None or q_out is not None:
        raise ValueError("q_rows and q_out go together")
    table, rope_len = None, 0
    if rope is not None:
        if rope.dtype is not torch.float32 or not rope.is_contiguous() or rope.device != p.device or \
                rope.shape[1:] != (p.head_dim // 2, 2):
            raise ValueError(f"rope: need a contiguous fp32 [rope_len, {p.head_dim // 2}, 2] on {p.device}")
        table, rope_len = rope.data_ptr(), rope.shape[0]
    _check(lib.kvr_paged_append(p.addr, n, cu, pos, kp, ks, vp, vs, table, rope_len, qp, qs, qo, hq,
                                _paged_stream(p, stream)), "kvr_paged_append")


def kvr_paged_read(p: kvr_pages, cu_rows, positions, k_out=None, v_out=None, stream=None):
    """k_out, v_out: [n_rows, n_kv_heads, head_dim] in the row type, or None."""
    n, cu, pos = _rows(p, cu_rows, positions)
    args = []
    for t, what in ((k_out, "k_out"), (v_out, "v_out")):
        ptr, stride, heads = (None, 0, p.n_kv_heads) if t is None else _packed_rows(p, t, what, n)
        if heads != p.n_kv_heads:
            raise ValueError(f"{what}: need {p.n_kv_heads} heads")
        args += (ptr, stride)
    _check(lib.kvr_paged_read(p.addr, n, cu, pos, *args, _paged_stream(p, stream)), "kvr_paged_read")


def kvr_paged_workspace_bytes(p: kvr_pages, n_q_heads: int, n_rows: int, max_rows: int) -> int:
    return int(lib.kvr_paged_workspace_bytes(C.byref(p), n_q_heads, n_rows, max_rows))


def kvr_paged_attend(p: kvr_pages, opts: Optional[kvr_score_opts], max_rows: int, cu_rows, positions, q, out,
                     workspace, stream=None):
    """q, out: [n_rows, n_q_heads, head_dim]; workspace: uint8 of
    kvr_paged_workspace_bytes; opts: score_opts(...) or None."""
    n, cu, pos = _rows(p, cu_rows, positions)
    qp, qs, hq = _packed_rows(p, q, "q", n)
    op, os_, ho = _packed_rows(p, out, "out", n)
    if ho != hq:
        raise ValueError("out: need q's heads")
    if opts is not None:
        words = -(-p.max_pages * p.page_size // 32) * p.batch
        for (what, numel, device), need in zip(opts.given, (words, words, hq, n, n)):
            if numel is not None and (numel < need or device != p.device):
                raise ValueError(f"{what}: need {need} elements on {p.device}")
    if workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.device != p.device:
        _want(workspace, "workspace", torch.uint8, 1, p.device)
    _check(lib.kvr_paged_attend(p.addr, None if opts is None else opts.addr, hq, n, max_rows, cu, pos, qp, qs, op, os_,
                                workspace.data_ptr(), workspace.numel(), _paged_stream(p, stream)),
           "kvr_paged_attend")


def kvr_paged_status(p: kvr_pages, stream=None):
    _check(lib.kvr_paged_status(C.byref(p), _paged_stream(p, stream)), "kvr_paged_status")
