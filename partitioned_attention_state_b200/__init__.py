"""Partitioned attention-state reuse on B200 (sm_100a): Python binding of libdt.

This module only marshals arguments to the C ABI declared in ``include/dt.h``
(same function names).  Every step of the path runs in libdt: the host plan
builder and the CUDA kernels.  There is no fallback: if the library is
missing, every call raises.

Tensors are torch tensors for device memory (``torch.cuda`` streams are passed
through as raw ``cudaStream_t``); plans and stamps are numpy arrays (host).
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np

__all__ = [
    "DtError", "PlanParams", "Plan", "lib_path", "load", "dt_status_string",
    "dt_plan_geometry", "dt_plan_build", "dt_attn_partial_fused", "dt_attn_partial_fused_heads", "dt_state_merge",
    "dt_state_cache_update", "dt_group_compose", "dt_window_residual", "dt_set_wait_limit_ns",
    "DT_OK", "DT_ERR_INVALID", "DT_ERR_UNSUPPORTED", "DT_ERR_CACHE_EMPTY", "DT_ERR_CUDA",
    "DT_ERR_TIMEOUT", "DT_MODE_ALL_COMPUTE", "DT_MODE_PROXIMITY", "DT_MODE_ALL_REUSE",
    "DT_MODE_EXPLICIT", "DT_MODE_WINDOW", "DT_PLAN_REUSE", "DT_PLAN_COMPUTE", "DT_WR_MAKE",
    "DT_WR_APPLY", "DT_TILE", "DT_STATE_F32", "DT_STATE_BF16", "DT_MODE_IMPORTANCE",
    "dt_plan_build_importance", "dt_state_importance", "dt_share_output", "dt_key_set_tiles",
    "dt_attn_cfg_shared", "dt_plan_share_counts", "DT_SHARE_CFG", "DT_SHARE_TIMESTEP",
    "DT_MODE_ANCHOR", "AnchorState", "dt_anchor_init", "dt_plan_build_anchor", "dt_anchor_update",
    "dt_attn_partial_fused_tracked", "DT_TYPE_BF16", "DT_TYPE_F16", "DT_TYPE_F32", "DT_ROPE_INTERLEAVED",
    "DT_ROPE_HALVES", "Strides", "RopeParams", "NormRopeParams", "SelectParams", "SparseParams", "rope_params",
    "norm_rope_params", "select_params", "sparse_params", "dt_rope_table", "dt_qk_norm_rope", "dt_block_select",
    "dt_attn_block_sparse",
]

DT_OK, DT_ERR_INVALID, DT_ERR_UNSUPPORTED, DT_ERR_CACHE_EMPTY, DT_ERR_CUDA, DT_ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
DT_MODE_IMPORTANCE = 5
DT_MODE_ANCHOR = 6
DT_STATE_F32, DT_STATE_BF16 = 0, 1
DT_MODE_ALL_COMPUTE, DT_MODE_PROXIMITY, DT_MODE_ALL_REUSE, DT_MODE_EXPLICIT, DT_MODE_WINDOW = 0, 1, 2, 3, 4
DT_PLAN_REUSE, DT_PLAN_COMPUTE = 0, 1
DT_WR_MAKE, DT_WR_APPLY = 0, 1
DT_SHARE_CFG, DT_SHARE_TIMESTEP = 0, 1
DT_TILE = 128
DT_TYPE_BF16, DT_TYPE_F16, DT_TYPE_F32 = 0, 1, 2
DT_ROPE_INTERLEAVED, DT_ROPE_HALVES = 0, 1
DT_ROPE_MAX_AXES = 4


class DtError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dt_status_string(status)} ({status})")


class PlanParams(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("S", ctypes.c_int32), ("D", ctypes.c_int32), ("P", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("reuse_per_row", ctypes.c_int32), ("window", ctypes.c_int32),
                ("step", ctypes.c_int32), ("group", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("plan", ctypes.POINTER(ctypes.c_uint8)), ("stamps", ctypes.POINTER(ctypes.c_int32)),
                ("computed_blocks", ctypes.c_int64), ("skipped_blocks", ctypes.c_int64),
                ("computed_flops", ctypes.c_int64), ("nqt", ctypes.c_int32), ("nseg", ctypes.c_int32)]


class AnchorState(ctypes.Structure):
    """dt_anchor_state: the host arrays are numpy buffers kept alive by the
    Python object (see new_anchor_state)."""
    _fields_ = [("weights", ctypes.POINTER(ctypes.c_float)), ("alpha", ctypes.POINTER(ctypes.c_float)),
                ("drift", ctypes.POINTER(ctypes.c_float)), ("eps", ctypes.c_float), ("theta", ctypes.c_float),
                ("target_ratio", ctypes.c_float), ("last_anchor", ctypes.c_int32), ("anchored", ctypes.c_int32)]


class Strides(ctypes.Structure):
    """dt_strides: element strides of the heads and rows of a [head][row][D] tensor."""
    _fields_ = [("head", ctypes.c_int64), ("row", ctypes.c_int64)]


class RopeParams(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("dim", ctypes.c_int32 * DT_ROPE_MAX_AXES),
                ("base", ctypes.c_double)]


class NormRopeParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "D", "H", "Hkv", "rot", "pairing", "in_type", "out_type", "norm",
                                              "q_block", "k_block")] + [("eps", ctypes.c_float)] + \
               [(n, Strides) for n in ("q_in", "k_in", "v_in", "q_out", "k_out", "v_out")]


class SelectParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("H", "Hkv", "nq", "nk", "D", "topk", "keep_first", "keep_last")] + \
               [("margin", ctypes.c_double)]


class SparseParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("H", "Hkv", "Sq", "Sk", "D", "k_block", "cap", "type", "out_type")] + \
               [(n, Strides) for n in ("q", "k", "v", "o")]


# the two structures above as packed fields
_NORM_ROPE, _SPARSE = struct.Struct("@11if12q"), struct.Struct("@9i8q")


_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB: Optional[ctypes.CDLL] = None


def lib_path() -> str:
    return os.path.join(_HERE, "libdt.so")


def load() -> ctypes.CDLL:
    """Load libdt.so from this package directory (raises if it is missing)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libdt.so not built ({path}); run python -m partitioned_attention_state_b200.build")
        lib = ctypes.CDLL(path)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        pp = ctypes.POINTER(PlanParams)
        sig = {
            "dt_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "dt_plan_geometry": ([pp, ctypes.POINTER(i32), ctypes.POINTER(i32)], ctypes.c_int),
            "dt_plan_build": ([pp, vp, ctypes.POINTER(Plan)], ctypes.c_int),
            "dt_attn_partial_fused": ([pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "dt_attn_partial_fused_heads": ([pp, i32, i32] + [vp] * 12, ctypes.c_int),
            "dt_state_merge": ([i32, i32, i32, i32, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "dt_state_cache_update": ([pp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "dt_window_residual": ([i32, i32, i32, i32, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "dt_group_compose": ([pp, i32, vp, vp, vp, vp, vp], ctypes.c_int),
            "dt_plan_build_importance": ([pp, vp, ctypes.POINTER(Plan)], ctypes.c_int),
            "dt_state_importance": ([pp, vp, vp, vp, vp, vp], ctypes.c_int),
            "dt_share_output": ([i32, i32, i32, vp, vp, vp, vp, vp], ctypes.c_int),
            "dt_attn_cfg_shared": ([pp] + [vp] * 12, ctypes.c_int),
            "dt_plan_share_counts": ([pp, i32, ctypes.POINTER(Plan)], ctypes.c_int),
            "dt_anchor_init": ([pp, ctypes.POINTER(AnchorState)], ctypes.c_int),
            "dt_plan_build_anchor": ([pp, ctypes.POINTER(AnchorState), ctypes.POINTER(Plan)], ctypes.c_int),
            "dt_anchor_update": ([pp, ctypes.POINTER(AnchorState), vp, vp, vp, vp], ctypes.c_int),
            "dt_attn_partial_fused_tracked": ([pp] + [vp] * 11 + [i32, vp], ctypes.c_int),
            "dt_key_set_tiles": ([pp, i32, i32, vp, vp, i32], ctypes.c_int),
            "dt_rope_table": ([ctypes.POINTER(RopeParams), vp, vp, vp], ctypes.c_int),
            "dt_qk_norm_rope": ([ctypes.POINTER(NormRopeParams)] + [vp] * 12, ctypes.c_int),
            "dt_block_select": ([ctypes.POINTER(SelectParams)] + [vp] * 5, ctypes.c_int),
            "dt_attn_block_sparse": ([ctypes.POINTER(SparseParams)] + [vp] * 9, ctypes.c_int),
            "dt_set_wait_limit_ns": ([i64], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, res
        _LIB = lib
    return _LIB


def _check(status: int, where: str) -> None:
    if status != DT_OK:
        raise DtError(status, where)


def _ptr(t) -> Optional[int]:
    """Device/host address of a torch tensor or numpy array (None passes NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def dt_status_string(status: int) -> str:
    return load().dt_status_string(status).decode()


def params(H, S, D, P=1, mode=DT_MODE_ALL_COMPUTE, reuse_per_row=0, window=0, step=1, group=0,
           state_dtype=0) -> PlanParams:
    return PlanParams(H, S, D, P, mode, reuse_per_row, window, step, group, state_dtype)


def dt_plan_geometry(p: PlanParams):
    nqt, nseg = ctypes.c_int32(), ctypes.c_int32()
    _check(load().dt_plan_geometry(ctypes.byref(p), ctypes.byref(nqt), ctypes.byref(nseg)), "dt_plan_geometry")
    return nqt.value, nseg.value


def dt_plan_build(p: PlanParams, stamps: Optional[np.ndarray] = None, explicit: Optional[np.ndarray] = None):
    """Host plan of one step.  Returns (plan uint8 [nqt][nseg], counts dict);
    ``stamps`` (int32 [nqt][nseg]) is updated in place when given."""
    nqt, nseg = dt_plan_geometry(p)
    plan = np.zeros((nqt, nseg), dtype=np.uint8)
    out = Plan()
    out.plan = plan.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8))
    if stamps is not None:
        assert stamps.dtype == np.int32 and stamps.flags.c_contiguous and stamps.size == nqt * nseg
        out.stamps = stamps.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    ex = None
    if explicit is not None:
        ex = np.ascontiguousarray(explicit, dtype=np.uint8)
    _check(load().dt_plan_build(ctypes.byref(p), _ptr(ex), ctypes.byref(out)), "dt_plan_build")
    return plan, {"computed_blocks": out.computed_blocks, "skipped_blocks": out.skipped_blocks,
                  "computed_flops": out.computed_flops}


def dt_plan_build_importance(p: PlanParams, weights: Optional[np.ndarray], stamps: Optional[np.ndarray] = None):
    """Importance plan of one step (p.mode = DT_MODE_IMPORTANCE).  weights:
    float32 [nqt][nseg] (host).  Returns (plan, counts) like dt_plan_build;
    ``stamps`` is updated in place when given."""
    nqt, nseg = dt_plan_geometry(p)
    plan = np.zeros((nqt, nseg), dtype=np.uint8)
    out = Plan()
    out.plan = plan.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8))
    if stamps is not None:
        assert stamps.dtype == np.int32 and stamps.flags.c_contiguous and stamps.size == nqt * nseg
        out.stamps = stamps.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    w = None
    if weights is not None:
        w = np.ascontiguousarray(weights, dtype=np.float32)
        assert w.size == nqt * nseg
    _check(load().dt_plan_build_importance(ctypes.byref(p), _ptr(w), ctypes.byref(out)), "dt_plan_build_importance")
    return plan, {"computed_blocks": out.computed_blocks, "skipped_blocks": out.skipped_blocks,
                  "computed_flops": out.computed_flops}


def dt_state_importance(p: PlanParams, cache_L, L, d_weights, d_status=None, stream=None) -> None:
    _check(load().dt_state_importance(ctypes.byref(p), _ptr(cache_L), _ptr(L), _ptr(d_weights), _ptr(d_status),
                                      _stream(stream)), "dt_state_importance")


def dt_key_set_tiles(p: PlanParams, qt: int, k: int):
    """Key tiles of key set k of query tile qt: list of (row0, rowend) with
    the tile's rows [row0, min(row0 + 128, rowend))."""
    n = load().dt_key_set_tiles(ctypes.byref(p), qt, k, None, None, 0)
    if n < 0:
        raise DtError(n, "dt_key_set_tiles")
    r0 = np.zeros(max(n, 1), np.int32)
    re = np.zeros(max(n, 1), np.int32)
    load().dt_key_set_tiles(ctypes.byref(p), qt, k, r0.ctypes.data, re.ctypes.data, n)
    return list(zip(r0[:n].tolist(), re[:n].tolist()))


def dt_share_output(n_heads: int, S: int, D: int, src_O, src_L, dst_O, dst_L, stream=None) -> None:
    _check(load().dt_share_output(n_heads, S, D, _ptr(src_O), _ptr(src_L), _ptr(dst_O), _ptr(dst_L),
                                  _stream(stream)), "dt_share_output")


def dt_attn_cfg_shared(p: PlanParams, d_plan, Q, K, V, cache_O, cache_L, R, O, L, d_counters, d_status,
                       stream=None) -> None:
    _check(load().dt_attn_cfg_shared(ctypes.byref(p), _ptr(d_plan), _ptr(Q), _ptr(K), _ptr(V), _ptr(cache_O),
                                     _ptr(cache_L), _ptr(R), _ptr(O), _ptr(L), _ptr(d_counters), _ptr(d_status),
                                     _stream(stream)), "dt_attn_cfg_shared")


def dt_plan_share_counts(p: PlanParams, kind: int, counts: Optional[dict] = None) -> dict:
    """Counts of a step under attention sharing (DT_SHARE_CFG: from the
    counts of the step's plan over all heads; DT_SHARE_TIMESTEP: nothing
    computed)."""
    io = Plan()
    if counts is not None:
        io.computed_blocks = counts["computed_blocks"]
        io.skipped_blocks = counts["skipped_blocks"]
        io.computed_flops = counts["computed_flops"]
    _check(load().dt_plan_share_counts(ctypes.byref(p), kind, ctypes.byref(io)), "dt_plan_share_counts")
    return {"computed_blocks": io.computed_blocks, "skipped_blocks": io.skipped_blocks,
            "computed_flops": io.computed_flops}


def new_anchor_state(p: PlanParams, target_ratio: float, theta: float):
    """A dt_anchor_state with its host arrays, initialised by dt_anchor_init.
    Returns (state, arrays) where arrays = {"weights", "alpha", "drift"} are
    the numpy views the state points into (keep them alive)."""
    nqt, nseg = dt_plan_geometry(p)
    arr = {"weights": np.zeros((max(nqt, 1), nseg), np.float32), "alpha": np.zeros((max(nqt, 1), nseg), np.float32),
           "drift": np.zeros(max(nqt, 1), np.float32)}
    fp = ctypes.POINTER(ctypes.c_float)
    st = AnchorState(arr["weights"].ctypes.data_as(fp), arr["alpha"].ctypes.data_as(fp),
                     arr["drift"].ctypes.data_as(fp), 0.0, theta, target_ratio, 0, 0)
    dt_anchor_init(p, st)
    return st, arr


def dt_anchor_init(p: PlanParams, st: AnchorState) -> None:
    _check(load().dt_anchor_init(ctypes.byref(p), ctypes.byref(st)), "dt_anchor_init")


def dt_plan_build_anchor(p: PlanParams, st: AnchorState, stamps: Optional[np.ndarray] = None):
    """Anchor-guided plan of one step (p.mode = DT_MODE_ANCHOR).  Returns
    (plan, counts, anchored); ``stamps`` is updated in place when given."""
    nqt, nseg = dt_plan_geometry(p)
    plan = np.zeros((nqt, nseg), dtype=np.uint8)
    out = Plan()
    out.plan = plan.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8))
    if stamps is not None:
        assert stamps.dtype == np.int32 and stamps.flags.c_contiguous and stamps.size == nqt * nseg
        out.stamps = stamps.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    _check(load().dt_plan_build_anchor(ctypes.byref(p), ctypes.byref(st), ctypes.byref(out)), "dt_plan_build_anchor")
    return plan, {"computed_blocks": out.computed_blocks, "skipped_blocks": out.skipped_blocks,
                  "computed_flops": out.computed_flops}, bool(st.anchored)


def dt_anchor_update(p: PlanParams, st: AnchorState, stamps_before: np.ndarray, plan: np.ndarray, err: np.ndarray,
                     weights_now: Optional[np.ndarray] = None) -> None:
    sb = np.ascontiguousarray(stamps_before, dtype=np.int32)
    pl = np.ascontiguousarray(plan, dtype=np.uint8)
    e = np.ascontiguousarray(err, dtype=np.float32)
    w = None if weights_now is None else np.ascontiguousarray(weights_now, dtype=np.float32)
    _check(load().dt_anchor_update(ctypes.byref(p), ctypes.byref(st), _ptr(sb), _ptr(pl), _ptr(e), _ptr(w)),
           "dt_anchor_update")


def dt_attn_partial_fused_tracked(p: PlanParams, d_plan, Q, K, V, cache_O, cache_L, O, L, d_counters, d_status,
                                  d_err, err_all: bool, stream=None) -> None:
    _check(load().dt_attn_partial_fused_tracked(ctypes.byref(p), _ptr(d_plan), _ptr(Q), _ptr(K), _ptr(V),
                                                _ptr(cache_O), _ptr(cache_L), _ptr(O), _ptr(L), _ptr(d_counters),
                                                _ptr(d_status), _ptr(d_err), 1 if err_all else 0, _stream(stream)),
           "dt_attn_partial_fused_tracked")


def dt_attn_partial_fused(p: PlanParams, d_plan, Q, K, V, cache_O, cache_L, R, O, L, d_counters, d_status,
                          stream=None) -> None:
    _check(load().dt_attn_partial_fused(ctypes.byref(p), _ptr(d_plan), _ptr(Q), _ptr(K), _ptr(V), _ptr(cache_O),
                                        _ptr(cache_L), _ptr(R), _ptr(O), _ptr(L), _ptr(d_counters),
                                        _ptr(d_status), _stream(stream)), "dt_attn_partial_fused")


def dt_attn_partial_fused_heads(p: PlanParams, head_begin: int, head_count: int, d_plan, Q, K, V, cache_O, cache_L,
                                R, O, L, d_counters, d_status, stream=None) -> None:
    _check(load().dt_attn_partial_fused_heads(ctypes.byref(p), head_begin, head_count, _ptr(d_plan), _ptr(Q), _ptr(K),
                                              _ptr(V), _ptr(cache_O), _ptr(cache_L), _ptr(R), _ptr(O), _ptr(L),
                                              _ptr(d_counters), _ptr(d_status), _stream(stream)),
           "dt_attn_partial_fused_heads")


def dt_group_compose(p: PlanParams, factor: int, stamps: Optional[np.ndarray], cache_O, cache_L, d_status=None,
                     stream=None) -> Optional[np.ndarray]:
    """Regroup the cached states of layout p (p.group = g) into group size
    g * factor in place.  ``stamps`` (int32 [nqt][1+m], host) is rewritten in
    place; the returned view is its new [nqt][1+m'] shape (None if None)."""
    if stamps is not None:
        assert stamps.dtype == np.int32 and stamps.flags.c_contiguous
    _check(load().dt_group_compose(ctypes.byref(p), factor, _ptr(stamps), _ptr(cache_O), _ptr(cache_L),
                                   _ptr(d_status), _stream(stream)), "dt_group_compose")
    if stamps is None:
        return None
    nqt = stamps.shape[0]
    m = -(-p.P // p.group)
    m2 = -(-m // factor)
    return stamps.reshape(-1)[: nqt * (1 + m2)].reshape(nqt, 1 + m2)


def dt_state_merge(N, H, S, D, O_in, L_in, O_out, L_out, d_status=None, stream=None) -> None:
    _check(load().dt_state_merge(N, H, S, D, _ptr(O_in), _ptr(L_in), _ptr(O_out), _ptr(L_out), _ptr(d_status),
                                 _stream(stream)), "dt_state_merge")


def dt_state_cache_update(p: PlanParams, d_plan, fresh_O, fresh_L, cache_O, cache_L, d_status=None,
                          stream=None) -> None:
    _check(load().dt_state_cache_update(ctypes.byref(p), _ptr(d_plan), _ptr(fresh_O), _ptr(fresh_L),
                                        _ptr(cache_O), _ptr(cache_L), _ptr(d_status), _stream(stream)),
           "dt_state_cache_update")


def dt_window_residual(op, H, S, D, O_full, O_win, R, O, d_status=None, stream=None) -> None:
    _check(load().dt_window_residual(op, H, S, D, _ptr(O_full), _ptr(O_win), _ptr(R), _ptr(O), _ptr(d_status),
                                     _stream(stream)), "dt_window_residual")


# ---- block-sparse attention and the passes in front of it -------------------
# These take torch tensors, check them against the parameters (a wrong size
# would be read or written out of bounds on the device) and run on the tensors'
# device: on `stream` where given, else on that device's current stream.

_TYPES: dict = {}           # torch element type -> DT_TYPE_*, and back; filled with _torch by _init
_torch = None


def _init():
    """torch, imported on the first call that takes tensors."""
    global _torch
    if _torch is None:
        import torch
        for code, ty in ((DT_TYPE_BF16, torch.bfloat16), (DT_TYPE_F16, torch.float16), (DT_TYPE_F32, torch.float32)):
            _TYPES[ty], _TYPES[code] = code, ty
        _torch = torch
    return _torch


def _type_of(t) -> int:
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported element type {t.dtype}") from None


def _heads(t, name: str):
    """(head, row) strides of a [heads][rows][D] tensor or view whose rows are contiguous; (0, 0) for None."""
    if t is None:
        return 0, 0
    st = t.stride()
    if len(st) != 3 or (st[2] != 1 and t.shape[2] > 1):
        raise ValueError(f"{name}: expected [heads][rows][D] with contiguous rows, got {tuple(t.shape)} "
                         f"with strides {st}")
    return st[:2]


# The two checks below run for every tensor of every call: they return its address (None for None) and look closer
# only where the plain comparison fails.
def _flat(t, shape, dtype, name: str, device: int):
    """Address of t; raises unless t is a contiguous tensor of this shape and type on this device."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {shape} on device {device}, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()} on device {t.get_device()}")
    return t.data_ptr()


def _strided(t, shape, strides, dtype, name: str, device: int):
    """Address of t; raises unless t is the [heads][rows][D] tensor that the parameters were made for."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.get_device() == device:
        head, row, col = t.stride()
        if (col == 1 or shape[2] <= 1) and (row == strides.row or shape[1] <= 1) and \
                (head == strides.head or shape[0] <= 1):
            return t.data_ptr()
    raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} with strides {t.stride()} on device {t.get_device()} is "
                     f"not what the parameters describe: {dtype} {shape}, head stride {strides.head}, row stride "
                     f"{strides.row}, on device {device}")


def _call(name: str, device: int, stream, p, *args) -> None:
    """One C call with the tensors' device current (launches go to the current device)."""
    if device < 0:
        raise ValueError(f"{name}: expected CUDA tensors")
    f = getattr(_LIB or load(), name)
    if stream is None:          # the raw handle of the device's current stream, without a Stream object
        raw = _torch._C._cuda_getCurrentRawStream(device)
    else:
        raw = getattr(stream, "cuda_stream", stream)
    if device == _torch.cuda.current_device():
        status = f(ctypes.byref(p), *args, raw)
    else:
        with _torch.cuda.device(device):
            status = f(ctypes.byref(p), *args, raw)
    if status != DT_OK:
        raise DtError(status, name)


def rope_params(S: int, axes, base: float = 10000.0) -> RopeParams:
    """Rotation of S tokens over position axes; axes: rotated dimensions of each."""
    axes = list(axes)
    if not 1 <= len(axes) <= DT_ROPE_MAX_AXES:
        raise ValueError(f"1 to {DT_ROPE_MAX_AXES} axes, got {len(axes)}")
    return RopeParams(S, len(axes), (ctypes.c_int32 * DT_ROPE_MAX_AXES)(*axes), base)


def dt_rope_table(p: RopeParams, pos, table, stream=None) -> None:
    """pos: int32 [axes][S]; table: float32 [S][rot/2][2], written with (cos, sin)."""
    torch, dev, n = _init(), pos.get_device(), p.n_axes
    _call("dt_rope_table", dev, stream, p, _flat(pos, (n, p.S), torch.int32, "pos", dev),
          _flat(table, (p.S, sum(p.dim[:n]) // 2, 2), torch.float32, "table", dev))


def norm_rope_params(q=None, k=None, v=None, Q=None, K=None, V=None, rot: int = 0,
                     pairing: int = DT_ROPE_INTERLEAVED, norm: bool = True, eps: float = 1e-6, q_block: int = DT_TILE,
                     k_block: int = 64) -> NormRopeParams:
    """Parameters of dt_qk_norm_rope for tensors (or views) laid out like these:
    q [H][S][D], k and v [Hkv][S][D] inputs, Q, K, V outputs; a part may be
    None.  x.view(S, heads, D).transpose(0, 1) is a token-major projection."""
    _init()
    first = q if q is not None else k if k is not None else v
    if first is None:
        raise ValueError("no input")
    out = Q if Q is not None else K if K is not None else V
    kv = k if k is not None else v
    _, S, D = first.shape
    ity = _type_of(first)
    # packed in one go: setting the fields one by one costs as much as the launch
    return NormRopeParams.from_buffer_copy(_NORM_ROPE.pack(
        S, D, 0 if q is None else q.shape[0], 0 if kv is None else kv.shape[0], rot, pairing, ity,
        ity if out is None else _type_of(out), int(norm), q_block, k_block, eps, *_heads(q, "q"), *_heads(k, "k"),
        *_heads(v, "v"), *_heads(Q, "Q"), *_heads(K, "K"), *_heads(V, "V")))


def dt_qk_norm_rope(p: NormRopeParams, q, k, v, wq, wk, table, Q, K, V, q_mean=None, k_mean=None, stream=None) -> None:
    """Per-head RMS norm, rotation, layout change and block means in one pass
    (see norm_rope_params).  wq, wk: float32 [D] or None; table: dt_rope_table's,
    None with rot = 0; q_mean, k_mean: float32 [heads][blocks][D] or None."""
    f32 = _init().float32
    first = q if q is not None else k if k is not None else v
    if first is None:
        raise ValueError("no input")
    dev, S, D, rot, qb, kb = first.get_device(), p.S, p.D, p.rot, p.q_block, p.k_block
    qs, ks, ity, oty = (p.H, S, D), (p.Hkv, S, D), _TYPES.get(p.in_type), _TYPES.get(p.out_type)
    _call("dt_qk_norm_rope", dev, stream, p,
          _strided(q, qs, p.q_in, ity, "q", dev), _strided(k, ks, p.k_in, ity, "k", dev),
          _strided(v, ks, p.v_in, ity, "v", dev), _flat(wq, (D,), f32, "wq", dev), _flat(wk, (D,), f32, "wk", dev),
          _flat(table, (S, rot // 2, 2), f32, "table", dev) if rot else None,
          _strided(Q, qs, p.q_out, oty, "Q", dev), _strided(K, ks, p.k_out, oty, "K", dev),
          _strided(V, ks, p.v_out, oty, "V", dev),
          _flat(q_mean, (p.H, -(-S // qb) if qb > 0 else 0, D), f32, "q_mean", dev),
          _flat(k_mean, (p.Hkv, -(-S // kb) if kb > 0 else 0, D), f32, "k_mean", dev))


def select_params(H: int, Hkv: int, nq: int, nk: int, D: int, topk: int, keep_first: int = 0, keep_last: int = 0,
                  margin: float = float("inf")) -> SelectParams:
    return SelectParams(H, Hkv, nq, nk, D, topk, keep_first, keep_last, margin)


def dt_block_select(p: SelectParams, q_mean, k_mean, idx, count, stream=None) -> None:
    """Lists of key blocks by the scores of block means.  q_mean float32
    [H][nq][D], k_mean float32 [Hkv][nk][D]; idx int32 [H][nq][topk] and count
    int32 [H][nq] are written."""
    torch, dev, H, nq, D = _init(), q_mean.get_device(), p.H, p.nq, p.D
    _call("dt_block_select", dev, stream, p, _flat(q_mean, (H, nq, D), torch.float32, "q_mean", dev),
          _flat(k_mean, (p.Hkv, p.nk, D), torch.float32, "k_mean", dev),
          _flat(idx, (H, nq, p.topk), torch.int32, "idx", dev), _flat(count, (H, nq), torch.int32, "count", dev))


def sparse_params(Q, K, V, O, k_block: int = 64, cap: int = 0) -> SparseParams:
    """Parameters of dt_attn_block_sparse for tensors (or views) laid out like
    these: Q, O [H][Sq][D], K, V [Hkv][Sk][D]; cap entries per list."""
    _init()
    H, Sq, D = Q.shape
    Hkv, Sk, _ = K.shape
    return SparseParams.from_buffer_copy(_SPARSE.pack(H, Hkv, Sq, Sk, D, k_block, cap, _type_of(Q), _type_of(O),
                                                      *_heads(Q, "Q"), *_heads(K, "K"), *_heads(V, "V"),
                                                      *_heads(O, "O")))


def dt_attn_block_sparse(p: SparseParams, Q, K, V, idx, count, O, L, d_status, stream=None) -> None:
    """Attention of every 128-row query block over the key blocks of its list:
    the state (O, L).  idx int32 [H][ceil(Sq/128)][cap], count int32
    [H][ceil(Sq/128)] or None (cap entries each), L float32 [H][Sq], d_status
    int32 device status word."""
    torch, dev, H, Sq, D = _init(), Q.get_device(), p.H, p.Sq, p.D
    if d_status.dtype is not torch.int32 or d_status.numel() < 1 or d_status.get_device() != dev:
        raise ValueError("d_status: expected an int32 tensor on the inputs' device")
    qs, ks, ty, nqb = (H, Sq, D), (p.Hkv, p.Sk, D), _TYPES.get(p.type), -(-Sq // DT_TILE)
    _call("dt_attn_block_sparse", dev, stream, p, _strided(Q, qs, p.q, ty, "Q", dev),
          _strided(K, ks, p.k, ty, "K", dev), _strided(V, ks, p.v, ty, "V", dev),
          _flat(idx, (H, nqb, p.cap), torch.int32, "idx", dev), _flat(count, (H, nqb), torch.int32, "count", dev),
          _strided(O, qs, p.o, _TYPES.get(p.out_type), "O", dev), _flat(L, (H, Sq), torch.float32, "L", dev),
          d_status.data_ptr())


def dt_set_wait_limit_ns(ns: int) -> None:
    _check(load().dt_set_wait_limit_ns(int(ns)), "dt_set_wait_limit_ns")
