"""Exact attention forward for GB300 (sm_103a): Python binding of the C ABI.

The binding only marshals arguments to ``libfa_gb300.so`` (``include/fa.h``);
every step of the computation runs in the library's CUDA kernels.  PyTorch is
used for device memory and streams only.  There is no CPU fallback: if the
library is missing or a call fails, an exception is raised.

    from exact_attention_forward_08_gb300 import attention_forward
    o, lse = attention_forward(q, k, v, causal=True)   # q [B,Sq,Hq,d] bf16 on cuda
    o, lse = attention_forward_varlen(q, k, v, cu_q, cu_k)  # q [total_q,Hq,d], cu_q int32 [B+1]
    kv_append(k, v, k_cache, v_cache, k_scale, v_scale, table, lens, cu_q)  # paged 8-bit cache
    o, lse = attention_forward_paged(q, k_cache, v_cache, k_scale, v_scale, table, lens, cu_q, max_seqlen_q)
    table = rotary_table(positions, rot_dim); q, k = rotary(q, k, table)   # dq, dk = rotary_backward(dq, dk, table)
    kv_bounds(k_cache, k_bounds, table, lens, cu_q)                         # sparse attention over selected pages
    lists, list_lens = kv_select(q, k_bounds, k_scale, table, lens, cu_q, max_seqlen_q, page_size, top)
    o, lse = attention_forward_lists(q, k_cache, v_cache, k_scale, v_scale, lists, list_lens)
    table, lens, refs = kv_fork(parents, k_cache, v_cache, k_scale, v_scale, table, lens, refs)  # the cache's pages
    table, refs, page_map, used = kv_compact(k_cache, v_cache, k_scale, v_scale, table, lens, refs)

Raw entry points with the C names: ``fa_fwd``, ``fa_fwd_ex``, ``fa_fwd_varlen``,
``fa_fwd_varlen_ex``, ``fa_varlen_workspace_size``, ``fa_varlen_plan_host``,
``fa_device_status``, ``fa_status_string``, ``fa_make_plan``, ``fa_plan_task``, ``fa_plan_set_grid``,
``fa_plan_block_masked``, ``fa_plan_first_masked_block``, ``fa_version``, ``fa_kv_append``, ``fa_fwd_paged``,
``fa_fwd_paged_workspace_size``, ``fa_rotary_table``, ``fa_rotary``, ``fa_kv_bounds``, ``fa_kv_select``,
``fa_kv_select_workspace_size``, ``fa_fwd_lists``, ``fa_fwd_lists_workspace_size``, ``fa_kv_fork``, ``fa_kv_compact``,
``fa_kv_pages_workspace_size``.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

from . import _build

__all__ = ["fa_fwd", "fa_fwd_ex", "fa_fwd_varlen", "fa_fwd_varlen_ex", "fa_varlen_workspace_size",
           "fa_varlen_plan_host", "fa_fwd_splitkv", "fa_splitkv_workspace_size", "fa_splitkv_num_splits",
           "attention_forward_splitkv", "fa_bwd", "fa_bwd_workspace_size", "attention_backward",
           "fa_bwd_varlen", "fa_bwd_varlen_workspace_size", "attention_backward_varlen",
           "fa_fwd_varlen_noalloc", "fa_noalloc_scratch_bytes", "fa_device_status", "fa_device_status_code", "fa_status_string", "fa_selftest_exp2", "fa_make_plan",
           "fa_plan_task", "fa_plan_set_grid", "fa_plan_block_masked", "fa_plan_first_masked_block", "fa_version", "FaOptions", "FaPlan",
           "FaTask", "FaVarlenTask", "attention_forward", "attention_forward_varlen", "FaError", "load_library",
           "LIB_PATH", "STATUS", "VARLEN_HEADER_BYTES", "FaKvCache", "fa_kv_append", "fa_fwd_paged",
           "fa_fwd_paged_workspace_size", "kv_append", "attention_forward_paged", "FaRotaryScaling", "ROTARY_SCALING",
           "fa_rotary_table", "fa_rotary", "rotary_table", "rotary", "rotary_backward", "fa_kv_bounds", "fa_kv_select",
           "fa_kv_select_workspace_size", "fa_fwd_lists", "fa_fwd_lists_workspace_size", "kv_bounds", "kv_select",
           "attention_forward_lists", "fa_kv_fork", "fa_kv_compact", "fa_kv_pages_workspace_size", "kv_fork",
           "kv_compact"]

LIB_PATH = _build.LIB
STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_CUDA",
          4: "FA_ERR_DEVICE_TIMEOUT", 5: "FA_ERR_DEVICE_CHECK"}
FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_DEVICE_TIMEOUT, FA_ERR_DEVICE_CHECK = range(6)


class FaError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}" if what else STATUS.get(code, str(code)))


class FaOptions(ctypes.Structure):
    _fields_ = [("tau", ctypes.c_float), ("pack", ctypes.c_int), ("grid", ctypes.c_int),
                ("timeout_s", ctypes.c_double), ("debug_flags", ctypes.c_int), ("exp_emu", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("store_mode", ctypes.c_int), ("no_balance", ctypes.c_int),
                ("trace", ctypes.c_void_p), ("trace_ctas", ctypes.c_int), ("trace_cap", ctypes.c_int),
                ("stagger", ctypes.c_int)]


# bytes of the optional fixed-length scheduling workspace (fa_options.workspace)
SCHED_WORKSPACE_BYTES = 16


class FaPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads_q", "heads_kv", "seqlen_q", "seqlen_k", "causal",
                                            "pack", "groups", "pos_per_tile", "tiles", "mblocks", "kv_blocks",
                                            "ratio", "section_units", "heavy_levels")] + [("num_tasks", ctypes.c_int64),
                                                                                          ("tail_first", ctypes.c_int64),
                                                                                          ("grid", ctypes.c_int)]


class FaTask(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int), ("g", ctypes.c_int), ("mblock", ctypes.c_int), ("kv_head", ctypes.c_int),
                ("pos0", ctypes.c_int * 2), ("n_blocks", ctypes.c_int * 2), ("key_split", ctypes.c_int)]


class FaVarlenTask(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("b", "g", "mblock", "reserved", "q_row0", "seqlen_q", "k_row0",
                                            "seqlen_k")]


class FaKvCache(ctypes.Structure):
    """``fa_kv_cache`` of include/fa.h: pointers as integers, strides in bytes."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "block_table", "seqlens_k")] + \
               [("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3), ("table_stride", ctypes.c_int64)] + \
               [(n, ctypes.c_int) for n in ("num_pages", "page_size", "heads_kv", "d_qk", "d_v", "max_pages")]


class FaRotaryScaling(ctypes.Structure):
    """``fa_rotary_scaling`` of include/fa.h."""
    _fields_ = [("kind", ctypes.c_int)] + [(n, ctypes.c_double) for n in ("factor", "original", "low", "high", "magnitude")]


# names of the kinds of scaling (enum fa_rotary_kind)
ROTARY_SCALING = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}


# a varlen workspace holds the task count at byte 0 and the task records from this offset
VARLEN_HEADER_BYTES = 256

_lib = None

_I = ctypes.c_int
_P = ctypes.c_void_p
_FWD_ARGS = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float]


def load_library(path: str | None = None):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FaError(FA_ERR_CUDA, f"CUDA library not built ({p}); run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    lib.fa_fwd.argtypes = _FWD_ARGS + [_P]
    lib.fa_fwd.restype = _I
    lib.fa_fwd_ex.argtypes = _FWD_ARGS + [ctypes.POINTER(FaOptions), _P]
    lib.fa_fwd_ex.restype = _I
    lib.fa_options_default.argtypes = [ctypes.POINTER(FaOptions)]
    lib.fa_options_default.restype = None
    lib.fa_device_status.argtypes = [_P, ctypes.POINTER(_I)]
    lib.fa_device_status.restype = _I
    lib.fa_device_status_detail.argtypes = [_P, ctypes.POINTER(_I), ctypes.POINTER(ctypes.c_uint)]
    lib.fa_device_status_detail.restype = _I
    lib.fa_debug_rescale_count.argtypes = [_P, ctypes.POINTER(ctypes.c_uint)]
    lib.fa_debug_rescale_count.restype = _I
    lib.fa_status_string.argtypes = [_I]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = _I
    lib.fa_make_plan.argtypes = [_I] * 8 + [ctypes.c_int64, _I, ctypes.POINTER(FaPlan)]
    lib.fa_make_plan.restype = _I
    lib.fa_plan_task.argtypes = [ctypes.POINTER(FaPlan), ctypes.c_int64, ctypes.POINTER(FaTask)]
    lib.fa_plan_task.restype = _I
    lib.fa_plan_set_grid.argtypes = [ctypes.POINTER(FaPlan), _I]
    lib.fa_plan_set_grid.restype = _I
    lib.fa_plan_block_masked.argtypes = [ctypes.POINTER(FaPlan), _I, _I]
    lib.fa_plan_block_masked.restype = _I
    lib.fa_selftest_exp2.argtypes = [_P, _P, _P, _I, _P]
    lib.fa_selftest_exp2.restype = _I
    lib.fa_plan_first_masked_block.argtypes = [ctypes.POINTER(FaPlan), _I]
    lib.fa_plan_first_masked_block.restype = _I
    lib.fa_varlen_workspace_size.argtypes = [_I, _I, ctypes.c_int64]
    lib.fa_varlen_workspace_size.restype = ctypes.c_size_t
    vl = [_P, _P, _P, _P, _P, _P, _P, _I, ctypes.c_int64, ctypes.c_int64, _I, _I, _I, _I, _I, ctypes.c_float, _P,
          ctypes.c_size_t]
    lib.fa_fwd_varlen.argtypes = vl + [_P]
    lib.fa_fwd_varlen.restype = _I
    lib.fa_fwd_varlen_ex.argtypes = vl + [ctypes.POINTER(FaOptions), _P]
    lib.fa_fwd_varlen_ex.restype = _I
    lib.fa_fwd_splitkv.argtypes = _FWD_ARGS + [_I, _P, ctypes.c_size_t, _P]
    lib.fa_fwd_splitkv.restype = _I
    lib.fa_fwd_splitkv_ex.argtypes = _FWD_ARGS + [_I, _P, ctypes.c_size_t, ctypes.POINTER(FaOptions), _P]
    lib.fa_fwd_splitkv_ex.restype = _I
    lib.fa_splitkv_workspace_size.argtypes = [_I] * 5
    lib.fa_splitkv_workspace_size.restype = ctypes.c_size_t
    lib.fa_splitkv_num_splits.argtypes = [_I] * 10
    lib.fa_splitkv_num_splits.restype = _I
    bw = [_P] * 9 + [_I] * 8 + [ctypes.c_float, _P, ctypes.c_size_t]
    lib.fa_bwd.argtypes = bw + [_P]
    lib.fa_bwd.restype = _I
    bvl = [_P] * 11 + [_I, ctypes.c_int64, ctypes.c_int64] + [_I] * 5 + [ctypes.c_float, _P, ctypes.c_size_t]
    lib.fa_bwd_varlen.argtypes = bvl + [_P]
    lib.fa_bwd_varlen.restype = _I
    lib.fa_bwd_varlen_ex.argtypes = bvl + [ctypes.POINTER(FaOptions), _P]
    lib.fa_bwd_varlen_ex.restype = _I
    lib.fa_bwd_varlen_workspace_size.argtypes = [_I, _I, _I, ctypes.c_int64, ctypes.c_int64]
    lib.fa_bwd_varlen_workspace_size.restype = ctypes.c_size_t
    lib.fa_bwd_ex.argtypes = bw + [ctypes.POINTER(FaOptions), _P]
    lib.fa_bwd_ex.restype = _I
    lib.fa_bwd_workspace_size.argtypes = [_I, _I, _I]
    lib.fa_bwd_workspace_size.restype = ctypes.c_size_t
    lib.fa_fwd_varlen_noalloc.argtypes = vl[:16] + [_P]
    lib.fa_fwd_varlen_noalloc.restype = _I
    lib.fa_noalloc_scratch_bytes.argtypes = []
    lib.fa_noalloc_scratch_bytes.restype = ctypes.c_size_t
    lib.fa_varlen_plan_host.argtypes = [_P, _P] + [_I] * 6 + [ctypes.c_int64, _I, ctypes.POINTER(FaVarlenTask),
                                                             ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    lib.fa_varlen_plan_host.restype = _I
    i64 = ctypes.c_int64
    lib.fa_kv_append.argtypes = [_P, _P, _P, _P, i64, i64, i64, _P, _P, _I, i64, _I, _P, _I, _I,
                                 _I, _P]
    lib.fa_kv_append.restype = _I
    lib.fa_fwd_paged.argtypes = [_P, _P, _P, _P, _P, _I, i64, _I, i64, _I, _I, ctypes.c_float, _P,
                                 ctypes.c_size_t, _P]
    lib.fa_fwd_paged.restype = _I
    lib.fa_fwd_paged_workspace_size.argtypes = [_I, _I, _I, i64, _I, i64, _I, _I]
    lib.fa_fwd_paged_workspace_size.restype = ctypes.c_size_t
    lib.fa_rotary_table.argtypes = [_P, _I, _I, ctypes.c_double, ctypes.POINTER(FaRotaryScaling), _P]
    lib.fa_rotary_table.restype = _I
    lib.fa_rotary.argtypes = [_P, _P, _P, _P, i64, i64, i64, i64, _P, _P, _I, i64, i64, _I, _I, _I, _P, _I, _I, _I, _I, _P]
    lib.fa_rotary.restype = _I
    lib.fa_kv_bounds.argtypes = [_P, _P, _P, _I, i64, _P]
    lib.fa_kv_bounds.restype = _I
    lib.fa_kv_select_workspace_size.argtypes = [_I, i64, _I, _I]
    lib.fa_kv_select_workspace_size.restype = ctypes.c_size_t
    lib.fa_kv_select.argtypes = [_P, _P, _P, _P, i64, _P, _P, _I, i64] + [_I] * 11 + [_P, _P, _P, ctypes.c_size_t, _P]
    lib.fa_kv_select.restype = _I
    lib.fa_fwd_lists_workspace_size.argtypes = [_I, _I, _I]
    lib.fa_fwd_lists_workspace_size.restype = ctypes.c_size_t
    lib.fa_fwd_lists.argtypes = [_P, _P, _P, _P, _I, _P, _P, i64, _I, ctypes.c_float, _P, ctypes.c_size_t, _P]
    lib.fa_fwd_lists.restype = _I
    lib.fa_kv_pages_workspace_size.argtypes = [_I, _I, _I]
    lib.fa_kv_pages_workspace_size.restype = ctypes.c_size_t
    lib.fa_kv_fork.argtypes = [_P, _P, _P, _I, _P, _P, _I, _P, i64, _P, _P, _P, ctypes.c_size_t, _P]
    lib.fa_kv_fork.restype = _I
    lib.fa_kv_compact.argtypes = [_P, _P, _P, _I, _P, i64, _P, _P, _P, _P, ctypes.c_size_t, _P]
    lib.fa_kv_compact.restype = _I
    if path is None:
        _lib = lib
    return lib


# ---------------------------------------------------------------------------
# raw C entry points (pointers and sizes)
# ---------------------------------------------------------------------------

def fa_fwd(q, k, v, o, lse, batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, causal, scale, stream) -> int:
    """``fa_fwd`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_fwd(q, k, v, o, lse, batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v,
                                 int(causal), float(scale), stream)


def default_options() -> FaOptions:
    o = FaOptions()
    load_library().fa_options_default(ctypes.byref(o))
    return o


def fa_fwd_ex(q, k, v, o, lse, batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, causal, scale, opts,
              stream) -> int:
    """``fa_fwd_ex``: ``opts`` is an ``FaOptions`` or None."""
    return load_library().fa_fwd_ex(q, k, v, o, lse, batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v,
                                    int(causal), float(scale), ctypes.byref(opts) if opts is not None else None,
                                    stream)


def fa_device_status(stream=None):
    """Synchronise ``stream`` and read/clear the device status through
    ``fa_device_status_detail``: (code, (code, site, block))."""
    out = _I(0)
    detail = (ctypes.c_uint * 3)()
    rc = load_library().fa_device_status_detail(stream, ctypes.byref(out), detail)
    if rc != FA_OK:
        raise FaError(rc, "fa_device_status_detail")
    return out.value, tuple(detail)


def fa_device_status_code(stream=None) -> int:
    """``fa_device_status``: synchronise ``stream``, read and clear the status code."""
    out = _I(0)
    rc = load_library().fa_device_status(stream, ctypes.byref(out))
    if rc != FA_OK:
        raise FaError(rc, "fa_device_status")
    return out.value


# fa_options.debug_flags bits
DEBUG_SKIP_P_ARRIVE = 1
DEBUG_COUNT_RESCALE = 2
DEBUG_CHECKS = 4        # the checking build of the forward kernel
DEBUG_PLANT_BAD_TASK = 8  # with DEBUG_CHECKS: task 0 decodes out of range (the checks must catch it)


def fa_debug_rescale_count(stream=None) -> int:
    """Synchronise ``stream``, read and clear the count of O rescales (forward
    calls made with ``debug_flags`` bit 1): one per warp of 32 rows and K/V
    block whose correction warps rescaled O."""
    out = ctypes.c_uint(0)
    rc = load_library().fa_debug_rescale_count(stream, ctypes.byref(out))
    if rc != FA_OK:
        raise FaError(rc, "fa_debug_rescale_count")
    return int(out.value)


def fa_selftest_exp2(x, y_fma, y_mufu, n, stream) -> int:
    """``fa_selftest_exp2``: device pointers as integers."""
    return load_library().fa_selftest_exp2(x, y_fma, y_mufu, n, stream)


def fa_status_string(code: int) -> str:
    return load_library().fa_status_string(code).decode()


def fa_version() -> int:
    return load_library().fa_version()


def fa_make_plan(batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, causal, l2_bytes=0, pack=0) -> FaPlan:
    plan = FaPlan()
    rc = load_library().fa_make_plan(batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, int(causal), l2_bytes,
                                     pack, ctypes.byref(plan))
    if rc != FA_OK:
        raise FaError(rc, "fa_make_plan")
    return plan


def fa_plan_task(plan: FaPlan, task: int) -> FaTask:
    t = FaTask()
    rc = load_library().fa_plan_task(ctypes.byref(plan), task, ctypes.byref(t))
    if rc != FA_OK:
        raise FaError(rc, "fa_plan_task")
    return t


def fa_plan_set_grid(plan: FaPlan, grid: int) -> FaPlan:
    """Apply the balanced static order the kernel runs on `grid` CTAs (in place)."""
    rc = load_library().fa_plan_set_grid(ctypes.byref(plan), grid)
    if rc != FA_OK:
        raise FaError(rc, "fa_plan_set_grid")
    return plan


def fa_plan_block_masked(plan: FaPlan, pos0: int, j: int) -> bool:
    return bool(load_library().fa_plan_block_masked(ctypes.byref(plan), pos0, j))


def fa_plan_first_masked_block(plan: FaPlan, pos0: int) -> int:
    return load_library().fa_plan_first_masked_block(ctypes.byref(plan), pos0)


def fa_varlen_workspace_size(batch: int, heads_q: int, total_q: int) -> int:
    return load_library().fa_varlen_workspace_size(batch, heads_q, total_q)


def fa_fwd_varlen(q, k, v, o, lse, cu_q, cu_k, batch, total_q, total_k, heads_q, heads_kv, d_qk, d_v, causal, scale,
                  workspace, workspace_bytes, stream) -> int:
    """``fa_fwd_varlen`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_fwd_varlen(q, k, v, o, lse, cu_q, cu_k, batch, total_q, total_k, heads_q, heads_kv, d_qk,
                                        d_v, int(causal), float(scale), workspace, workspace_bytes, stream)


def fa_fwd_varlen_ex(q, k, v, o, lse, cu_q, cu_k, batch, total_q, total_k, heads_q, heads_kv, d_qk, d_v, causal,
                     scale, workspace, workspace_bytes, opts, stream) -> int:
    return load_library().fa_fwd_varlen_ex(q, k, v, o, lse, cu_q, cu_k, batch, total_q, total_k, heads_q, heads_kv,
                                           d_qk, d_v, int(causal), float(scale), workspace, workspace_bytes,
                                           ctypes.byref(opts) if opts is not None else None, stream)


def fa_fwd_splitkv(q, k, v, o, lse, batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, causal, scale,
                   num_splits, workspace, workspace_bytes, stream, opts=None) -> int:
    """``fa_fwd_splitkv_ex`` (``opts`` None: defaults); pointers as integers."""
    return load_library().fa_fwd_splitkv_ex(q, k, v, o, lse, batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v,
                                            int(causal), float(scale), num_splits, workspace, workspace_bytes,
                                            ctypes.byref(opts) if opts is not None else None, stream)


def fa_splitkv_workspace_size(batch, heads_q, seqlen_q, d_v, num_splits) -> int:
    return load_library().fa_splitkv_workspace_size(batch, heads_q, seqlen_q, d_v, num_splits)


def fa_splitkv_num_splits(batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, causal, num_sms, pack=0) -> int:
    return load_library().fa_splitkv_num_splits(batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, int(causal),
                                                pack, num_sms)


def attention_forward_splitkv(q, k, v, causal: bool = False, scale: float | None = None, num_splits: int = 0,
                              out=None, lse=None, workspace=None, stream=None, options: FaOptions | None = None):
    """Split-KV forward (decode / short Q): same tensors as ``attention_forward``.

    ``num_splits`` 0 lets the library choose; the workspace (uint8) is
    allocated for the count the call will use when not given.  Returns (O, LSE).
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 4-D bf16 CUDA tensor")
    B, Sq, Hq, dqk = q.shape
    _, Sk, Hkv, _ = k.shape
    dv = v.shape[3]
    if out is None:
        out = torch.empty((B, Sq, Hq, dv), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    splits = num_splits
    if splits == 0:
        sms = torch.cuda.get_device_properties(q.device).multi_processor_count
        splits = fa_splitkv_num_splits(B, Hq, Hkv, Sq, Sk, dqk, dv, causal, sms,
                                       options.pack if options is not None else 0)
    need = fa_splitkv_workspace_size(B, Hq, Sq, dv, splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    s = 0.0 if scale is None else float(scale)
    rc = fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sq, Sk,
                        dqk, dv, causal, s, num_splits, workspace.data_ptr(),
                        workspace.numel() * workspace.element_size(), sptr, options)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_splitkv")
    return out, lse


def fa_bwd_workspace_size(batch: int, heads_q: int, seqlen_q: int) -> int:
    return load_library().fa_bwd_workspace_size(batch, heads_q, seqlen_q)


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, batch, heads_q, heads_kv, seqlen_q, seqlen_k, d_qk, d_v, causal, scale,
           workspace, workspace_bytes, stream, opts=None) -> int:
    """``fa_bwd_ex`` of include/fa.h (``opts`` None: defaults); pointers as integers."""
    return load_library().fa_bwd_ex(q, k, v, o, lse, dout, dq, dk, dv, batch, heads_q, heads_kv, seqlen_q, seqlen_k,
                                    d_qk, d_v, int(causal), float(scale), workspace, workspace_bytes,
                                    ctypes.byref(opts) if opts is not None else None, stream)


def attention_backward(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, dq=None, dk=None,
                       dv=None, workspace=None, stream=None, options: FaOptions | None = None):
    """(dQ, dK, dV) for bf16 CUDA tensors laid out as ``attention_forward``'s
    (q, k, v, its outputs o and lse, and dout = dLoss/dO).  Allocates the
    gradients and the workspace when not given."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 4-D bf16 CUDA tensor")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous():
        raise FaError(FA_ERR_INVALID_ARG, "lse must be a contiguous fp32 CUDA tensor")
    B, Sq, Hq, dqk = q.shape
    _, Sk, Hkv, _ = k.shape
    dvh = v.shape[3]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = fa_bwd_workspace_size(B, Hq, Sq)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    s = 0.0 if scale is None else float(scale)
    rc = fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Sq, Sk, dqk, dvh, causal, s,
                workspace.data_ptr(), workspace.numel() * workspace.element_size(), sptr, options)
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd")
    return dq, dk, dv


def fa_fwd_varlen_noalloc(q, k, v, o, lse, cu_q, cu_k, batch, total_q, total_k, heads_q, heads_kv, d_qk, d_v,
                          causal, scale, stream) -> int:
    """``fa_fwd_varlen_noalloc``: the varlen call with the library's static scratch (no workspace)."""
    return load_library().fa_fwd_varlen_noalloc(q, k, v, o, lse, cu_q, cu_k, batch, total_q, total_k, heads_q,
                                                heads_kv, d_qk, d_v, int(causal), float(scale), stream)


def fa_noalloc_scratch_bytes() -> int:
    return load_library().fa_noalloc_scratch_bytes()


def fa_varlen_plan_host(cu_q, cu_k, heads_q, heads_kv, d_qk, d_v, causal, l2_bytes=0, pack=0):
    """Host copy of the planning kernel's task list for int sequences ``cu_q``, ``cu_k`` (length B + 1)."""
    batch = len(cu_q) - 1
    cq = (ctypes.c_int * len(cu_q))(*[int(x) for x in cu_q])
    ck = (ctypes.c_int * len(cu_k))(*[int(x) for x in cu_k])
    n = ctypes.c_int64(0)
    lib = load_library()
    rc = lib.fa_varlen_plan_host(cq, ck, batch, heads_q, heads_kv, d_qk, d_v, int(causal), l2_bytes, pack, None, 0,
                                 ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_varlen_plan_host")
    out = (FaVarlenTask * max(n.value, 1))()
    rc = lib.fa_varlen_plan_host(cq, ck, batch, heads_q, heads_kv, d_qk, d_v, int(causal), l2_bytes, pack, out,
                                 n.value, ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_varlen_plan_host")
    return list(out)[: n.value]


# ---------------------------------------------------------------------------
# torch convenience wrapper (allocation and argument marshalling only)
# ---------------------------------------------------------------------------

def attention_forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
                      return_lse: bool = True, stream=None, options: FaOptions | None = None, workspace=None):
    """O (and LSE) for bf16 CUDA tensors q [B,Sq,Hq,dqk], k [B,Sk,Hkv,dqk], v [B,Sk,Hkv,dv].

    Allocates ``out`` [B,Sq,Hq,dv] bf16 and ``lse`` [B,Hq,Sq] fp32 when not given.
    ``workspace`` (a CUDA tensor of at least SCHED_WORKSPACE_BYTES bytes) selects
    dynamic task assignment (``fa_options.workspace``).  Launches on ``stream``
    (default: torch's current stream).  Raises FaError on any non-OK status.
    """
    import torch

    if workspace is not None:
        if not workspace.is_cuda or workspace.numel() * workspace.element_size() < SCHED_WORKSPACE_BYTES:
            raise FaError(FA_ERR_INVALID_ARG, f"workspace must be a CUDA tensor of >= {SCHED_WORKSPACE_BYTES} bytes")
        base = options if options is not None else default_options()
        options = FaOptions.from_buffer_copy(base)
        options.workspace = workspace.data_ptr()

    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 4-D bf16 CUDA tensor")
    B, Sq, Hq, dqk = q.shape
    _, Sk, Hkv, _ = k.shape
    dv = v.shape[3]
    if out is None:
        out = torch.empty((B, Sq, Hq, dv), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    s = 0.0 if scale is None else float(scale)
    rc = fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                   lse.data_ptr() if lse is not None else None, B, Hq, Hkv, Sq, Sk, dqk, dv, causal, s, options, sptr)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd")
    return (out, lse) if return_lse else out


def attention_forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, causal: bool = False, scale: float | None = None,
                             out=None, lse=None, return_lse: bool = True, workspace=None, stream=None,
                             options: FaOptions | None = None):
    """O (and LSE) of a variable-length batch: q [total_q,Hq,dqk], k [total_k,Hkv,dqk], v [total_k,Hkv,dv]
    bf16 CUDA tensors, cu_seqlens_q / cu_seqlens_k int32 CUDA tensors [B+1].

    Allocates ``out`` [total_q,Hq,dv] bf16, ``lse`` [Hq,total_q] fp32 and the
    planning workspace (uint8) when not given.  Bad cu_seqlens are detected on
    the device and reported by ``fa_device_status``.
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 3-D bf16 CUDA tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.dim() != 1:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 1-D int32 CUDA tensor")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 1:
        raise FaError(FA_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_k must both hold batch + 1 offsets")
    batch = cu_seqlens_q.numel() - 1
    total_q, Hq, dqk = q.shape
    total_k, Hkv, _ = k.shape
    dv = v.shape[2]
    if out is None:
        out = torch.empty((total_q, Hq, dv), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    need = fa_varlen_workspace_size(batch, Hq, total_q)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    s = 0.0 if scale is None else float(scale)
    rc = fa_fwd_varlen_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                          lse.data_ptr() if lse is not None else None, cu_seqlens_q.data_ptr(),
                          cu_seqlens_k.data_ptr(), batch, total_q, total_k, Hq, Hkv, dqk, dv, causal, s,
                          workspace.data_ptr(), workspace.numel(), options, sptr)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_varlen")
    return (out, lse) if return_lse else out


def flops(batch, heads_q, seqlen_q, seqlen_k, d_qk, d_v, causal) -> float:
    """2*B*Hq*Sq*Sk*(d_qk + d_v), halved for causal (the nominal convention)."""
    f = 2.0 * batch * heads_q * seqlen_q * seqlen_k * (d_qk + d_v)
    return f / 2 if causal else f


def default_scale(d_qk: int) -> float:
    return 1.0 / math.sqrt(d_qk)


def fa_bwd_varlen_workspace_size(batch: int, heads_q: int, heads_kv: int, total_q: int, total_k: int) -> int:
    return load_library().fa_bwd_varlen_workspace_size(batch, heads_q, heads_kv, total_q, total_k)


def fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, batch, total_q, total_k, heads_q, heads_kv, d_qk,
                  d_v, causal, scale, workspace, workspace_bytes, stream, opts=None) -> int:
    """``fa_bwd_varlen_ex`` of include/fa.h (``opts`` None: defaults); pointers as integers."""
    return load_library().fa_bwd_varlen_ex(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, batch, total_q, total_k,
                                           heads_q, heads_kv, d_qk, d_v, int(causal), float(scale), workspace,
                                           workspace_bytes, ctypes.byref(opts) if opts is not None else None,
                                           stream)


def attention_backward_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, causal: bool = False,
                              scale: float | None = None, dq=None, dk=None, dv=None, workspace=None, stream=None,
                              options: FaOptions | None = None):
    """(dQ, dK, dV) of a variable-length batch laid out as
    ``attention_forward_varlen``'s: q [total_q,Hq,dqk], k [total_k,Hkv,dqk],
    v [total_k,Hkv,dv], its outputs o [total_q,Hq,dv] and lse [Hq,total_q],
    dout like o; cu_seqlens int32 CUDA tensors [B+1].  Allocates the gradients
    and the workspace when not given."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 3-D bf16 CUDA tensor")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous():
        raise FaError(FA_ERR_INVALID_ARG, "lse must be a contiguous fp32 CUDA tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.dim() != 1:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 1-D int32 CUDA tensor")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 1:
        raise FaError(FA_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_k must both hold batch + 1 offsets")
    batch = cu_seqlens_q.numel() - 1
    total_q, Hq, dqk = q.shape
    total_k, Hkv, _ = k.shape
    dvh = v.shape[2]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = fa_bwd_varlen_workspace_size(batch, Hq, Hkv, total_q, total_k)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    s = 0.0 if scale is None else float(scale)
    rc = fa_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                       dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                       batch, total_q, total_k, Hq, Hkv, dqk, dvh, causal, s, workspace.data_ptr(),
                       workspace.numel() * workspace.element_size(), sptr, options)
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_varlen")
    return dq, dk, dv


# ---------------------------------------------------------------------------
# the paged 8-bit key/value cache
# ---------------------------------------------------------------------------

def fa_kv_append(cache: FaKvCache, q, k, v, q_stride, k_stride, v_stride, q_out, cu_seqlens, batch, total, heads_q,
                 cos_sin, max_positions, rot_dim, interleaved, stream) -> int:
    """``fa_kv_append`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_kv_append(ctypes.byref(cache) if cache is not None else None, q, k, v, q_stride, k_stride,
                                       v_stride, q_out, cu_seqlens, batch, total, heads_q, cos_sin, max_positions,
                                       rot_dim, int(interleaved), stream)


def fa_fwd_paged_workspace_size(batch, heads_q, heads_kv, total_q, max_seqlen_q, total_k, d_qk, d_v) -> int:
    return load_library().fa_fwd_paged_workspace_size(batch, heads_q, heads_kv, total_q, max_seqlen_q, total_k, d_qk,
                                                      d_v)


def fa_fwd_paged(q, cache: FaKvCache, o, lse, cu_seqlens_q, batch, total_q, max_seqlen_q, total_k, heads_q, causal,
                 scale, workspace, workspace_bytes, stream) -> int:
    """``fa_fwd_paged`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_fwd_paged(q, ctypes.byref(cache) if cache is not None else None, o, lse, cu_seqlens_q,
                                       batch, total_q, max_seqlen_q, total_k, heads_q, int(causal), float(scale),
                                       workspace, workspace_bytes, stream)


def _bad(what: str):
    raise FaError(FA_ERR_INVALID_ARG, what)


# an fa_kv_cache as bytes: what FaKvCache lays out, built in one step
_KV_CACHE = struct.Struct("6P7q6i")


def _paged_cache(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens, index):
    """(fa_kv_cache as bytes, heads_kv, d_qk, d_v, batch, capacity) of the cache's tensors, which are checked."""
    import torch

    f8, e8, i32 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.int32
    kd, vd, td = k_cache.shape, v_cache.shape, block_table.shape
    if not (len(kd) == 4 and len(vd) == 4 and kd[:3] == vd[:3] and k_cache.dtype is f8 and v_cache.dtype is f8 and
            k_scale.dtype is e8 and v_scale.dtype is e8 and k_scale.shape == kd[:2] and v_scale.shape == kd[:2] and
            k_scale.is_contiguous() and v_scale.is_contiguous() and len(td) == 2 and block_table.dtype is i32 and
            seqlens_k.dtype is i32 and cu_seqlens.dtype is i32 and seqlens_k.shape == td[:1] and
            cu_seqlens.dim() == 1 and cu_seqlens.shape[0] == td[0] + 1 and seqlens_k.is_contiguous() and
            cu_seqlens.is_contiguous()):  # where they lie, the library checks
        _paged_cache_error(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens, index)
    ks, vs, ts = k_cache.stride(), v_cache.stride(), block_table.stride()
    if (ks[3] != 1 and kd[3] > 1) or (vs[3] != 1 and vd[3] > 1) or (ts[1] != 1 and td[1] > 1):
        _bad("the codes of a token and the entries of a row of block_table must be contiguous")
    pages, heads, page, d_qk = kd
    batch, width = td
    packed = _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                            block_table.data_ptr(), seqlens_k.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
                            ts[0] if batch > 1 else width, pages, page, heads, d_qk, vd[3], width)
    return packed, heads, d_qk, vd[3], batch, width * page


def _paged_cache_error(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens, index):
    """Says which tensor is wrong."""
    import torch

    for name, t, dtype, dim in (("k_cache", k_cache, torch.float8_e4m3fn, 4), ("v_cache", v_cache, torch.float8_e4m3fn, 4),
                                ("k_scale", k_scale, torch.float8_e8m0fnu, 2), ("v_scale", v_scale, torch.float8_e8m0fnu, 2),
                                ("block_table", block_table, torch.int32, 2), ("seqlens_k", seqlens_k, torch.int32, 1),
                                ("cu_seqlens", cu_seqlens, torch.int32, 1)):
        if t.dtype != dtype or t.dim() != dim or t.get_device() != index:
            _bad(f"{name} must be a {dim}-D {str(dtype).removeprefix('torch.')} tensor on cuda:{index}")
        if dim < 4 and name != "block_table" and not t.is_contiguous():
            _bad(f"{name} must be contiguous")
    if v_cache.shape[:3] != k_cache.shape[:3]:
        _bad("k_cache and v_cache must be [num_pages, heads_kv, page_size, d]")
    if k_scale.shape != k_cache.shape[:2] or v_scale.shape != k_cache.shape[:2]:
        _bad("k_scale and v_scale must be [num_pages, heads_kv]")
    _bad("block_table, seqlens_k and cu_seqlens must hold batch rows, batch lengths and batch + 1 offsets")


def _call_stream(index, stream):
    """(pointer of the call's stream, pointer of the current one) on device `index`."""
    import torch

    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is None:
        return current, current
    return (stream.cuda_stream if hasattr(stream, "cuda_stream") else stream) or 0, current


def _empty(shape, dtype, index, ptr, current):
    """torch.empty whose memory is not reused before the work on the stream `ptr` has run."""
    import torch

    if ptr == current:
        return torch.empty(shape, dtype=dtype, device=index)
    with torch.cuda.stream(torch.cuda.ExternalStream(ptr, device=index)):
        return torch.empty(shape, dtype=dtype, device=index)


def _zeros(shape, dtype, index, ptr, current):
    """``_empty`` filled with zeros on the stream `ptr`."""
    import torch

    if ptr == current:
        return torch.zeros(shape, dtype=dtype, device=index)
    with torch.cuda.stream(torch.cuda.ExternalStream(ptr, device=index)):
        return torch.zeros(shape, dtype=dtype, device=index)


# rows (new tokens x query heads a key/value head) up to which a sequence is read straight from the pages
_PAGED_ROWS = 128


def _paged_total_k(batch, capacity, total_q, ratio):
    """The most keys that the sequences of more than _PAGED_ROWS rows can have, if each can have `capacity`."""
    return min(batch, total_q // (_PAGED_ROWS // ratio + 1)) * capacity


@functools.lru_cache(maxsize=256)
def _paged_workspace_bytes(*sizes):
    return load_library().fa_fwd_paged_workspace_size(*sizes)


def _token_stride(name, t, total, heads, d):
    """Elements from token to token of a bf16 tensor [total, heads, d] whose heads lie side by side."""
    import torch

    if t.dtype is not torch.bfloat16 or t.shape != (total, heads, d):
        _bad(f"{name} must be a bf16 tensor [{total}, {heads}, {d}]")
    st = t.stride()
    if total == 0 or (st[2] == 1 and (heads == 1 or st[1] == d)):
        return st[0] if total > 1 else heads * d
    _bad(f"{name}: a token's heads must be contiguous")


def kv_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens, q=None, cos_sin=None,
              interleaved: bool = False, q_out=None, stream=None):
    """Append the new tokens' keys and values to a paged 8-bit cache (``fa_kv_append`` of include/fa.h).

    k [total,Hkv,dqk], v [total,Hkv,dv] and, to be rotated along with the keys, q [total,Hq,dqk] are bf16 CUDA tensors
    whose tokens may lie apart (views of one projection's output); k_cache, v_cache float8_e4m3fn
    [num_pages,Hkv,page_size,d] with contiguous codes and strides of multiples of 16, k_scale, v_scale float8_e8m0fnu [num_pages,Hkv];
    block_table int32 [B,max_pages], seqlens_k int32 [B] (lengths with the new tokens), cu_seqlens int32 [B+1];
    cos_sin fp32 [positions, rot_dim] or None (no rotation).  The cache is updated in place; returns q_out (allocated
    when not given; may be q), None without q.  Launches on ``stream`` (default: torch's current stream).  Offsets,
    lengths and pages out of range are detected on the device and reported by ``fa_device_status``.
    """
    import torch

    index = k.get_device()
    if index < 0:
        _bad("k must be a CUDA tensor")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return kv_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens, q, cos_sin,
                             interleaved, q_out, stream)
    cache, heads, d_qk, d_v, batch, _ = _paged_cache(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k,
                                                     cu_seqlens, index)
    total = k.shape[0] if k.dim() else 0
    ks = _token_stride("k", k, total, heads, d_qk)
    vs = _token_stride("v", v, total, heads, d_v)
    rot = positions = 0
    cs = qp = qo = None
    if cos_sin is not None:
        if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            _bad("cos_sin must be a contiguous 2-D fp32 tensor")
        positions, rot = cos_sin.shape
        cs = cos_sin.data_ptr()
    ptr, current = _call_stream(index, stream)
    heads_q = qs = 0
    if q is not None:
        shape = q.shape
        heads_q = shape[1] if len(shape) == 3 else 0
        qs = _token_stride("q", q, total, heads_q, d_qk)
        if q_out is None:
            q_out = _empty(shape, torch.bfloat16, index, ptr, current)
        elif q_out.dtype is not torch.bfloat16 or q_out.shape != shape or not q_out.is_contiguous():
            _bad("q_out must be a contiguous bf16 tensor of q's shape")
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        _bad("q_out without q")
    rc = load_library().fa_kv_append(cache, qp, k.data_ptr(), v.data_ptr(), qs, ks, vs, qo, cu_seqlens.data_ptr(), batch,
                                     total, heads_q, cs, positions, rot, interleaved, ptr)
    if rc != FA_OK:
        raise FaError(rc, "fa_kv_append")
    return q_out


def attention_forward_paged(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens_q,
                            max_seqlen_q: int, causal: bool = True, scale: float | None = None,
                            total_k: int | None = None, out=None, lse=None, return_lse: bool = True, workspace=None,
                            stream=None):
    """O (and LSE) of new tokens over a paged 8-bit cache (``fa_fwd_paged`` of include/fa.h).

    q [total_q,Hq,dqk] bf16 (packed, cu_seqlens_q int32 [B+1], at most ``max_seqlen_q`` tokens a sequence); the cache
    as ``kv_append`` fills it, seqlens_k the lengths with the new tokens.  ``total_k``: an upper limit of their sum over
    the sequences of more than 128 rows (new tokens x query heads a key/value head), whose unpacked keys the workspace
    holds (default: what the block table can hold of as many such sequences as total_q tokens can make).
    Allocates ``out`` [total_q,Hq,dv] bf16, ``lse`` [Hq,total_q] fp32 and the workspace (uint8) when not given.
    Offsets, lengths and pages out of range are detected on the device and reported by ``fa_device_status``.
    """
    import torch

    index = q.get_device()
    qd = q.shape
    if index < 0 or q.dtype is not torch.bfloat16 or len(qd) != 3 or not q.is_contiguous():
        _bad("q must be a contiguous 3-D bf16 CUDA tensor")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return attention_forward_paged(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens_q,
                                           max_seqlen_q, causal, scale, total_k, out, lse, return_lse, workspace, stream)
    cache, heads, d_qk, d_v, batch, capacity = _paged_cache(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k,
                                                            cu_seqlens_q, index)
    total_q, heads_q, d = qd
    if d != d_qk:
        _bad(f"q must be [total_q, heads_q, {d_qk}]")
    if total_k is None:
        total_k = _paged_total_k(batch, capacity, total_q, max(heads_q // max(heads, 1), 1))
    ptr, current = _call_stream(index, stream)
    if out is None:
        out = _empty((total_q, heads_q, d_v), torch.bfloat16, index, ptr, current)
    elif out.dtype is not torch.bfloat16 or out.shape != (total_q, heads_q, d_v) or not out.is_contiguous():
        _bad(f"out must be a contiguous bf16 tensor [total_q, heads_q, {d_v}]")
    if lse is None:
        if return_lse:
            lse = _empty((heads_q, total_q), torch.float32, index, ptr, current)
    elif lse.dtype is not torch.float32 or lse.shape != (heads_q, total_q) or not lse.is_contiguous():
        _bad("lse must be a contiguous fp32 tensor [heads_q, total_q]")
    if workspace is None:
        size = _paged_workspace_bytes(batch, heads_q, heads, total_q, max_seqlen_q, total_k, d_qk, d_v)
        workspace = _empty((size or 16,), torch.uint8, index, ptr, current)
    else:
        if not workspace.is_contiguous():
            _bad("workspace must be contiguous")
        size = workspace.numel() * workspace.element_size()
    rc = load_library().fa_fwd_paged(q.data_ptr(), cache, out.data_ptr(), lse.data_ptr() if lse is not None else None,
                                     cu_seqlens_q.data_ptr(), batch, total_q, max_seqlen_q, total_k, heads_q,
                                     1 if causal else 0, 0.0 if scale is None else scale, workspace.data_ptr(), size, ptr)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_paged")
    return (out, lse) if return_lse else out


_INT_MAX = 2 ** 31 - 1  # of the C interface's int: ctypes would keep the lower 32 bits of what is larger


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def fa_rotary_table(cos_sin, positions, rot_dim, base, scaling: FaRotaryScaling | None, stream) -> int:
    """``fa_rotary_table`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_rotary_table(cos_sin, positions, rot_dim, float(base),
                                          ctypes.byref(scaling) if scaling is not None else None, stream)


def fa_rotary(q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, positions, cu_seqlens, batch, seqlen,
              total, heads_q, heads_k, d, cos_sin, max_positions, rot_dim, interleaved, backward, stream) -> int:
    """``fa_rotary`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_rotary(q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, positions,
                                    cu_seqlens, batch, seqlen, total, heads_q, heads_k, d, cos_sin, max_positions, rot_dim,
                                    int(interleaved), int(backward), stream)


def rotary_table(positions: int, rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original: float = 0.0, low: float = 1.0, high: float = 32.0, magnitude: float = 1.0, out=None, device=None,
                 stream=None):
    """Cosines and sines of positions 0 .. positions - 1 (``fa_rotary_table`` of include/fa.h), fp32 [positions, rot_dim],
    as ``kv_append`` and ``rotary`` take them.

    ``scaling`` is "none", "linear", "base" or "by_parts" (with ``factor``, and for the last ``original``, the trained
    length, and ``low`` and ``high``, turns within it); every value is multiplied by ``magnitude``.  Allocates ``out`` on
    ``device`` (default: the current CUDA device) when not given."""
    import torch

    if scaling not in ROTARY_SCALING:
        _bad(f"scaling must be one of {', '.join(ROTARY_SCALING)}")
    if not (0 <= positions <= _INT_MAX and 0 <= rot_dim <= _INT_MAX):
        _bad("positions and rot_dim must not be negative, nor beyond 32 bits")
    if out is not None:
        if out.dtype is not torch.float32 or out.shape != (positions, rot_dim) or not out.is_contiguous() or not out.is_cuda:
            _bad(f"out must be a contiguous fp32 CUDA tensor [{positions}, {rot_dim}]")
        index = out.get_device()
    else:
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            _bad("device must be a CUDA device")
        index = torch._C._cuda_getDevice() if device.index is None else device.index
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return rotary_table(positions, rot_dim, base, scaling, factor, original, low, high, magnitude, out, index, stream)
    ptr = current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None:
        ptr, current = _call_stream(index, stream)
    if out is None:
        out = _empty((positions, rot_dim), torch.float32, index, ptr, current)
    spec = FaRotaryScaling(ROTARY_SCALING[scaling], factor, original, low, high, magnitude)
    rc = fa_rotary_table(out.data_ptr(), positions, rot_dim, base, spec, ptr)
    if rc != FA_OK:
        raise FaError(rc, "fa_rotary_table")
    return out


def _rotary_rows(torch, name, t, tokens, d):
    """(heads, stride from token to token) of a bf16 tensor [*tokens, heads, d]."""
    shape, st = t.shape, t.stride()
    if t.dtype is not torch.bfloat16 or shape[:-2] != tokens or shape[-1] != d:
        _bad(f"{name} must be a bf16 tensor of tokens {list(tokens)} with heads of {d}")
    heads = shape[-2]
    if st[-1] == 1 and (st[-2] == d or heads == 1):
        if len(tokens) == 1:
            return heads, st[0] if tokens[0] > 1 else heads * d
        batch, seqlen = tokens
        if batch <= 1 or seqlen <= 1 or st[0] == seqlen * st[1]:
            return heads, st[1] if seqlen > 1 else st[0] if batch > 1 else heads * d
        _bad(f"{name}: the step from sequence to sequence must be that of seqlen tokens")
    if t.numel() == 0:
        return heads, heads * d
    _bad(f"{name}: a token's heads must be contiguous")


def _rotary(q, k, cos_sin, positions, cu_seqlens, interleaved, q_out, k_out, stream, backward):
    import torch

    ref = q if q is not None else k
    if ref is None:
        _bad("neither q nor k")
    index = ref.get_device()
    if index < 0:
        _bad("q and k must be CUDA tensors")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _rotary(q, k, cos_sin, positions, cu_seqlens, interleaved, q_out, k_out, stream, backward)
    shape = ref.shape
    if len(shape) not in (3, 4):
        _bad("q and k must be [total, heads, d] or [batch, seqlen, heads, d]")
    tokens, d = shape[:-2], shape[-1]
    total = tokens[0] if len(tokens) == 1 else tokens[0] * tokens[1]
    table = cos_sin.shape
    if cos_sin.dtype is not torch.float32 or len(table) != 2 or not cos_sin.is_contiguous():
        _bad("cos_sin must be a contiguous 2-D fp32 tensor")
    pos = cu = None
    batch = seqlen = 0
    if positions is not None:
        if cu_seqlens is not None:
            _bad("positions and cu_seqlens exclude each other")
        _int32(torch, "positions", positions, tokens)
        pos = positions.data_ptr()
    elif cu_seqlens is not None:
        batch = cu_seqlens.numel() - 1
        if len(tokens) != 1 or batch < 0:
            _bad("cu_seqlens must hold batch + 1 offsets into [total, heads, d]")
        _int32(torch, "cu_seqlens", cu_seqlens, (batch + 1,))
        cu = cu_seqlens.data_ptr()
    else:
        seqlen = tokens[-1] or 1  # without a batch: one sequence
    ptr = current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None:
        ptr, current = _call_stream(index, stream)
    qp = kp = qo = ko = None
    hq = hk = qs = ks = qos = kos = 0
    if q is not None:
        hq, qs = _rotary_rows(torch, "q", q, tokens, d)
        if q_out is None:
            q_out = _empty(q.shape, torch.bfloat16, index, ptr, current)
        ho, qos = _rotary_rows(torch, "q_out", q_out, tokens, d)
        if ho != hq:
            _bad("q_out must have q's shape")
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        _bad("q_out without q")
    if k is not None:
        hk, ks = _rotary_rows(torch, "k", k, tokens, d)
        if k_out is None:
            k_out = _empty(k.shape, torch.bfloat16, index, ptr, current)
        ho, kos = _rotary_rows(torch, "k_out", k_out, tokens, d)
        if ho != hk:
            _bad("k_out must have k's shape")
        kp, ko = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        _bad("k_out without k")
    rc = load_library().fa_rotary(qp, kp, qo, ko, qs, ks, qos, kos, pos, cu, batch, seqlen, total, hq, hk, d,
                                  cos_sin.data_ptr(), table[0], table[1], 1 if interleaved else 0, backward, ptr)
    if rc != FA_OK:
        raise FaError(rc, "fa_rotary")
    return q_out, k_out


def rotary(q, k, cos_sin, positions=None, cu_seqlens=None, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """(q, k) rotated by their positions (``fa_rotary`` of include/fa.h); either may be None.

    bf16 CUDA tensors [total,H,d] or [B,S,H,d] whose tokens may lie apart (views of one projection's output); cos_sin fp32
    [max_positions, rot_dim] as ``rotary_table`` makes it.  Positions: ``positions`` int32 of the tokens' shape, or the
    index in the sequence that ``cu_seqlens`` int32 [B+1] gives (rows of no sequence are left as they are), or without both
    the index in the sequence [B,S] (in the whole of [total]).  ``q_out`` and ``k_out`` (allocated when not given) may be q
    and k.  Positions outside the table are detected on the device and reported by ``fa_device_status``."""
    return _rotary(q, k, cos_sin, positions, cu_seqlens, interleaved, q_out, k_out, stream, 0)


def rotary_backward(dq, dk, cos_sin, positions=None, cu_seqlens=None, interleaved: bool = False, q_out=None, k_out=None,
                    stream=None):
    """The gradients of ``rotary``'s q and k from those of its results: the transposed rotation, arguments alike."""
    return _rotary(dq, dk, cos_sin, positions, cu_seqlens, interleaved, q_out, k_out, stream, 1)


# ---------------------------------------------------------------------------
# sparse attention over selected pages
# ---------------------------------------------------------------------------

def fa_kv_bounds(cache: FaKvCache, k_bounds, cu_seqlens, batch, total, stream) -> int:
    """``fa_kv_bounds`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_kv_bounds(ctypes.byref(cache) if cache is not None else None, k_bounds, cu_seqlens, batch,
                                       total, stream)


def fa_kv_select_workspace_size(batch: int, total_q: int, heads_kv: int, max_pages: int) -> int:
    return load_library().fa_kv_select_workspace_size(batch, total_q, heads_kv, max_pages)


def fa_kv_select(q, k_bounds, k_scale, block_table, table_stride, seqlens_k, cu_seqlens_q, batch, total_q, max_seqlen_q,
                 heads_q, heads_kv, d_qk, num_pages, page_size, max_pages, causal, top, keep_first, keep_last, lists,
                 list_lens, workspace, workspace_bytes, stream) -> int:
    """``fa_kv_select`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_kv_select(q, k_bounds, k_scale, block_table, table_stride, seqlens_k, cu_seqlens_q, batch,
                                       total_q, max_seqlen_q, heads_q, heads_kv, d_qk, num_pages, page_size, max_pages,
                                       int(causal), top, keep_first, keep_last, lists, list_lens, workspace,
                                       workspace_bytes, stream)


def fa_fwd_lists_workspace_size(heads_q: int, heads_kv: int, d_v: int) -> int:
    return load_library().fa_fwd_lists_workspace_size(heads_q, heads_kv, d_v)


def fa_fwd_lists(q, cache: FaKvCache, lists, list_lens, width, o, lse, total_q, heads_q, scale, workspace, workspace_bytes,
                 stream) -> int:
    """``fa_fwd_lists`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_fwd_lists(q, ctypes.byref(cache) if cache is not None else None, lists, list_lens, width, o,
                                       lse, total_q, heads_q, float(scale), workspace, workspace_bytes, stream)


def _int32(torch, name, t, shape):
    """Checks a contiguous int32 tensor of a shape."""
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        _bad(f"{name} must be a contiguous int32 tensor {list(shape)}")


def _table_rows(torch, block_table, seqlens_k):
    """(batch, max_pages, row stride) of a block table beside its lengths."""
    td, st = block_table.shape, block_table.stride()
    if block_table.dtype is not torch.int32 or len(td) != 2 or (st[1] != 1 and td[1] > 1):
        _bad("block_table must be a 2-D int32 tensor whose rows are contiguous")
    batch, width = td
    if seqlens_k.dtype is not torch.int32 or seqlens_k.shape != td[:1] or not seqlens_k.is_contiguous():
        _bad(f"seqlens_k must be a contiguous int32 tensor [{batch}]")
    return batch, width, st[0] if batch > 1 else width


def _bounds(torch, k_bounds, pages, heads, d):
    if k_bounds.dtype is not torch.float8_e4m3fn or k_bounds.shape != (pages, heads, 2, d) or not k_bounds.is_contiguous():
        _bad(f"k_bounds must be a contiguous float8_e4m3fn tensor [{pages}, {heads}, 2, {d}]")
    return k_bounds.data_ptr()


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, *sizes):
    """What the library's function `name` says, 16 at least; it depends on the sizes alone."""
    return getattr(load_library(), name)(*sizes) or 16


def _workspace(torch, workspace, stream, name, *sizes):
    """(pointer, bytes, whether it is to be freed) of a call's workspace: the caller's tensor, or memory of the caching
    allocator on the call's stream that goes back to it when the call has been issued (what is allocated there later runs
    after it).  A tensor of its own would cost 6 us a call."""
    if workspace is None:
        size = _workspace_bytes(name, *sizes)
        return torch._C._cuda_cudaCachingAllocator_raw_alloc(size, stream), size, True
    if not workspace.is_contiguous():
        _bad("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), False


def kv_bounds(k_cache, k_bounds, block_table, seqlens_k, cu_seqlens, total: int, stream=None):
    """Update the bounds of the pages that hold a step's new tokens (``fa_kv_bounds`` of include/fa.h), after ``kv_append``.

    k_bounds float8_e4m3fn [num_pages,Hkv,2,dqk] (largest and smallest code of each channel) is written in place and
    returned; the other tensors as for ``kv_append``, cu_seqlens int32 [B+1] of the ``total`` new tokens."""
    import torch

    index = k_cache.get_device()
    kd, ks = k_cache.shape, k_cache.stride()
    if index < 0 or k_cache.dtype is not torch.float8_e4m3fn or len(kd) != 4 or ks[3] != 1:
        _bad("k_cache must be a 4-D float8_e4m3fn CUDA tensor whose tokens' codes are contiguous")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return kv_bounds(k_cache, k_bounds, block_table, seqlens_k, cu_seqlens, total, stream)
    pages, heads, page, d = kd
    batch, width, ts = _table_rows(torch, block_table, seqlens_k)
    if not 0 <= total <= _INT_MAX:
        _bad("total must not be negative, nor beyond 32 bits")
    _int32(torch, "cu_seqlens", cu_seqlens, (batch + 1,))
    bounds = _bounds(torch, k_bounds, pages, heads, d)
    ptr = torch._C._cuda_getCurrentRawStream(index) if stream is None else _call_stream(index, stream)[0]
    cache = _KV_CACHE.pack(k_cache.data_ptr(), 0, 0, 0, block_table.data_ptr(), seqlens_k.data_ptr(), ks[0], ks[1], ks[2],
                           0, 0, 0, ts, pages, page, heads, d, 0, width)
    rc = load_library().fa_kv_bounds(cache, bounds, cu_seqlens.data_ptr(), batch, total, ptr)
    if rc != FA_OK:
        raise FaError(rc, "fa_kv_bounds")
    return k_bounds


def kv_select(q, k_bounds, k_scale, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q: int, page_size: int, top: int,
              causal: bool = True, keep_first: int = 0, keep_last: int = 1, lists=None, list_lens=None, workspace=None,
              stream=None):
    """The ``top`` pages that each new token and key/value head attends to (``fa_kv_select`` of include/fa.h).

    q [total_q,Hq,dqk] bf16 (packed by cu_seqlens_q int32 [B+1], at most ``max_seqlen_q`` tokens a sequence), k_bounds as
    ``kv_bounds`` keeps it, k_scale float8_e8m0fnu [num_pages,Hkv], block_table and seqlens_k as for
    ``attention_forward_paged``.  The first ``keep_first`` and the last ``keep_last`` (1 at least) pages that a token sees
    are always taken, the others by the sum over the query heads of the largest score that a key within the bounds can
    have.  Returns (lists int32 [total_q,Hkv,top], list_lens int32 [total_q]) for ``attention_forward_lists``, allocated
    when not given, as is the workspace (uint8), which grows with total_q * Hkv * the width of block_table.  Rows of tokens
    of no sequence (a padded batch) have a list_lens of 0 if it is allocated here, and are left as they are if it is given:
    then it has to hold a length for them, 0 for none."""
    import torch

    index = q.get_device()
    qd, sd = q.shape, k_scale.shape
    if index < 0 or q.dtype is not torch.bfloat16 or len(qd) != 3 or not q.is_contiguous():
        _bad("q must be a contiguous 3-D bf16 CUDA tensor")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return kv_select(q, k_bounds, k_scale, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q, page_size, top,
                             causal, keep_first, keep_last, lists, list_lens, workspace, stream)
    if k_scale.dtype is not torch.float8_e8m0fnu or len(sd) != 2 or not k_scale.is_contiguous():
        _bad("k_scale must be a contiguous float8_e8m0fnu tensor [num_pages, heads_kv]")
    total_q, heads_q, d = qd
    pages, heads = sd
    bounds = _bounds(torch, k_bounds, pages, heads, d)
    batch, width, ts = _table_rows(torch, block_table, seqlens_k)
    _int32(torch, "cu_seqlens_q", cu_seqlens_q, (batch + 1,))
    if max(max_seqlen_q, page_size, top, keep_first, keep_last) > _INT_MAX or \
            min(max_seqlen_q, page_size, top, keep_first, keep_last) < 0:
        _bad("max_seqlen_q, page_size, top, keep_first and keep_last must not be negative, nor beyond 32 bits")
    ptr = current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None:
        ptr, current = _call_stream(index, stream)
    if lists is None:
        lists = _empty((total_q, heads, top), torch.int32, index, ptr, current)
    else:
        _int32(torch, "lists", lists, (total_q, heads, top))
    if list_lens is None:
        # attention_forward_lists knows no sequences: rows of none are to be rows without a key (8 us of the host's time,
        # which callers that keep their own list_lens save)
        list_lens = _zeros((total_q,), torch.int32, index, ptr, current)
    else:
        _int32(torch, "list_lens", list_lens, (total_q,))
    ws, size, own = _workspace(torch, workspace, ptr, "fa_kv_select_workspace_size", batch, total_q, heads, width)
    try:
        rc = load_library().fa_kv_select(q.data_ptr(), bounds, k_scale.data_ptr(), block_table.data_ptr(), ts,
                                         seqlens_k.data_ptr(), cu_seqlens_q.data_ptr(), batch, total_q, max_seqlen_q,
                                         heads_q, heads, d, pages, page_size, width, 1 if causal else 0, top, keep_first,
                                         keep_last, lists.data_ptr(), list_lens.data_ptr(), ws, size, ptr)
    finally:
        if own:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ws)
    if rc != FA_OK:
        raise FaError(rc, "fa_kv_select")
    return lists, list_lens


def _pool(torch, k_cache, v_cache, k_scale, v_scale, table, seqlens, width, table_stride):
    """(fa_kv_cache as bytes, num_pages, heads_kv, d_qk, d_v) of the cache's tensors, which are checked."""
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    kd, vd = k_cache.shape, v_cache.shape
    head = kd[:2]
    ks, vs = k_cache.stride(), v_cache.stride()
    if not (len(kd) == 4 and len(vd) == 4 and kd[:3] == vd[:3] and k_cache.dtype is f8 and v_cache.dtype is f8 and
            k_scale.dtype is e8 and v_scale.dtype is e8 and k_scale.shape == head and v_scale.shape == head and
            k_scale.is_contiguous() and v_scale.is_contiguous() and ks[3] == 1 and vs[3] == 1):
        _pool_error(k_cache, v_cache, k_scale, v_scale)
    pages, heads, page, d_qk = kd
    d_v = vd[3]
    packed = _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), table, seqlens,
                            ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], table_stride, pages, page, heads, d_qk, d_v, width)
    return packed, pages, heads, d_qk, d_v


def _pool_error(k_cache, v_cache, k_scale, v_scale):
    """Says which tensor is wrong."""
    import torch

    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype is not torch.float8_e4m3fn or t.dim() != 4 or t.stride(3) != 1:
            _bad(f"{name} must be a 4-D float8_e4m3fn tensor whose tokens' codes are contiguous")
    if k_cache.shape[:3] != v_cache.shape[:3]:
        _bad("k_cache and v_cache must be [num_pages, heads_kv, page_size, d]")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dtype is not torch.float8_e8m0fnu or t.shape != k_cache.shape[:2] or not t.is_contiguous():
            _bad(f"{name} must be a contiguous float8_e8m0fnu tensor [num_pages, heads_kv]")
    _bad("the cache's tensors do not fit each other")


def attention_forward_lists(q, k_cache, v_cache, k_scale, v_scale, lists, list_lens, scale: float | None = None, out=None,
                            lse=None, return_lse: bool = True, workspace=None, stream=None):
    """O (and LSE) of tokens over lists of a paged 8-bit cache's pages (``fa_fwd_lists`` of include/fa.h).

    q [total_q,Hq,dqk] bf16; lists int32 [total_q,Hkv,width] and list_lens int32 [total_q] from ``kv_select`` or made by
    the caller: token t and key/value head h see the first list_lens[t] tokens of the pages lists[t,h].  Allocates ``out``
    [total_q,Hq,dv] bf16, ``lse`` [Hq,total_q] fp32 and the workspace (uint8) when not given.  Lengths and pages out of
    range are detected on the device and reported by ``fa_device_status``."""
    import torch

    index = q.get_device()
    qd = q.shape
    if index < 0 or q.dtype is not torch.bfloat16 or len(qd) != 3 or not q.is_contiguous():
        _bad("q must be a contiguous 3-D bf16 CUDA tensor")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return attention_forward_lists(q, k_cache, v_cache, k_scale, v_scale, lists, list_lens, scale, out, lse,
                                           return_lse, workspace, stream)
    total_q, heads_q, d = qd
    ld = lists.shape
    width = ld[2] if len(ld) == 3 else -1
    cache, _, heads, d_qk, d_v = _pool(torch, k_cache, v_cache, k_scale, v_scale, lists.data_ptr(), list_lens.data_ptr(), width,
                                       width)
    if d != d_qk or width < 0:
        _bad(f"q must be [total_q, heads_q, {d_qk}] and lists [total_q, {heads}, width]")
    _int32(torch, "lists", lists, (total_q, heads, width))
    _int32(torch, "list_lens", list_lens, (total_q,))
    ptr = current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None:
        ptr, current = _call_stream(index, stream)
    if out is None:
        out = _empty((total_q, heads_q, d_v), torch.bfloat16, index, ptr, current)
    elif out.dtype is not torch.bfloat16 or out.shape != (total_q, heads_q, d_v) or not out.is_contiguous():
        _bad(f"out must be a contiguous bf16 tensor [total_q, heads_q, {d_v}]")
    if lse is None:
        if return_lse:
            lse = _empty((heads_q, total_q), torch.float32, index, ptr, current)
    elif lse.dtype is not torch.float32 or lse.shape != (heads_q, total_q) or not lse.is_contiguous():
        _bad("lse must be a contiguous fp32 tensor [heads_q, total_q]")
    ws, size, own = _workspace(torch, workspace, ptr, "fa_fwd_lists_workspace_size", heads_q, heads, d_v)
    try:
        rc = load_library().fa_fwd_lists(q.data_ptr(), cache, lists.data_ptr(), list_lens.data_ptr(), width, out.data_ptr(),
                                         lse.data_ptr() if lse is not None else None, total_q, heads_q,
                                         0.0 if scale is None else scale, ws, size, ptr)
    finally:
        if own:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ws)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_lists")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------------------
# the cache's pages among the rows of a block table
# ---------------------------------------------------------------------------

def fa_kv_pages_workspace_size(batch: int, rows: int, num_pages: int) -> int:
    return load_library().fa_kv_pages_workspace_size(batch, rows, num_pages)


def fa_kv_fork(cache: FaKvCache, k_bounds, page_refs, batch, parents, new_tokens, rows, table_out, table_out_stride,
               seqlens_out, refs_out, workspace, workspace_bytes, stream) -> int:
    """``fa_kv_fork`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_kv_fork(ctypes.byref(cache) if cache is not None else None, k_bounds, page_refs, batch,
                                     parents, new_tokens, rows, table_out, table_out_stride, seqlens_out, refs_out,
                                     workspace, workspace_bytes, stream)


def fa_kv_compact(cache: FaKvCache, k_bounds, page_refs, batch, table_out, table_out_stride, refs_out, page_map, used,
                  workspace, workspace_bytes, stream) -> int:
    """``fa_kv_compact`` of include/fa.h; pointer arguments are integers (device addresses)."""
    return load_library().fa_kv_compact(ctypes.byref(cache) if cache is not None else None, k_bounds, page_refs, batch,
                                        table_out, table_out_stride, refs_out, page_map, used, workspace, workspace_bytes,
                                        stream)


def _table_out(torch, table_out, rows, width, index, ptr, current):
    """(tensor, row stride) of the table that is written."""
    if table_out is None:
        return _empty((rows, width), torch.int32, index, ptr, current), width
    st = table_out.stride()
    if table_out.dtype is not torch.int32 or table_out.shape != (rows, width) or (st[1] != 1 and width > 1):
        _bad(f"table_out must be an int32 tensor [{rows}, {width}] whose rows are contiguous")
    return table_out, st[0] if rows > 1 else width


def _int32_out(torch, name, t, n, index, ptr, current):
    if t is None:
        return _empty((n,), torch.int32, index, ptr, current)
    if t.dtype is not torch.int32 or t.shape != (n,) or not t.is_contiguous():
        _bad(f"{name} must be a contiguous int32 tensor [{n}]")
    return t


def kv_fork(parents, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, page_refs, new_tokens=None, k_bounds=None,
            table_out=None, seqlens_out=None, refs_out=None, workspace=None, stream=None):
    """Rows of a block table taken over by others, with pages for new tokens (``fa_kv_fork`` of include/fa.h).

    Row r of the result takes over row parents[r] (int32 [rows]; -1: it starts empty) and gets room for new_tokens[r]
    (int32 [rows]) more tokens: beams that fork, requests that end (no row names them) or begin, sequences that grow.
    Full pages are shared, page_refs (int32 [num_pages]) counts their uses; a last page that is not full stays with the
    first heir if nothing else uses it (another row or a holder that page_refs counts), other heirs get a copy.  Returns (table_out int32 [rows,max_pages], seqlens_out int32 [rows], refs_out int32
    [num_pages]), allocated when not given; refs_out may be page_refs.  The cache (and ``k_bounds``, if given) changes in
    new pages only.  Rows out of range and rows that find no free pages become empty, which ``fa_device_status`` reports.
    A pool begins with lengths and counts of 0, whatever the table holds."""
    import torch

    index = k_cache.get_device()
    if index < 0:
        _bad("k_cache must be a CUDA tensor")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return kv_fork(parents, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, page_refs, new_tokens,
                           k_bounds, table_out, seqlens_out, refs_out, workspace, stream)
    batch, width, ts = _table_rows(torch, block_table, seqlens_k)
    cache, pages, heads, d_qk, _ = _pool(torch, k_cache, v_cache, k_scale, v_scale, block_table.data_ptr(), seqlens_k.data_ptr(),
                                         width, ts)
    rows = parents.numel()
    _int32(torch, "parents", parents, (rows,))
    _int32(torch, "page_refs", page_refs, (pages,))
    grow = None
    if new_tokens is not None:
        _int32(torch, "new_tokens", new_tokens, (rows,))
        grow = new_tokens.data_ptr()
    bounds = _bounds(torch, k_bounds, pages, heads, d_qk) if k_bounds is not None else None
    ptr = current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None:
        ptr, current = _call_stream(index, stream)
    table_out, out_stride = _table_out(torch, table_out, rows, width, index, ptr, current)
    seqlens_out = _int32_out(torch, "seqlens_out", seqlens_out, rows, index, ptr, current)
    refs_out = _int32_out(torch, "refs_out", refs_out, pages, index, ptr, current)
    ws, size, own = _workspace(torch, workspace, ptr, "fa_kv_pages_workspace_size", batch, rows, pages)
    try:
        rc = load_library().fa_kv_fork(cache, bounds, page_refs.data_ptr(), batch, parents.data_ptr(), grow, rows,
                                       table_out.data_ptr(), out_stride, seqlens_out.data_ptr(), refs_out.data_ptr(),
                                       ws, size, ptr)
    finally:
        if own:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ws)
    if rc != FA_OK:
        raise FaError(rc, "fa_kv_fork")
    return table_out, seqlens_out, refs_out


def kv_compact(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, page_refs, k_bounds=None, table_out=None,
               refs_out=None, page_map=None, used=None, workspace=None, stream=None):
    """Move the cache's pages in use to its lowest indices (``fa_kv_compact`` of include/fa.h).

    Returns (table_out, refs_out, page_map int32 [num_pages]: each page's new index, -1 for a free one, used int32 [1]),
    allocated when not given; table_out may be block_table and refs_out page_refs."""
    import torch

    index = k_cache.get_device()
    if index < 0:
        _bad("k_cache must be a CUDA tensor")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return kv_compact(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, page_refs, k_bounds, table_out,
                              refs_out, page_map, used, workspace, stream)
    batch, width, ts = _table_rows(torch, block_table, seqlens_k)
    cache, pages, heads, d_qk, _ = _pool(torch, k_cache, v_cache, k_scale, v_scale, block_table.data_ptr(), seqlens_k.data_ptr(),
                                         width, ts)
    _int32(torch, "page_refs", page_refs, (pages,))
    bounds = _bounds(torch, k_bounds, pages, heads, d_qk) if k_bounds is not None else None
    ptr = current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None:
        ptr, current = _call_stream(index, stream)
    table_out, out_stride = _table_out(torch, table_out, batch, width, index, ptr, current)
    refs_out = _int32_out(torch, "refs_out", refs_out, pages, index, ptr, current)
    page_map = _int32_out(torch, "page_map", page_map, pages, index, ptr, current)
    used = _int32_out(torch, "used", used, 1, index, ptr, current)
    ws, size, own = _workspace(torch, workspace, ptr, "fa_kv_pages_workspace_size", batch, 0, pages)
    try:
        rc = load_library().fa_kv_compact(cache, bounds, page_refs.data_ptr(), batch, table_out.data_ptr(), out_stride,
                                          refs_out.data_ptr(), page_map.data_ptr(), used.data_ptr(), ws, size, ptr)
    finally:
        if own:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ws)
    if rc != FA_OK:
        raise FaError(rc, "fa_kv_compact")
    return table_out, refs_out, page_map, used
