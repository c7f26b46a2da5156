"""Thin ctypes binding of libattn_paged.so (include/attn_paged.h).

Argument marshalling only: every step of the attention runs in the library's CUDA
kernels.  Functions keep the C names.  Tensors are torch tensors (device memory and
streams come from PyTorch); the binding passes their raw pointers.  If the library
cannot be loaded the import fails loudly: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_WORKSPACE = -3
ATTN_ERR_CUDA = -4
ATTN_KV_BF16 = 0
ATTN_KV_FP8_E4M3 = 1
ATTN_KV_FP4_E2M1 = 2

EXPORTED = ("attn_plan", "attn_run_paged", "attn_run_phase", "attn_plan_destroy", "attn_get_device_error",
            "attn_status_string", "attn_plan_host", "attn_plan_info", "attn_plan_blocks",
            "attn_plan_segments", "attn_plan_cta_heads", "attn_plan_stage_units",
            "attn_plan_merge_ctas", "attn_plan_select_ctas",
            "attn_debug_tc_gemm", "attn_debug_stamps",
            "attn_run_paged_no_workspace",
            "attn_append_kv", "attn_append_kv_rope", "attn_read_kv", "attn_kv_row_bytes",
            "attn_append_kv_mrope", "attn_bounds_row_bytes", "attn_update_bounds", "attn_read_bounds",
            "attn_select_blocks", "attn_run_sparse",
            "attn_plan_replayable", "attn_plan_replayable_host",
            "attn_plan_replan_host", "attn_plan_fetch_device")


class attn_problem_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim_qk", ctypes.c_int32),
                ("head_dim_v", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_table_stride", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int), ("window", ctypes.c_int32),
                ("has_sinks", ctypes.c_int32),
                ("qo_indptr_host", ctypes.POINTER(ctypes.c_int32)),
                ("seq_lens_host", ctypes.POINTER(ctypes.c_int32))]


class attn_rope_t(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("max_pos", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("rot_offset", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class attn_mrope_t(ctypes.Structure):
    _fields_ = [("rope", attn_rope_t), ("num_axes", ctypes.c_int32),
                ("pair_axis_host", ctypes.POINTER(ctypes.c_uint8)), ("position_delta", ctypes.c_void_p)]


class attn_sparse_t(ctypes.Structure):
    _fields_ = [("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("first_blocks", ctypes.c_int32), ("last_blocks", ctypes.c_int32)]


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {attn_status_string(status)} ({status})")


_LIB = None
_STAMPS = False      # load the profiling build (attn_debug_stamps records) instead


def library_path() -> str:
    return _build.lib_path(_STAMPS)


def use_stamps_build() -> None:
    """Make load() use the profiling build of the same sources, whose split-KV
    kernel records timestamps (include/attn_paged_debug.h, attn_debug_stamps).
    Call before the library is first loaded."""
    global _STAMPS
    if _LIB is not None and not _STAMPS:
        raise RuntimeError("the default library is already loaded")
    _STAMPS = True


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libattn_paged.so (building it first when missing or stale)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.build(stamps=_STAMPS) if build_if_missing else library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libattn_paged.so not found at {path}")
    L = ctypes.CDLL(path)
    vp, i32p = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)
    L.attn_plan.argtypes = [ctypes.POINTER(attn_problem_t), ctypes.c_int, ctypes.POINTER(vp),
                            ctypes.POINTER(ctypes.c_size_t)]
    L.attn_run_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int32, ctypes.c_float,
                                 ctypes.c_float, ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp]
    L.attn_run_phase.argtypes = [vp, ctypes.c_int32] + L.attn_run_paged.argtypes[1:]
    L.attn_run_paged_no_workspace.argtypes = L.attn_run_paged.argtypes[:14] + [vp]
    L.attn_append_kv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp]
    L.attn_append_kv_rope.argtypes = [vp, ctypes.POINTER(attn_rope_t)] + [vp] * 9 + \
        [ctypes.c_float, ctypes.c_float, vp]
    L.attn_read_kv.argtypes = [vp] * 6 + [ctypes.c_int64, vp, vp, ctypes.c_float, ctypes.c_float, vp]
    L.attn_kv_row_bytes.argtypes = [ctypes.c_int, ctypes.c_int32, i32p]
    L.attn_append_kv_mrope.argtypes = [vp, ctypes.POINTER(attn_mrope_t)] + L.attn_append_kv_rope.argtypes[2:]
    L.attn_bounds_row_bytes.argtypes = [ctypes.c_int32, i32p]
    L.attn_update_bounds.argtypes = [vp, ctypes.c_int32] + [vp] * 5 + [ctypes.c_int64, vp]
    L.attn_read_bounds.argtypes = [vp, ctypes.c_int32] + [vp] * 4 + [ctypes.c_int64, vp, vp]
    L.attn_select_blocks.argtypes = [vp, ctypes.POINTER(attn_sparse_t)] + [vp] * 7
    L.attn_plan_select_ctas.argtypes = [vp, ctypes.POINTER(attn_sparse_t), i32p]
    L.attn_run_sparse.argtypes = [vp, ctypes.POINTER(attn_sparse_t)] + [vp] * 8 + [ctypes.c_float] * 3 + [vp] * 3
    L.attn_plan_destroy.argtypes = [vp]
    L.attn_get_device_error.argtypes = [vp, vp, i32p]
    L.attn_status_string.argtypes = [ctypes.c_int]
    L.attn_status_string.restype = ctypes.c_char_p
    L.attn_plan_host.argtypes = [ctypes.POINTER(attn_problem_t), ctypes.c_int32, ctypes.POINTER(vp)]
    L.attn_plan_info.argtypes = [vp, i32p]
    L.attn_plan_blocks.argtypes = [vp, i32p]
    L.attn_plan_segments.argtypes = [vp, i32p]
    L.attn_plan_replayable.argtypes = L.attn_plan.argtypes
    L.attn_plan_replayable_host.argtypes = L.attn_plan_host.argtypes
    L.attn_plan_replan_host.argtypes = [vp, i32p, i32p]
    L.attn_plan_fetch_device.argtypes = [vp]
    L.attn_debug_tc_gemm.argtypes = [ctypes.c_int32] * 4 + [vp, vp, vp, vp, vp]
    L.attn_debug_stamps.argtypes = [vp, ctypes.c_int32]
    for name in EXPORTED:
        if name != "attn_status_string":
            getattr(L, name).restype = ctypes.c_int
    _LIB = L
    return L


def attn_status_string(status: int) -> str:
    return load().attn_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != ATTN_OK:
        raise AttnError(status, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


_RAW_STREAM = None


def _stream(stream, plan) -> int:
    """The raw handle of `stream`, by default torch's current stream on the plan's
    device (asked for without building a torch.cuda.Stream: 0.1 us for 3)."""
    global _RAW_STREAM
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    if plan.device < 0:          # a host plan: the library refuses to run it
        return 0
    if _RAW_STREAM is None:
        import torch
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _RAW_STREAM(plan.device)


class Plan:
    """Owns an attn_plan_t handle (destroyed with the object)."""

    def __init__(self, handle: int, workspace_bytes: int, device: int, keep, problem: attn_problem_t):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.device = device
        self.total_q = _total_q(problem)         # new tokens of the whole batch
        self.batch = problem.batch
        self.kv_heads = problem.num_kv_heads
        self.head_dim_qk = problem.head_dim_qk
        # bytes of a bounds array, per block size that the pages hold whole
        page = problem.num_pages * problem.num_kv_heads * attn_bounds_row_bytes(problem.head_dim_qk)
        self.bounds_bytes = {b: page * (problem.page_size // b) for b in (16, 32, 64, 128)
                             if problem.page_size % b == 0}
        self._keep = keep

    def destroy(self) -> None:
        if self.handle:
            load().attn_plan_destroy(ctypes.c_void_p(self.handle))
            self.handle = 0

    def __del__(self):
        try:
            self.destroy()
        except Exception:  # interpreter shutdown
            pass


def make_problem(batch, num_q_heads, num_kv_heads, page_size, num_pages, page_table_stride,
                 kv_dtype, window, has_sinks, qo_indptr, seq_lens, head_dim_qk=192,
                 head_dim_v=128):
    """Build an attn_problem_t from host int32 sequences (numpy arrays or lists)."""
    import numpy as np
    qo = np.ascontiguousarray(qo_indptr, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    p = attn_problem_t(batch, num_q_heads, num_kv_heads, head_dim_qk, head_dim_v, page_size,
                       num_pages, page_table_stride, int(kv_dtype), window, int(bool(has_sinks)),
                       qo.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                       sl.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    return p, (qo, sl)


def _total_q(problem: attn_problem_t) -> int:
    """Read once the library has accepted the problem."""
    return problem.qo_indptr_host[problem.batch] if problem.batch > 0 else 0


def attn_plan(problem: attn_problem_t, device: int, keep=None) -> Plan:
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(load().attn_plan(ctypes.byref(problem), int(device), ctypes.byref(h), ctypes.byref(ws)),
           "attn_plan")
    return Plan(h.value, ws.value, device, keep, problem)


def attn_plan_host(problem: attn_problem_t, num_sms: int, keep=None) -> Plan:
    h = ctypes.c_void_p()
    _check(load().attn_plan_host(ctypes.byref(problem), int(num_sms), ctypes.byref(h)),
           "attn_plan_host")
    return Plan(h.value, 0, -1, keep, problem)


def attn_plan_replayable(bounds: attn_problem_t, device: int, keep=None) -> Plan:
    """A plan whose lengths are read on the device at every run (seq_lens in
    `bounds` are upper bounds; the query layout is fixed)."""
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(load().attn_plan_replayable(ctypes.byref(bounds), int(device), ctypes.byref(h),
                                       ctypes.byref(ws)), "attn_plan_replayable")
    return Plan(h.value, ws.value, device, keep, bounds)


def attn_plan_replayable_host(bounds: attn_problem_t, num_sms: int, keep=None) -> Plan:
    h = ctypes.c_void_p()
    _check(load().attn_plan_replayable_host(ctypes.byref(bounds), int(num_sms), ctypes.byref(h)),
           "attn_plan_replayable_host")
    return Plan(h.value, 0, -1, keep, bounds)


def attn_plan_replan_host(plan: Plan, seq_lens) -> int:
    """Rebuild a replayable plan's host work list for `seq_lens`; returns the
    device error bits the lengths would raise."""
    import numpy as np
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    err = ctypes.c_int32()
    _check(load().attn_plan_replan_host(ctypes.c_void_p(plan.handle),
                                        sl.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                        ctypes.byref(err)), "attn_plan_replan_host")
    return err.value


def attn_plan_fetch_device(plan: Plan) -> None:
    """Copy the work list the device planner last wrote into the host copy."""
    _check(load().attn_plan_fetch_device(ctypes.c_void_p(plan.handle)), "attn_plan_fetch_device")


def attn_plan_destroy(plan: Plan) -> None:
    plan.destroy()


def _run_args(plan, q, k_cache, v_cache, page_table, seq_lens, qo_indptr, sinks, window,
              softmax_scale, k_scale, v_scale, out, lse_out, workspace, stream):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seq_lens),
            _ptr(qo_indptr), _ptr(sinks), int(window), float(softmax_scale), float(k_scale),
            float(v_scale), _ptr(out), _ptr(lse_out), _ptr(workspace), ws_bytes,
            _stream(stream, plan))


def attn_run_paged(plan: Plan, q, k_cache, v_cache, page_table, seq_lens, qo_indptr, sinks,
                   window: int, softmax_scale: float, k_scale: float, v_scale: float, out,
                   lse_out=None, workspace=None, stream=None) -> None:
    """Launch on `stream` (a torch.cuda.Stream, a raw handle, or None for torch's
    current stream).  Pointer-only; nothing is synchronised."""
    args = _run_args(plan, q, k_cache, v_cache, page_table, seq_lens, qo_indptr, sinks, window,
                     softmax_scale, k_scale, v_scale, out, lse_out, workspace, stream)
    _check(load().attn_run_paged(plan.handle, *args), "attn_run_paged")


def attn_run_phase(plan: Plan, phase: int, q, k_cache, v_cache, page_table, seq_lens,
                   qo_indptr, sinks, window: int, softmax_scale: float, k_scale: float,
                   v_scale: float, out, lse_out=None, workspace=None, stream=None) -> None:
    """One of the two launches of attn_run_paged (0: split-KV kernel, 1: merge)."""
    args = _run_args(plan, q, k_cache, v_cache, page_table, seq_lens, qo_indptr, sinks, window,
                     softmax_scale, k_scale, v_scale, out, lse_out, workspace, stream)
    _check(load().attn_run_phase(plan.handle, int(phase), *args),
           "attn_run_phase")


NO_WORKSPACE_MAX_BYTES = 16 * 1024 * 1024


def attn_run_paged_no_workspace(plan: Plan, q, k_cache, v_cache, page_table, seq_lens, qo_indptr,
                                sinks, window: int, softmax_scale: float, k_scale: float,
                                v_scale: float, out, lse_out=None, stream=None) -> None:
    """attn_run_paged on the library's own scratch (no workspace argument), for
    callers that cannot allocate device memory."""
    args = _run_args(plan, q, k_cache, v_cache, page_table, seq_lens, qo_indptr, sinks, window,
                     softmax_scale, k_scale, v_scale, out, lse_out, None, stream)
    args = args[:13] + args[15:]        # drop the workspace pointer and size
    _check(load().attn_run_paged_no_workspace(plan.handle, *args),
           "attn_run_paged_no_workspace")


def attn_append_kv(plan: Plan, k_new, v_new, k_cache, v_cache, page_table, seq_lens, qo_indptr,
                   k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Write the plan's new tokens' K/V rows into the paged caches (FP8 caches
    get E4M3 codes of value / scale, 4-bit ones E2M1 codes with block scales)."""
    st = (_LIB or load()).attn_append_kv(
        plan.handle, _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seq_lens),
        _ptr(qo_indptr), float(k_scale), float(v_scale), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_append_kv")


def attn_kv_row_bytes(kv_dtype: int, head_dim: int) -> int:
    """Bytes of one cached row of head_dim values of one KV head."""
    n = ctypes.c_int32()
    _check(load().attn_kv_row_bytes(int(kv_dtype), int(head_dim), ctypes.byref(n)), "attn_kv_row_bytes")
    return n.value


def make_rope(cos_sin, rot_dim: int, rot_offset: int = 0, interleaved: bool = False,
              positions=None) -> attn_rope_t:
    """The rotation of attn_append_kv_rope.  cos_sin: fp32 [max_pos, rot_dim] on the
    device, cosines then sines; positions: int32 [total_q] on the device, or None for
    the tokens' own.  The result keeps both tensors alive.  Shapes and types, which
    the library cannot see, are checked here, once for all steps."""
    import torch
    if cos_sin.dim() != 2 or cos_sin.shape[1] != rot_dim or cos_sin.dtype != torch.float32 or \
            not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous fp32 [max_pos, rot_dim]")
    if positions is not None and (positions.dtype != torch.int32 or not positions.is_contiguous()):
        raise ValueError("positions must be contiguous int32")
    r = attn_rope_t(_ptr(cos_sin), _ptr(positions), int(cos_sin.shape[0]), int(rot_dim),
                    int(rot_offset), int(bool(interleaved)))
    r.keep = (cos_sin, positions)
    return r


def attn_append_kv_rope(plan: Plan, rope: attn_rope_t, q, k_new, v_new, q_out, k_cache, v_cache,
                        page_table, seq_lens, qo_indptr, k_scale: float = 1.0, v_scale: float = 1.0,
                        stream=None) -> None:
    """attn_append_kv with the keys rotated on the way, and the queries into q_out
    (may be q; both None: no queries).  The rope's positions, where given, are
    one per new token of the plan, or more."""
    positions = rope.keep[1] if hasattr(rope, "keep") else None
    if positions is not None and positions.numel() < plan.total_q:
        raise ValueError(f"positions has {positions.numel()} entries for the plan's {plan.total_q} tokens")
    st = (_LIB or load()).attn_append_kv_rope(
        plan.handle, rope, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(q_out), _ptr(k_cache), _ptr(v_cache),
        _ptr(page_table), _ptr(seq_lens), _ptr(qo_indptr), float(k_scale), float(v_scale), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_append_kv_rope")


def attn_read_kv(plan: Plan, k_cache, v_cache, page_table, seq_lens, kv_indptr, k_out, v_out,
                 k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Cached rows as bf16: the last kv_indptr[b + 1] - kv_indptr[b] positions of every
    request b, into k_out [rows, Hkv, Dqk] and v_out [rows, Hkv, 128]."""
    if k_out.shape[0] != v_out.shape[0]:
        raise ValueError(f"k_out has {k_out.shape[0]} rows and v_out {v_out.shape[0]}")
    st = (_LIB or load()).attn_read_kv(
        plan.handle, _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seq_lens), _ptr(kv_indptr),
        k_out.shape[0], _ptr(k_out), _ptr(v_out), float(k_scale), float(v_scale), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_read_kv")


def _contiguous(name: str, t, dtype, shape=None) -> None:
    """What the library cannot see of a tensor that it gets as a pointer."""
    if t.dtype != dtype or not t.is_contiguous() or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be contiguous {dtype}" + (f" {tuple(shape)}" if shape is not None else "") +
                         f", not {t.dtype} {tuple(t.shape)}")


def make_mrope(cos_sin, rot_dim: int, pair_axis, positions=None, position_delta=None, rot_offset: int = 0,
               interleaved: bool = False) -> attn_mrope_t:
    """The rotation of attn_append_kv_mrope: as make_rope, with the axis of every pair in
    pair_axis (rot_dim / 2 numbers, see mrope_axes), positions int32 [num_axes, total_q]
    on the device or None for the tokens' own, then shifted by position_delta (int32
    [batch] on the device) where that is given."""
    import torch
    axes = [int(x) for x in pair_axis]
    if len(axes) != rot_dim // 2 or min(axes, default=0) < 0 or max(axes, default=0) > 255:
        raise ValueError(f"pair_axis must hold rot_dim / 2 = {rot_dim // 2} axes")
    rope = make_rope(cos_sin, rot_dim, rot_offset, interleaved, None)
    num_axes = max(axes, default=0) + 1
    if positions is not None:
        if positions.dim() != 2 or positions.shape[0] < num_axes:
            raise ValueError(f"positions must be [num_axes, total_q] with {num_axes} axes or more")
        _contiguous("positions", positions, torch.int32)
        num_axes = positions.shape[0]
        rope.positions = _ptr(positions)
    if position_delta is not None:
        _contiguous("position_delta", position_delta, torch.int32)
    m = attn_mrope_t(rope, num_axes, (ctypes.c_uint8 * len(axes))(*axes), _ptr(position_delta))
    m.keep = (cos_sin, positions, position_delta)
    return m


def mrope_axes(sections, in_turn: bool = False) -> list:
    """pair_axis for sections[a] pairs of each axis a: one section after the other, or the
    axes in turn until each has had its pairs."""
    if any(n < 0 for n in sections):
        raise ValueError(f"sections must not be negative: {list(sections)}")
    if not in_turn:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def attn_append_kv_mrope(plan: Plan, mrope: attn_mrope_t, q, k_new, v_new, q_out, k_cache, v_cache,
                         page_table, seq_lens, qo_indptr, k_scale: float = 1.0, v_scale: float = 1.0,
                         stream=None) -> None:
    """attn_append_kv_rope with positions of several axes."""
    _, positions, delta = getattr(mrope, "keep", (None, None, None))
    if positions is not None and positions.shape[1] != plan.total_q:
        raise ValueError(f"positions has {positions.shape[1]} columns for the plan's {plan.total_q} tokens")
    if delta is not None and delta.numel() < plan.batch:
        raise ValueError(f"position_delta has {delta.numel()} entries for the plan's {plan.batch} requests")
    st = (_LIB or load()).attn_append_kv_mrope(
        plan.handle, mrope, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(q_out), _ptr(k_cache), _ptr(v_cache),
        _ptr(page_table), _ptr(seq_lens), _ptr(qo_indptr), float(k_scale), float(v_scale), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_append_kv_mrope")


def make_sparse(block_size: int, num_blocks: int, first_blocks: int = 1, last_blocks: int = 1) -> attn_sparse_t:
    """How attn_select_blocks chooses: num_blocks blocks of block_size keys per (token, KV
    head), the first_blocks and last_blocks always among them."""
    return attn_sparse_t(int(block_size), int(num_blocks), int(first_blocks), int(last_blocks))


def attn_bounds_row_bytes(head_dim: int) -> int:
    """Bytes of one block's bounds for one KV head: the last dimension of the bounds array,
    uint8 [num_pages, page_size / block_size, Hkv, bytes]."""
    n = ctypes.c_int32()
    _check(load().attn_bounds_row_bytes(int(head_dim), ctypes.byref(n)), "attn_bounds_row_bytes")
    return n.value


def _bounds_array(plan: Plan, block_size: int, bounds) -> None:
    """Records of another block size, type or order than the call's would be read or written past
    the array's end.  (A missing array, another block size and a host plan the library refuses.)"""
    import torch
    need = plan.bounds_bytes.get(block_size)
    if bounds is None or need is None or plan.device < 0:
        return
    if bounds.dtype != torch.uint8 or not bounds.is_contiguous() or bounds.numel() < need:
        raise ValueError(f"bounds must be contiguous uint8 of {need} bytes for blocks of {block_size}, "
                         f"not {bounds.dtype} {tuple(bounds.shape)}")


def attn_update_bounds(plan: Plan, block_size: int, k_cache, bounds, page_table, seq_lens, kv_indptr,
                       rows: int, stream=None) -> None:
    """Bounds of the blocks that the last kv_indptr[b + 1] - kv_indptr[b] positions of every
    request b complete; rows = kv_indptr[batch]."""
    _bounds_array(plan, block_size, bounds)
    st = (_LIB or load()).attn_update_bounds(
        plan.handle, int(block_size), _ptr(k_cache), _ptr(bounds), _ptr(page_table), _ptr(seq_lens),
        _ptr(kv_indptr), int(rows), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_update_bounds")


def attn_read_bounds(plan: Plan, block_size: int, bounds, page_table, seq_lens, block_indptr, out,
                     stream=None) -> None:
    """The bounds as bf16: the last block_indptr[b + 1] - block_indptr[b] complete blocks of
    every request b, into out [rows, Hkv, 2, Dqk] (upper, lower)."""
    import torch
    if out is None:
        raise ValueError("out is missing")
    _contiguous("out", out, torch.bfloat16)
    if out.numel() != out.shape[0] * plan.kv_heads * 2 * plan.head_dim_qk:
        raise ValueError(f"out must be [rows, {plan.kv_heads}, 2, {plan.head_dim_qk}], not {tuple(out.shape)}")
    _bounds_array(plan, block_size, bounds)
    st = (_LIB or load()).attn_read_bounds(
        plan.handle, int(block_size), _ptr(bounds), _ptr(page_table), _ptr(seq_lens), _ptr(block_indptr),
        out.shape[0], _ptr(out), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_read_bounds")


def _block_lists(plan: Plan, sparse: attn_sparse_t, block_idx) -> None:
    import torch
    _contiguous("block_idx", block_idx, torch.int32)
    if block_idx.numel() != plan.total_q * plan.kv_heads * sparse.num_blocks:
        raise ValueError(f"block_idx has {block_idx.numel()} entries for {plan.total_q} tokens, "
                         f"{plan.kv_heads} KV heads and {sparse.num_blocks} blocks")


def attn_select_blocks(plan: Plan, sparse: attn_sparse_t, q, bounds, page_table, seq_lens, qo_indptr,
                       block_idx, stream=None) -> None:
    """Every new token's blocks into block_idx, int32 [total_q, Hkv, num_blocks]."""
    _block_lists(plan, sparse, block_idx)
    _bounds_array(plan, sparse.block_size, bounds)
    st = (_LIB or load()).attn_select_blocks(
        plan.handle, sparse, _ptr(q), _ptr(bounds), _ptr(page_table), _ptr(seq_lens), _ptr(qo_indptr),
        _ptr(block_idx), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_select_blocks")


def attn_run_sparse(plan: Plan, sparse: attn_sparse_t, q, k_cache, v_cache, page_table, seq_lens, qo_indptr,
                    block_idx, sinks, softmax_scale: float, k_scale: float, v_scale: float, out,
                    lse_out=None, stream=None) -> None:
    """Attention of every new token over the blocks of its lists."""
    _block_lists(plan, sparse, block_idx)
    st = (_LIB or load()).attn_run_sparse(
        plan.handle, sparse, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seq_lens),
        _ptr(qo_indptr), _ptr(block_idx), _ptr(sinks), float(softmax_scale), float(k_scale), float(v_scale),
        _ptr(out), _ptr(lse_out), _stream(stream, plan))
    if st:
        raise AttnError(st, "attn_run_sparse")


def attn_get_device_error(plan: Plan) -> int:
    err = ctypes.c_int32()
    _check(load().attn_get_device_error(ctypes.c_void_p(plan.handle), None, ctypes.byref(err)),
           "attn_get_device_error")
    return err.value


def attn_plan_info(plan: Plan) -> dict:
    info = (ctypes.c_int32 * 8)()
    _check(load().attn_plan_info(ctypes.c_void_p(plan.handle), info), "attn_plan_info")
    return dict(blocks=info[0], segments=info[1], ctas=info[2], rows_per_block=info[3],
                key_tile=info[4], multi_split_blocks=info[5],
                workspace_bytes=(info[7] << 31) | info[6])


def attn_plan_blocks(plan: Plan):
    import numpy as np
    n = attn_plan_info(plan)["blocks"]
    arr = np.zeros((max(n, 1), 8), np.int32)
    _check(load().attn_plan_blocks(ctypes.c_void_p(plan.handle),
                                   arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))),
           "attn_plan_blocks")
    return arr[:n]


def attn_plan_segments(plan: Plan):
    import numpy as np
    n = attn_plan_info(plan)["segments"]
    arr = np.zeros((max(n, 1), 5), np.int32)
    _check(load().attn_plan_segments(ctypes.c_void_p(plan.handle),
                                     arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))),
           "attn_plan_segments")
    return arr[:n]


def attn_plan_cta_heads(plan: Plan):
    """Each CTA's head record as 20 int32 (see attn_plan_cta_heads)."""
    import numpy as np
    n = attn_plan_info(plan)["ctas"]
    arr = np.zeros((max(n, 1), 20), np.int32)
    _check(load().attn_plan_cta_heads(ctypes.c_void_p(plan.handle),
                                      arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))),
           "attn_plan_cta_heads")
    return arr[:n]


def attn_plan_merge_ctas(plan: Plan) -> int:
    """CTAs of the merge kernel a run of `plan` launches (0: none)."""
    n = ctypes.c_int32(0)
    _check(load().attn_plan_merge_ctas(ctypes.c_void_p(plan.handle), ctypes.byref(n)),
           "attn_plan_merge_ctas")
    return n.value


def attn_plan_select_ctas(plan: Plan, sparse: attn_sparse_t) -> int:
    """CTAs of a cluster of the kernel that selects blocks for chunks of tokens (0: the plan's
    tokens are taken one by one)."""
    n = ctypes.c_int32(0)
    _check(load().attn_plan_select_ctas(ctypes.c_void_p(plan.handle), sparse, ctypes.byref(n)),
           "attn_plan_select_ctas")
    return n.value


def attn_plan_stage_units(plan: Plan):
    """A prefill plan's staging units as 8 int32 each (see attn_plan_stage_units)."""
    import numpy as np
    n = ctypes.c_int32(0)
    _check(load().attn_plan_stage_units(ctypes.c_void_p(plan.handle), ctypes.byref(n), None),
           "attn_plan_stage_units")
    arr = np.zeros((max(n.value, 1), 8), np.int32)
    _check(load().attn_plan_stage_units(ctypes.c_void_p(plan.handle), ctypes.byref(n),
                                        arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))),
           "attn_plan_stage_units")
    return arr[:n.value]


def attn_debug_tc_gemm(mode: int, variant: int, ab_type: int, n: int, a, b, d, status,
                       stream=None) -> None:
    """Tensor-core building-block self test (include/attn_paged_debug.h)."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    _check(load().attn_debug_tc_gemm(int(mode), int(variant), int(ab_type), int(n), _ptr(a),
                                     _ptr(b), _ptr(d), _ptr(status), ctypes.c_void_p(int(stream))),
           "attn_debug_tc_gemm")


ATTN_DEBUG_STAMP_CTAS = 160
ATTN_DEBUG_STAMP_EVENTS = 16


def attn_debug_stamps(clear: bool = True):
    """Timestamps of the split-KV kernel's last launches, a
    [ATTN_DEBUG_STAMP_CTAS, ATTN_DEBUG_STAMP_EVENTS] uint64 array (profiling build
    only; the default build raises ATTN_ERR_UNSUPPORTED)."""
    import numpy as np
    arr = np.zeros((ATTN_DEBUG_STAMP_CTAS, ATTN_DEBUG_STAMP_EVENTS), dtype=np.uint64)
    _check(load().attn_debug_stamps(ctypes.c_void_p(arr.ctypes.data), int(bool(clear))),
           "attn_debug_stamps")
    return arr
