"""Python binding of libdash (deterministic attention backward for GB300 / sm_103a).

Argument marshalling only: every computation runs in the library's CUDA
kernels.  The functions named ``dash_*`` mirror the C ABI in include/dash.h
one to one and take torch tensors (device tensors unless stated), passing
their data pointers and the current CUDA stream.  ``attn_fwd`` / ``attn_bwd``
allocate the outputs for convenience.

The library must be built first (``__graft_entry__.build()`` or
``python -m deterministic_attention_backward_fa_gb300._build``); importing a
function without it raises, there is no fallback.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import math
import os

import numpy as np
import torch

from . import _build

SCHEDULES = {"atomic": 0, "serial": 1, "descending_q": 2, "shift": 3, "symmetric_shift": 4}
STATUS = {0: "DASH_OK", 1: "DASH_ERR_INVALID_ARG", 2: "DASH_ERR_UNSUPPORTED", 3: "DASH_ERR_CUDA",
          4: "DASH_ERR_TIMEOUT", 5: "DASH_ERR_NO_MEMORY", 6: "DASH_ERR_SCHEDULE"}
TASK_FIRST = 1 << 28
TASK_LAST = 1 << 29
TASK_RANK_MASK = (1 << 24) - 1

# Launches of this library per backward call: preprocess, main, dQ convert.
KERNELS_PER_BWD = 3
KERNELS_PER_FWD = 1


class DashError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class BwdOptions(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("num_ctas", ctypes.c_int), ("cost_c", ctypes.c_int),
                ("cost_r", ctypes.c_int), ("spin_limit_ns", ctypes.c_longlong),
                ("dq_accum_out", ctypes.c_void_p), ("tasks", ctypes.c_void_p), ("cta_off", ctypes.c_void_p),
                ("main_begin_event", ctypes.c_void_p), ("main_end_event", ctypes.c_void_p),
                ("dq_chains", ctypes.c_int), ("shift_fill", ctypes.c_int), ("trust_table", ctypes.c_int),
                ("trace", ctypes.c_void_p), ("die_aware", ctypes.c_int), ("cluster_size", ctypes.c_int),
                ("shift_split", ctypes.c_int), ("rank_order", ctypes.c_int)]

# Slots of a trace row (dash_bwd_options_t.trace): see include/dash.h.
TRACE_SLOTS = 21


_LIB = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_F = ctypes.c_float

_SIGS = {
    "dash_attn_fwd": ([_P] * 5 + [_I] * 5 + [_F, _P], _I),
    "dash_attn_fwd_ex": ([_P] * 5 + [_I] * 5 + [_F, _I, _P], _I),
    "dash_attn_bwd": ([_P] * 9 + [_I] * 5 + [_F, _I, _P], _I),
    "dash_attn_bwd_ex": ([_P] * 9 + [_I] * 5 + [_F, _I, ctypes.POINTER(BwdOptions), _P], _I),
    "dash_attn_bwd_host": ([_P] * 9 + [_I] * 5 + [_F, _I, _P], _I),
    "dash_attn_bwd_noalloc": ([_P] * 9 + [_I] * 5 + [_F, _I, _P], _I),
    "dash_schedule_num_tasks": ([_I, _I, _I, _I], ctypes.c_longlong),
    "dash_build_schedule": ([_I, _I, _I, _I, _I, _I, _I, _P, _P, ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_build_shift_fill": ([_I] * 7 + [_P, _P, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I),
                                          ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_choose_ctas": ([_I] * 7, _I),
    "dash_build_split_schedule": ([_I] * 8 + [_P, _P, ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_build_schedule_ex": ([_I] * 9 + [_P, _P, ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_choose_split_ctas": ([_I] * 8, _I),
    "dash_choose_split": ([_I] * 8 + [ctypes.POINTER(_I), ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_choose_schedule_split": ([_I] * 6 + [ctypes.POINTER(_I), ctypes.POINTER(_I),
                                               ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_choose_layout": ([_I] * 6 + [ctypes.POINTER(_I)] * 3 + [ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_check_table": ([_I] * 4 + [_P, _P, _I], _I),
    "dash_fit_costs": ([_I] * 4 + [ctypes.c_double] * 2 + [ctypes.POINTER(_I)] * 2, _I),
    "dash_choose_schedule": ([_I] * 6 + [ctypes.POINTER(_I), ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_cluster_latencies": ([_P, _I, _I, _P, _P], _I),
    "dash_place_schedule": ([_P, _P] + [_I] * 5 + [_P, _I, _P, _I, _P, _I, _P, _I, _I, _P, _P], _I),
    "dash_die_map": ([_P, _P, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "dash_cluster_links": ([_P, _P] + [_I] * 5 + [_P, ctypes.POINTER(ctypes.c_longlong)], _I),
    "dash_packed_plan_create": ([_P] + [_I] * 6 + [ctypes.POINTER(_P)], _I),
    "dash_packed_plan_destroy": ([_P], None),
    "dash_packed_plan_spin_limit": ([_P, _L], _I),
    "dash_packed_bwd_workspace": ([_P], _L),
    "dash_build_packed_items": ([_P] + [_I] * 6 + [_P, _P, ctypes.POINTER(_I), ctypes.POINTER(_L)], _I),
    "dash_attn_packed_fwd": ([_P] * 6 + [_L, _P, _F, _P], _I),
    "dash_attn_packed_bwd": ([_P] * 10 + [_L, _P, _F, _P, _L, _P], _I),
    "dash_attn_decode": ([_P] * 7 + [_I] * 7 + [_P, _F, _P, _L, _P], _I),
    "dash_decode_workspace": ([_I] * 5, _L),
    "dash_cache_write": ([_P] * 7 + [_L] + [_I] * 6 + [_P, _P], _I),
    "dash_cache_copy": ([_P] * 4 + [_I] * 5 + [_P, _P], _I),
    "dash_sync_status": ([_P], _I),
    "dash_release_workspace": ([], None),
    "dash_last_error": ([], ctypes.c_char_p),
    "dash_version": ([], _I),
}


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded libdash.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(path)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _LIB = L
    return _LIB


def _check(code: int):
    if code != 0:
        raise DashError(code, lib().dash_last_error().decode())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _shape(q: torch.Tensor):
    if q.dim() != 4:
        raise ValueError("tensors are [B, H, S, D]")
    return tuple(int(x) for x in q.shape)


def _sched(s) -> int:
    return SCHEDULES[s] if isinstance(s, str) else int(s)


# ------------------------------------------------------------ C mirrors
def dash_attn_fwd(q, k, v, o, lse, causal: bool, scale: float, stream=None):
    B, H, S, D = _shape(q)
    bf = torch.bfloat16
    _check(lib().dash_attn_fwd(_dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"), _dev(o, bf, "o"),
                               _dev(lse, torch.float32, "lse"), B, H, S, D, int(causal), float(scale),
                               _stream(stream)))


def dash_attn_fwd_ex(q, k, v, o, lse, causal: bool, scale: float, cta_pair: int = -1, stream=None):
    """``cta_pair``: 0 = one CTA per Q tile, 1 = CTA-pair (cta_group::2) kernel (D = 128), -1 = default."""
    B, H, S, D = _shape(q)
    bf = torch.bfloat16
    _check(lib().dash_attn_fwd_ex(_dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"), _dev(o, bf, "o"),
                                  _dev(lse, torch.float32, "lse"), B, H, S, D, int(causal), float(scale),
                                  int(cta_pair), _stream(stream)))


def dash_attn_bwd(q, k, v, o, do, lse, dq, dk, dv, causal: bool, scale: float, schedule, stream=None):
    B, H, S, D = _shape(q)
    bf = torch.bfloat16
    _check(lib().dash_attn_bwd(_dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"), _dev(o, bf, "o"),
                               _dev(do, bf, "do"), _dev(lse, torch.float32, "lse"), _dev(dq, bf, "dq"),
                               _dev(dk, bf, "dk"), _dev(dv, bf, "dv"), B, H, S, D, int(causal), float(scale),
                               _sched(schedule), _stream(stream)))


def dash_attn_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, causal: bool, scale: float, schedule, tile=0,
                     num_ctas=0, cost_c=0, cost_r=0, spin_limit_ns=0, dq_accum_out=None, tasks=None,
                     cta_off=None, main_events=None, stream=None, dq_chains=0, shift_fill=0, trust_table=0,
                     trace=None, die_aware=0, cluster_size=0, shift_split=0, rank_order=0):
    """``main_events``: optional pair of recorded torch.cuda.Event objects (enable_timing) that the
    library records around the main kernel on the call's stream.  ``dq_chains=2`` splits each dQ
    tile's ordered reduction into two chains by rank parity; ``shift_fill=1`` runs some heads of a
    shift backward with the serial schedule on the SMs that whole gangs leave idle (see
    dash_bwd_options_t).  ``trace``: optional int64 device tensor [n_tasks, TRACE_SLOTS] that the traced
    main kernel fills with per-task phase stamps.  ``die_aware=1`` places each gang of a shift schedule
    on one die with its semaphores homed there; ``cluster_size`` (0 or 1 = none; 2, 4, 8, 16) sets the thread-block
    clusters whose ranks hand the dQ turn over through shared memory; ``shift_split=k`` runs each gang of a
    shift or symmetric-shift schedule as k sub-gangs, and ``shift_split=-1`` lets the library pick k by
    simulated makespan; ``rank_order=1`` reduces each dQ tile in the order the simulated schedule reaches
    it (timed ranks; see dash_bwd_options_t)."""
    B, H, S, D = _shape(q)
    bf = torch.bfloat16
    opt = BwdOptions(tile, num_ctas, cost_c, cost_r, spin_limit_ns, None, None, None, None, None, dq_chains,
                     shift_fill, trust_table)
    if main_events is not None:
        opt.main_begin_event = main_events[0].cuda_event
        opt.main_end_event = main_events[1].cuda_event
    keep = []
    if dq_accum_out is not None:
        opt.dq_accum_out = _dev(dq_accum_out, torch.float32, "dq_accum_out").value
    if trace is not None:
        opt.trace = _dev(trace, torch.int64, "trace").value
    opt.die_aware = die_aware
    opt.cluster_size = cluster_size
    opt.shift_split = shift_split
    opt.rank_order = rank_order
    if tasks is not None:
        t = np.ascontiguousarray(tasks, dtype=np.int32)
        o_ = np.ascontiguousarray(cta_off, dtype=np.int32)
        keep += [t, o_]
        opt.tasks = t.ctypes.data
        opt.cta_off = o_.ctypes.data
        opt.num_ctas = len(o_) - 1
    _check(lib().dash_attn_bwd_ex(_dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"), _dev(o, bf, "o"),
                                  _dev(do, bf, "do"), _dev(lse, torch.float32, "lse"), _dev(dq, bf, "dq"),
                                  _dev(dk, bf, "dk"), _dev(dv, bf, "dv"), B, H, S, D, int(causal),
                                  float(scale), _sched(schedule), ctypes.byref(opt), _stream(stream)))


def dash_attn_bwd_host(q, k, v, o, do, lse, dq, dk, dv, causal: bool, scale: float, schedule, stream=None):
    """All tensors are CPU tensors (pinned for full copy bandwidth); blocks until dq/dk/dv are filled."""
    B, H, S, D = _shape(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do), ("lse", lse), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor")
    _check(lib().dash_attn_bwd_host(*(ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, o, do, lse, dq, dk, dv)),
                                    B, H, S, D, int(causal), float(scale), _sched(schedule), _stream(stream)))


def dash_attn_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, causal: bool, scale: float, schedule, stream=None):
    """dash_attn_bwd without device allocation (fixed 32 MiB library-owned workspace; synchronises)."""
    B, H, S, D = _shape(q)
    bf = torch.bfloat16
    _check(lib().dash_attn_bwd_noalloc(_dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"), _dev(o, bf, "o"),
                                       _dev(do, bf, "do"), _dev(lse, torch.float32, "lse"), _dev(dq, bf, "dq"),
                                       _dev(dk, bf, "dk"), _dev(dv, bf, "dv"), B, H, S, D, int(causal),
                                       float(scale), _sched(schedule), _stream(stream)))


def dash_schedule_num_tasks(BH: int, n: int, causal: bool, schedule) -> int:
    return int(lib().dash_schedule_num_tasks(BH, n, int(causal), _sched(schedule)))


def dash_build_schedule(BH: int, n: int, causal: bool, schedule, P: int, cost_c: int = 4, cost_r: int = 1):
    """Host-only.  Returns (tasks int32 [N, 4], cta_off int32 [P+1], makespan)."""
    nt = dash_schedule_num_tasks(BH, n, causal, schedule)
    if nt < 0:
        raise DashError(2, "schedule invalid for this mask / n")
    tasks = np.zeros((max(nt, 1), 4), dtype=np.int32)
    off = np.zeros(P + 1, dtype=np.int32)
    ms = ctypes.c_longlong(0)
    _check(lib().dash_build_schedule(BH, n, int(causal), _sched(schedule), P, cost_c, cost_r,
                                     tasks.ctypes.data_as(ctypes.c_void_p), off.ctypes.data_as(ctypes.c_void_p),
                                     ctypes.byref(ms)))
    return tasks[:nt], off, int(ms.value)


def dash_build_shift_fill(BH: int, n: int, causal: bool, schedule, max_ctas: int, cost_c: int = 4, cost_r: int = 1):
    """Host-only.  Returns (tasks int32 [N, 4], cta_off int32 [P+1], P, shift_heads, fill schedule name or
    None, makespan)."""
    nt = dash_schedule_num_tasks(BH, n, causal, schedule)
    if nt < 0:
        raise DashError(2, "schedule invalid for this mask / n")
    tasks = np.zeros((max(nt, 1), 4), dtype=np.int32)
    off = np.zeros(max_ctas + 1, dtype=np.int32)
    P, hs, fm, ms = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(-1), ctypes.c_longlong(0)
    _check(lib().dash_build_shift_fill(BH, n, int(causal), _sched(schedule), max_ctas, cost_c, cost_r,
                                       tasks.ctypes.data_as(ctypes.c_void_p), off.ctypes.data_as(ctypes.c_void_p),
                                       ctypes.byref(P), ctypes.byref(hs), ctypes.byref(fm), ctypes.byref(ms)))
    fill = next(k for k, v in SCHEDULES.items() if v == fm.value) if fm.value >= 0 else None
    return tasks[:nt], off[:P.value + 1], int(P.value), int(hs.value), fill, int(ms.value)


def dash_check_table(BH: int, n: int, causal: bool, tasks, cta_off, dq_chains: int = 0):
    """Host-only.  Raises DashError (code 6) if the table's dQ orders could not finish."""
    t = np.ascontiguousarray(tasks, dtype=np.int32).reshape(-1, 4)
    o = np.ascontiguousarray(cta_off, dtype=np.int32)
    _check(lib().dash_check_table(BH, n, int(causal), dq_chains, t.ctypes.data_as(ctypes.c_void_p),
                                  o.ctypes.data_as(ctypes.c_void_p), len(o) - 1))


def dash_fit_costs(BH: int, n: int, causal: bool, max_ctas: int, atomic_ms: float, serial_ms: float):
    """Host-only.  Returns (cost_c, cost_r) fitted to the measured atomic and serial times."""
    c, r = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().dash_fit_costs(BH, n, int(causal), max_ctas, float(atomic_ms), float(serial_ms), ctypes.byref(c),
                                ctypes.byref(r)))
    return int(c.value), int(r.value)


def dash_choose_ctas(BH: int, n: int, causal: bool, schedule, max_ctas: int, cost_c: int = 4, cost_r: int = 1):
    return int(lib().dash_choose_ctas(BH, n, int(causal), _sched(schedule), max_ctas, cost_c, cost_r))


def dash_build_schedule_ex(BH: int, n: int, causal: bool, schedule, split: int, rank_order: int, P: int,
                           cost_c: int = 4, cost_r: int = 1):
    """Host-only tables with split gangs and / or timed ranks.  Returns (tasks int32 [N, 4], cta_off int32 [P+1],
    makespan)."""
    nt = dash_schedule_num_tasks(BH, n, causal, schedule)
    if nt < 0:
        raise DashError(2, "schedule invalid for this mask / n")
    tasks = np.zeros((max(nt, 1), 4), dtype=np.int32)
    off = np.zeros(P + 1, dtype=np.int32)
    ms = ctypes.c_longlong(0)
    _check(lib().dash_build_schedule_ex(BH, n, int(causal), _sched(schedule), split, rank_order, P, cost_c, cost_r,
                                        tasks.ctypes.data, off.ctypes.data, ctypes.byref(ms)))
    return tasks[:nt], off, ms.value


def dash_build_split_schedule(BH: int, n: int, causal: bool, schedule, split: int, P: int, cost_c: int = 4,
                              cost_r: int = 1):
    """Host-only split-gang tables (an extension).  Returns (tasks int32 [N, 4], cta_off int32 [P+1], makespan)."""
    nt = dash_schedule_num_tasks(BH, n, causal, schedule)
    if nt < 0:
        raise DashError(2, "schedule invalid for this mask / n")
    tasks = np.zeros((max(nt, 1), 4), dtype=np.int32)
    off = np.zeros(P + 1, dtype=np.int32)
    ms = ctypes.c_longlong(0)
    _check(lib().dash_build_split_schedule(BH, n, int(causal), _sched(schedule), split, P, cost_c, cost_r,
                                           tasks.ctypes.data, off.ctypes.data, ctypes.byref(ms)))
    return tasks[:nt], off, ms.value


def dash_choose_split(BH: int, n: int, causal: bool, schedule, max_ctas: int, num_ctas: int = 0, cost_c: int = 4,
                      cost_r: int = 1):
    """Host-only.  The split that ``shift_split=-1`` picks: returns (k, CTA count, simulated makespan), k = -1
    where split gangs do not apply."""
    P, ms = _I(0), ctypes.c_longlong(0)
    k = lib().dash_choose_split(BH, n, int(causal), _sched(schedule), max_ctas, num_ctas, cost_c, cost_r,
                                ctypes.byref(P), ctypes.byref(ms))
    return int(k), P.value, ms.value


def dash_choose_split_ctas(BH: int, n: int, causal: bool, schedule, split: int, max_ctas: int, cost_c: int = 4,
                           cost_r: int = 1):
    return int(lib().dash_choose_split_ctas(BH, n, int(causal), _sched(schedule), split, max_ctas, cost_c, cost_r))


def dash_choose_schedule_split(BH: int, n: int, causal: bool, max_ctas: int, cost_c: int = 4, cost_r: int = 1):
    """Host-only.  ``dash_choose_schedule`` with split gangs among the candidates.  Returns (schedule name, CTA
    count, split, simulated makespan)."""
    P, k, ms = _I(0), _I(0), ctypes.c_longlong(0)
    s = lib().dash_choose_schedule_split(BH, n, int(causal), max_ctas, cost_c, cost_r, ctypes.byref(P),
                                         ctypes.byref(k), ctypes.byref(ms))
    if s < 0:
        raise DashError(1, dash_last_error())
    return {v: k_ for k_, v in SCHEDULES.items()}[s], P.value, k.value, ms.value


def dash_choose_layout(BH: int, n: int, causal: bool, max_ctas: int, cost_c: int = 4, cost_r: int = 1):
    """Host-only.  The runtime choice over every deterministic layout: returns (schedule name, CTA count, split,
    rank_order, simulated makespan)."""
    P, k, ro, ms = _I(0), _I(0), _I(0), ctypes.c_longlong(0)
    s = lib().dash_choose_layout(BH, n, int(causal), max_ctas, cost_c, cost_r, ctypes.byref(P), ctypes.byref(k),
                                 ctypes.byref(ro), ctypes.byref(ms))
    if s < 0:
        raise DashError(1, dash_last_error())
    return {v: k_ for k_, v in SCHEDULES.items()}[s], P.value, k.value, ro.value, ms.value


def dash_choose_schedule(BH: int, n: int, causal: bool, max_ctas: int, cost_c: int = 4, cost_r: int = 1):
    """Host-only.  Returns (schedule name, CTA count, simulated makespan) of the
    deterministic schedule with the smallest simulated makespan."""
    P, ms = _I(0), ctypes.c_longlong(0)
    s = lib().dash_choose_schedule(BH, n, int(causal), max_ctas, cost_c, cost_r, ctypes.byref(P), ctypes.byref(ms))
    if s < 0:
        raise DashError(1, dash_last_error())
    return {v: k for k, v in SCHEDULES.items()}[s], P.value, ms.value


def dash_cluster_latencies(lat):
    """Host-only.  lat: [n_sms, n_lines] latencies (clocks).  Returns (group per SM, home per line)."""
    L = np.ascontiguousarray(lat, dtype=np.uint32)
    g = np.zeros(L.shape[0], dtype=np.int32)
    h = np.zeros(L.shape[1], dtype=np.int32)
    _check(lib().dash_cluster_latencies(L.ctypes.data_as(ctypes.c_void_p), L.shape[0], L.shape[1],
                                        g.ctypes.data_as(ctypes.c_void_p), h.ctypes.data_as(ctypes.c_void_p)))
    return g, h


def dash_place_schedule(tasks, cta_off, gang: int, BH: int, n: int, chains: int, smids, lines, max_smid: int):
    """Host-only.  smids, lines: pairs of int lists (group 0, group 1).  Returns (slot_of_smid, sem_idx)."""
    t = np.ascontiguousarray(tasks, dtype=np.int32).reshape(-1, 4)
    o = np.ascontiguousarray(cta_off, dtype=np.int32)
    a = [np.ascontiguousarray(x, dtype=np.int32) for x in (*smids, *lines)]
    slot = np.zeros(max_smid + 1, dtype=np.int32)
    sem = np.zeros(BH * n * chains, dtype=np.int32)
    p = lambda x: x.ctypes.data_as(ctypes.c_void_p)
    _check(lib().dash_place_schedule(p(t), p(o), len(o) - 1, gang, BH, n, chains, p(a[0]), len(a[0]), p(a[1]),
                                     len(a[1]), p(a[2]), len(a[2]), p(a[3]), len(a[3]), max_smid, p(slot), p(sem)))
    return slot, sem


def dash_cluster_links(tasks, cta_off, C: int, BH: int, n: int, chains: int = 1):
    """Host-only.  Returns (link word per task, number of linked hand-offs) for clusters of C."""
    t = np.ascontiguousarray(tasks, dtype=np.int32).reshape(-1, 4)
    o = np.ascontiguousarray(cta_off, dtype=np.int32)
    out = np.zeros(len(t), dtype=np.int32)
    k = ctypes.c_longlong(0)
    _check(lib().dash_cluster_links(t.ctypes.data_as(ctypes.c_void_p), o.ctypes.data_as(ctypes.c_void_p),
                                    len(o) - 1, C, BH, n, chains, out.ctypes.data_as(ctypes.c_void_p),
                                    ctypes.byref(k)))
    return out, int(k.value)


def dash_die_map(max_sm: int = 1023, stream=None):
    """The device's SM groups as the stream's workspace measures them: (group per SM id, -1 for ids the
    device does not have; n0, n1)."""
    g = np.zeros(max_sm + 1, dtype=np.int32)
    n0, n1 = _I(0), _I(0)
    _check(lib().dash_die_map(_stream(stream), g.ctypes.data_as(ctypes.c_void_p), max_sm, ctypes.byref(n0),
                              ctypes.byref(n1)))
    return g, n0.value, n1.value


# ---- packed, grouped-head attention and the paged cache
def _stream_on(device, stream):
    """The raw stream to run on: the given one, or ``device``'s current one."""
    if stream is None:  # without the Stream object that torch.cuda.current_stream makes: 0.1 us a call against 2
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, not to {device}")
    return stream.cuda_stream


_HERE = contextlib.nullcontext()


def _device(dev):
    """Makes ``dev`` current, at no cost when it is already."""
    return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _rows(name, t, heads, dim, rows, device):
    """Checks a [rows, heads, D] bf16 tensor whose last dimension is contiguous (None: any extent)."""
    shape = t.shape
    if len(shape) != 3 or t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(2) != 1 or \
            (heads is not None and shape[1] != heads) or (dim is not None and shape[2] != dim) or \
            (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} must be a CUDA torch.bfloat16 tensor [{'rows' if rows is None else rows}, "
                         f"{heads or 'heads'}, {dim or 'D'}], contiguous in its last dimension, not {t.dtype} "
                         f"{list(shape)} on {t.device} with strides {t.stride()}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _plain(name, t, dtype, shape, device):
    """A contiguous CUDA tensor of the given type and shape (None: any extent)."""
    if t.dtype != dtype or (t.shape != shape and (
            len(t.shape) != len(shape) or any(b is not None and a != b for a, b in zip(t.shape, shape)))):
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)}, not {t.dtype} {list(t.shape)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous on {device}")
    return t


def _strides(*tensors):
    """Row and head strides, or None when every tensor is contiguous."""
    if all([t.is_contiguous() for t in tensors]):
        return None
    v = [x for t in tensors for x in t.stride()[:2]]
    return (ctypes.c_int64 * len(v))(*v)


class PackedPlan:
    """Tables of one set of sequence lengths (host ints) on a GPU, for ``heads`` Q heads that share ``kv_heads``
    K/V heads: made once per batch, used by every layer's ``attn_packed_fwd`` and, with ``backward=True``,
    ``attn_packed_bwd``.  Read-only once made; keep it while work that uses it (replays of captured graphs
    included) may still run.  ``spin_limit_ns`` bounds each device wait (0: 2 s)."""

    def __init__(self, lengths, heads: int, kv_heads: int, head_dim: int, causal: bool = True,
                 backward: bool = False, device=None, spin_limit_ns: int = 0):
        self._handle = None
        values = lengths.tolist() if hasattr(lengths, "tolist") else list(lengths)
        self.lengths = tuple(int(x) for x in values)
        self.heads, self.kv_heads, self.head_dim, self.causal = int(heads), int(kv_heads), int(head_dim), bool(causal)
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("a plan needs a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(self.device):
            self._handle = dash_packed_plan_create(self.lengths, self.heads, self.kv_heads, self.head_dim,
                                                   self.causal, backward)
        dash_packed_plan_spin_limit(self._handle, spin_limit_ns)
        self.rows = sum(self.lengths)
        self.workspace_bytes = dash_packed_bwd_workspace(self._handle) if backward else -1

    def __del__(self):
        if getattr(self, "_handle", None) is not None and _LIB is not None:
            dash_packed_plan_destroy(self._handle)
            self._handle = None


def _handle(plan):
    return plan._handle if isinstance(plan, PackedPlan) else plan


def dash_packed_plan_create(lengths, heads: int, kv_heads: int, head_dim: int, causal: bool, backward: bool):
    """The plan's handle on the current device (``PackedPlan`` owns one and frees it)."""
    if any(not -2**31 <= x < 2**31 for x in lengths):
        raise ValueError("lengths must fit 32 bits")
    arr = (ctypes.c_int32 * max(len(lengths), 1))(*lengths)
    out = _P()
    _check(lib().dash_packed_plan_create(arr, len(lengths), heads, kv_heads, head_dim, int(causal), int(backward),
                                         ctypes.byref(out)))
    return out


def dash_packed_plan_destroy(plan):
    lib().dash_packed_plan_destroy(_handle(plan))


def dash_packed_plan_spin_limit(plan, ns: int):
    _check(lib().dash_packed_plan_spin_limit(_handle(plan), ns))


def dash_packed_bwd_workspace(plan) -> int:
    return int(lib().dash_packed_bwd_workspace(_handle(plan)))


def dash_build_packed_items(lengths, heads: int, kv_heads: int, causal: bool, kernel: int, P: int):
    """Host-only.  The items of the forward (kernel 0), dQ (1) or dK and dV (2): (int32 [N, 16, 8 or 12], cta_off)."""
    arr = (ctypes.c_int32 * max(len(lengths), 1))(*lengths)
    n, ctas = _L(0), _I(0)
    head = (arr, len(lengths), heads, kv_heads, int(causal), kernel, P)
    _check(lib().dash_build_packed_items(*head, None, None, ctypes.byref(ctas), ctypes.byref(n)))
    items = np.zeros((max(n.value, 1), (16, 8, 12)[kernel]), dtype=np.int32)
    off = np.zeros(ctas.value + 1, dtype=np.int32)
    _check(lib().dash_build_packed_items(*head, items.ctypes.data, off.ctypes.data, None, ctypes.byref(n)))
    return items[:n.value], off


def _packed_fwd(plan, q, k, v, o, lse, scale, stream):
    dev = plan.device
    with _device(dev):
        _check(lib().dash_attn_packed_fwd(plan._handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                          lse.data_ptr(), q.shape[0], _strides(q, k, v, o), scale,
                                          _stream_on(dev, stream)))


def _packed_inputs(plan, q, k, v):
    dev, dim = plan.device, plan.head_dim
    _rows("q", q, plan.heads, dim, None, dev)
    _rows("k", k, plan.kv_heads, dim, q.shape[0], dev)
    _rows("v", v, plan.kv_heads, dim, q.shape[0], dev)


def dash_attn_packed_fwd(plan: PackedPlan, q, k, v, o, lse, scale: float, stream=None):
    _packed_inputs(plan, q, k, v)
    _rows("o", o, plan.heads, plan.head_dim, q.shape[0], plan.device)
    _plain("lse", lse, torch.float32, (plan.heads, q.shape[0]), plan.device)
    _packed_fwd(plan, q, k, v, o, lse, float(scale), stream)


def _packed_bwd(plan, q, k, v, o, do, lse, dq, dk, dv, scale, workspace, stream):
    dev = plan.device
    with _device(dev):
        _check(lib().dash_attn_packed_bwd(plan._handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                          do.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                          q.shape[0], _strides(q, k, v, o, do, dq, dk, dv), scale,
                                          workspace.data_ptr(), workspace.numel(), _stream_on(dev, stream)))


def _packed_saved(plan, q, o, do, lse):
    dev, rows = plan.device, q.shape[0]
    _rows("o", o, plan.heads, plan.head_dim, rows, dev)
    _rows("do", do, plan.heads, plan.head_dim, rows, dev)
    _plain("lse", lse, torch.float32, (plan.heads, rows), dev)


def dash_attn_packed_bwd(plan: PackedPlan, q, k, v, o, do, lse, dq, dk, dv, scale: float, workspace, stream=None):
    dev, rows = plan.device, q.shape[0]
    _packed_inputs(plan, q, k, v)
    _packed_saved(plan, q, o, do, lse)
    _rows("dq", dq, plan.heads, plan.head_dim, rows, dev)
    _rows("dk", dk, plan.kv_heads, plan.head_dim, rows, dev)
    _rows("dv", dv, plan.kv_heads, plan.head_dim, rows, dev)
    _plain("workspace", workspace, torch.uint8, (None,), dev)
    _packed_bwd(plan, q, k, v, o, do, lse, dq, dk, dv, float(scale), workspace, stream)


def _cache(k_pages, v_pages, device):
    shape = k_pages.shape
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or len(t.shape) != 4 or t.stride(3) != 1:
            raise ValueError(f"{name} must be a CUDA bfloat16 tensor [pages, tokens, heads, D], contiguous in D")
        if device is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
    if shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    return shape


def _cache_strides(a, b, k_pages, v_pages, table):
    """The strides of two row tensors, the cache and the page table, or None when all are contiguous."""
    if all([t.is_contiguous() for t in (a, b, k_pages, v_pages, table)]):
        return None
    v = (*a.stride()[:2], *b.stride()[:2], *k_pages.stride()[:3], *v_pages.stride()[:3], table.stride(0))
    return (ctypes.c_int64 * 11)(*v)


def _table(page_table, n_seqs, device):
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != n_seqs:
        raise ValueError(f"page_table must be int32 [{n_seqs}, pages]")
    if page_table.device != device or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError(f"page_table must lie on {device} with contiguous rows")


@functools.lru_cache(maxsize=64)
def dash_decode_workspace(B: int, heads: int, head_dim: int, page_size: int, max_pages: int) -> int:
    return int(lib().dash_decode_workspace(B, heads, head_dim, page_size, max_pages))


def _decode(q, k_pages, v_pages, page_table, lengths, o, lse, scale, workspace, stream):
    dev = q.device
    n_pages, page, hkv, D = k_pages.shape
    with _device(dev):
        _check(lib().dash_attn_decode(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                                      lengths.data_ptr(), o.data_ptr(), None if lse is None else lse.data_ptr(),
                                      q.shape[0], q.shape[1], hkv, D, n_pages, page, page_table.shape[1],
                                      _cache_strides(q, o, k_pages, v_pages, page_table), scale,
                                      None if workspace is None else workspace.data_ptr(),
                                      0 if workspace is None else workspace.numel(), _stream_on(dev, stream)))


def _decode_inputs(q, k_pages, v_pages, page_table, lengths):
    _rows("q", q, None, None, None, None)
    dev, B = q.device, q.shape[0]
    if _cache(k_pages, v_pages, dev)[3] != q.shape[2]:
        raise ValueError(f"q has head dimension {q.shape[2]}, the cache {k_pages.shape[3]}")
    _table(page_table, B, dev)
    _plain("lengths", lengths, torch.int32, (B,), dev)


def dash_attn_decode(q, k_pages, v_pages, page_table, lengths, o, lse, scale: float, workspace=None, stream=None):
    """``lse`` may be None; ``workspace`` as dash_decode_workspace asks for (uint8)."""
    _decode_inputs(q, k_pages, v_pages, page_table, lengths)
    dev = q.device
    _rows("o", o, q.shape[1], q.shape[2], q.shape[0], dev)
    if lse is not None:
        _plain("lse", lse, torch.float32, (q.shape[0], q.shape[1]), dev)
    if workspace is not None:
        _plain("workspace", workspace, torch.uint8, (None,), dev)
    _decode(q, k_pages, v_pages, page_table, lengths, o, lse, float(scale), workspace, stream)


def dash_cache_write(k, v, k_pages, v_pages, page_table, starts, cu_new, stream=None):
    dev = k.device
    n_pages, page, hkv, D = _cache(k_pages, v_pages, dev)
    _rows("k", k, hkv, D, None, None)
    _rows("v", v, hkv, D, k.shape[0], dev)
    _plain("starts", starts, torch.int32, (None,), dev)
    B = starts.shape[0]
    _plain("cu_new", cu_new, torch.int32, (B + 1,), dev)
    _table(page_table, B, dev)
    with _device(dev):
        _check(lib().dash_cache_write(k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                      page_table.data_ptr(), starts.data_ptr(), cu_new.data_ptr(), k.shape[0], B, hkv,
                                      D, n_pages, page, page_table.shape[1],
                                      _cache_strides(k, v, k_pages, v_pages, page_table), _stream_on(dev, stream)))


def dash_cache_copy(k_pages, v_pages, src, dst, stream=None):
    """``src``, ``dst``: page numbers on the host (lists, arrays or CPU tensors)."""
    n_pages, page, hkv, D = _cache(k_pages, v_pages, k_pages.device)
    s, d = (array.array("i", x if isinstance(x, (list, tuple)) else x.tolist()) for x in (src, dst))
    if len(s) != len(d):
        raise ValueError("src and dst must have the same length")
    dev, strides = k_pages.device, None
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        strides = (ctypes.c_int64 * 6)(*k_pages.stride()[:3], *v_pages.stride()[:3])
    with _device(dev):
        _check(lib().dash_cache_copy(k_pages.data_ptr(), v_pages.data_ptr(), s.buffer_info()[0], d.buffer_info()[0],
                                     len(s), hkv, D, n_pages, page, strides, _stream_on(dev, stream)))


def dash_sync_status(stream=None):
    _check(lib().dash_sync_status(_stream(stream)))


def dash_release_workspace():
    lib().dash_release_workspace()


def dash_last_error() -> str:
    return lib().dash_last_error().decode()


def dash_version() -> int:
    return int(lib().dash_version())


# ------------------------------------------------------------ conveniences
# The packed and paged ones take a ``stream`` to run on that waits for what the current stream holds by then; the
# caller makes the current stream wait for it before it uses the results.  The dash_ forms do not wait.
@contextlib.contextmanager
def _side(stream, tensors):
    stream.wait_stream(torch.cuda.current_stream(stream.device))
    with torch.cuda.stream(stream):
        yield
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _using(stream, *tensors):
    """Runs torch's own work on ``stream`` if one is given, which waits for the current stream's work so far, and
    tells the allocator that it uses the tensors, inputs and outputs: what the caller drops once the call has
    returned is not handed out again before the stream has passed."""
    return _HERE if stream is None else _side(stream, tensors)


def attn_fwd(q, k, v, causal: bool, scale: float | None = None, stream=None, cta_pair: int = -1):
    """O (bf16) and LSE (fp32, natural log) of softmax attention."""
    B, H, S, D = _shape(q)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    if cta_pair == -1:
        dash_attn_fwd(q, k, v, o, lse, causal, scale, stream)
    else:
        dash_attn_fwd_ex(q, k, v, o, lse, causal, scale, cta_pair, stream)
    return o, lse


def attn_bwd(q, k, v, o, do, lse, causal: bool, scale: float | None = None, schedule="serial",
             dq_accum: bool = False, stream=None, **opts):
    """dQ, dK, dV (bf16); with ``dq_accum`` also the unscaled fp32 dQ accumulator."""
    B, H, S, D = _shape(q)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    acc = torch.empty(q.shape, dtype=torch.float32, device=q.device) if dq_accum else None
    if acc is None and not opts:
        dash_attn_bwd(q, k, v, o, do, lse, dq, dk, dv, causal, scale, schedule, stream)
    else:
        dash_attn_bwd_ex(q, k, v, o, do, lse, dq, dk, dv, causal, scale, schedule, dq_accum_out=acc,
                         stream=stream, **opts)
    return (dq, dk, dv, acc) if dq_accum else (dq, dk, dv)


def attn_packed_fwd(plan: PackedPlan, q, k, v, scale: float | None = None, stream=None):
    """O [rows, heads, D] (bf16) and LSE [heads, rows] (fp32) of attention over the plan's packed sequences.  Rows
    behind the last sequence are zero (-inf in LSE)."""
    _packed_inputs(plan, q, k, v)
    scale = 1.0 / math.sqrt(plan.head_dim) if scale is None else float(scale)
    rows = q.shape[0]
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty((plan.heads, rows), dtype=torch.float32, device=q.device)
    with _using(stream, q, k, v, o, lse):
        _packed_fwd(plan, q, k, v, o, lse, scale, stream)
        if rows > plan.rows:
            o[plan.rows:].zero_()
            lse[:, plan.rows:].fill_(float("-inf"))
    return o, lse


def attn_packed_bwd(plan: PackedPlan, q, k, v, o, do, lse, scale: float | None = None, stream=None):
    """dQ [rows, heads, D], dK, dV [rows, kv_heads, D] (bf16); zero behind the last sequence."""
    _packed_inputs(plan, q, k, v)
    _packed_saved(plan, q, o, do, lse)
    scale = 1.0 / math.sqrt(plan.head_dim) if scale is None else float(scale)
    rows, kv_shape = q.shape[0], (q.shape[0], plan.kv_heads, plan.head_dim)
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dk = torch.empty(kv_shape, dtype=q.dtype, device=q.device)
    dv = torch.empty(kv_shape, dtype=q.dtype, device=q.device)
    ws = torch.empty(max(plan.workspace_bytes, 0), dtype=torch.uint8, device=q.device)
    with _using(stream, q, k, v, o, do, lse, dq, dk, dv, ws):
        _packed_bwd(plan, q, k, v, o, do, lse, dq, dk, dv, scale, ws, stream)
        if rows > plan.rows:
            for t in (dq, dk, dv):
                t[plan.rows:].zero_()
    return dq, dk, dv


def attn_decode(q, k_pages, v_pages, page_table, lengths, scale: float | None = None, stream=None):
    """O [B, heads, D] (bf16) and LSE [B, heads] (fp32) of one new token per sequence over a paged cache."""
    _decode_inputs(q, k_pages, v_pages, page_table, lengths)
    B, heads, dim = q.shape
    scale = 1.0 / math.sqrt(dim) if scale is None else float(scale)
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty((B, heads), dtype=torch.float32, device=q.device)
    need = dash_decode_workspace(B, heads, dim, k_pages.shape[1], page_table.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 0 else None
    with _using(stream, q, k_pages, v_pages, page_table, lengths, o, lse, ws):
        _decode(q, k_pages, v_pages, page_table, lengths, o, lse, scale, ws, stream)
    return o, lse


def cache_write(k, v, k_pages, v_pages, page_table, starts, cu_new, stream=None):
    """Writes new tokens' K and V rows into the pages of their sequences, in place (see dash_cache_write)."""
    with _using(stream, k, v, k_pages, v_pages, page_table, starts, cu_new):
        dash_cache_write(k, v, k_pages, v_pages, page_table, starts, cu_new, stream)


def cache_copy(k_pages, v_pages, src, dst, stream=None):
    """Copies pages ``src`` to pages ``dst`` (host page numbers) inside the cache, in place."""
    with _using(stream, k_pages, v_pages):
        dash_cache_copy(k_pages, v_pages, src, dst, stream)
