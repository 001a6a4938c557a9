"""ctypes binding of libmoe_arena.so -- argument marshalling only.

Every function here has the name and argument order of the C entry point it
wraps (include/moe_arena.h) and returns that entry point's status code.
Pointer arguments accept an int address, None (NULL) or any object with a
data_ptr() method (a torch tensor); stream arguments accept an int handle,
None (the null stream) or an object with a cuda_stream attribute (a torch
stream); event arguments accept an int, None or an object with cuda_event.
No computation of the layer happens in Python.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_arena.so")

MOE_OK = 0
MOE_EINVAL = -1
MOE_EUNSUPPORTED = -2
MOE_EWORKSPACE = -3
MOE_EHIP = -4
MOE_ESCRATCH = -5
MOE_EIO = -6
MOE_EFORMAT = -7
MOE_NOALLOC_SCRATCH_BYTES = 16 << 20
MOE_OP_ROUTE = 0
MOE_OP_DEMAND = 1
MOE_OP_EXPERTS = 2
MOE_OP_HOT_PICK = 3
MOE_OP_EXPERTS_SHARED = 4
MOE_OP_ACT_MXFP6 = 0x10
MOE_ACT_MXFP4 = 0
MOE_ACT_MXFP6 = 1
MOE_DT_BF16 = 0
MOE_DT_FP16 = 1
MOE_DT_FP32 = 2
MOE_INT_MAX = 2 ** 31 - 1
MOE_MAX_E = 1024
MOE_MAX_K = 32
MOE_MAX_S = 8192
MOE_MAX_RING_PAIRS = 16384
MOE_MAX_RING = 1024
MOE_MAX_RING_PER_STEP = 64

EXPORTS = ("moe_status_string", "moe_mxfp4_row_bytes", "moe_act_row_bytes", "moe_slot_bytes",
           "moe_slot_sections",
           "moe_workspace_bytes", "moe_route", "moe_demand_accumulate", "moe_experts_forward",
           "moe_experts_forward_noalloc", "moe_ring_plan", "moe_ring_install",
           "moe_history_save", "moe_history_load", "moe_boot_plan", "moe_history_scale",
           "moe_positions", "moe_dispatch", "moe_dispatch_backward", "moe_combine",
           "moe_combine_backward", "moe_int8_row_bytes", "moe_int8_quantize", "moe_int8_matmul",
           "moe_grouped_matmul", "moe_grouped_outer", "moe_grouped_outer_ws_bytes",
           "moe_swiglu_backward",
           "moe_int4_code_bytes", "moe_int4_scale_count", "moe_int4_quantize", "moe_int4_matmul",
           "arena_load_slot", "moe_hot_pick", "moe_hot_install", "moe_replan", "moe_test_mxfp4_probe",
           "moe_test_stream_read", "moe_test_mfma_loop")


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class RouteArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("E", ctypes.c_int),
                ("k", ctypes.c_int), ("S", ctypes.c_int),
                ("x", ctypes.c_void_p), ("w_router", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("expert_slot", ctypes.c_void_p), ("topk_expert", ctypes.c_void_p),
                ("topk_score", ctypes.c_void_p), ("sel_expert", ctypes.c_void_p),
                ("sel_weight", ctypes.c_void_p), ("sel_slot", ctypes.c_void_p),
                ("slot_offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("xq", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
                ("stage_events", ctypes.c_void_p), ("hist_row", ctypes.c_void_p),
                ("delta", ctypes.c_void_p), ("reuse_logits", ctypes.c_int),
                ("act_format", ctypes.c_int)]


class ExpertsArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int),
                ("k", ctypes.c_int), ("S", ctypes.c_int),
                ("xq", ctypes.c_void_p), ("arena", ctypes.c_void_p),
                ("slot_stride", ctypes.c_size_t), ("slot_offsets", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("sel_slot", ctypes.c_void_p),
                ("sel_weight", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
                ("stage_events", ctypes.c_void_p), ("defer_slot", ctypes.c_int),
                ("defer_event", ctypes.c_void_p), ("shared_expert", ctypes.c_void_p),
                ("act_format", ctypes.c_int)]


class RowsArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("k", ctypes.c_int),
                ("dtype", ctypes.c_int), ("perm", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("src", ctypes.c_void_p),
                ("src_stride", ctypes.c_size_t), ("dst", ctypes.c_void_p),
                ("dst_stride", ctypes.c_size_t), ("other", ctypes.c_void_p),
                ("other_stride", ctypes.c_size_t), ("dweight", ctypes.c_void_p)]


class Int8MatmulArgs(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("G", ctypes.c_int), ("swiglu", ctypes.c_int), ("a_rows", ctypes.c_int),
                ("a", ctypes.c_void_p), ("a_stride", ctypes.c_size_t),
                ("a_scale", ctypes.c_void_p), ("index", ctypes.c_void_p),
                ("index_div", ctypes.c_int), ("offsets", ctypes.c_void_p),
                ("b", ctypes.c_void_p), ("b_stride", ctypes.c_size_t),
                ("b_group_stride", ctypes.c_size_t), ("b_scale", ctypes.c_void_p),
                ("b_scale_group_stride", ctypes.c_size_t), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_size_t), ("out_dtype", ctypes.c_int)]


class GroupedMatmulArgs(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("G", ctypes.c_int), ("dtype", ctypes.c_int), ("swiglu", ctypes.c_int),
                ("b_across", ctypes.c_int), ("zero_rest", ctypes.c_int),
                ("a_rows", ctypes.c_int), ("a", ctypes.c_void_p), ("a_stride", ctypes.c_size_t),
                ("index", ctypes.c_void_p), ("index_div", ctypes.c_int),
                ("offsets", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("b_stride", ctypes.c_size_t), ("b_group_stride", ctypes.c_size_t),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_size_t),
                ("pre", ctypes.c_void_p), ("pre_stride", ctypes.c_size_t),
                ("out_dtype", ctypes.c_int), ("pos", ctypes.c_void_p)]


class GroupedOuterArgs(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("L", ctypes.c_int), ("R", ctypes.c_int),
                ("G", ctypes.c_int), ("dtype", ctypes.c_int), ("left_rows", ctypes.c_int),
                ("right_rows", ctypes.c_int), ("left", ctypes.c_void_p),
                ("left_stride", ctypes.c_size_t), ("left_index", ctypes.c_void_p),
                ("left_div", ctypes.c_int), ("right", ctypes.c_void_p),
                ("right_stride", ctypes.c_size_t), ("right_index", ctypes.c_void_p),
                ("right_div", ctypes.c_int), ("offsets", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_size_t),
                ("out_group_stride", ctypes.c_size_t), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t), ("pos", ctypes.c_void_p)]


class Int4MatmulArgs(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("G", ctypes.c_int), ("swiglu", ctypes.c_int), ("a_rows", ctypes.c_int),
                ("a", ctypes.c_void_p), ("a_stride", ctypes.c_size_t), ("a_dtype", ctypes.c_int),
                ("index", ctypes.c_void_p), ("index_div", ctypes.c_int),
                ("offsets", ctypes.c_void_p), ("group", ctypes.c_int),
                ("codes", ctypes.c_void_p), ("codes_group_stride", ctypes.c_size_t),
                ("scale", ctypes.c_void_p), ("scale_group_stride", ctypes.c_size_t),
                ("scale_dtype", ctypes.c_int), ("zero", ctypes.c_void_p),
                ("zero_group_stride", ctypes.c_size_t), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_size_t), ("out_dtype", ctypes.c_int)]


MOE_STAGE_EVENTS = 5
_lib = None


def load() -> ctypes.CDLL:
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python resident_expert_routing_amd/build.py`")
    # torch ships its own HIP runtime (libamdhip64.so, soname libamdhip64.so.7).  Loading
    # torch first makes this library's libamdhip64.so.7 dependency resolve to that same
    # copy, so device pointers and streams from torch are valid here; loading this
    # library first would map a second, independent HIP runtime into the process.
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.moe_status_string.argtypes = [i]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_mxfp4_row_bytes.argtypes = [i]
    lib.moe_mxfp4_row_bytes.restype = sz
    lib.moe_act_row_bytes.argtypes = [i, i]
    lib.moe_act_row_bytes.restype = sz
    lib.moe_slot_bytes.argtypes = [i, i]
    lib.moe_slot_bytes.restype = sz
    lib.moe_slot_sections.argtypes = [i, i, ctypes.POINTER(sz)]
    lib.moe_slot_sections.restype = i
    lib.moe_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.moe_workspace_bytes.restype = sz
    lib.moe_route.argtypes = [ctypes.POINTER(RouteArgs), vp]
    lib.moe_route.restype = i
    lib.moe_demand_accumulate.argtypes = [vp, vp, i, i, i, vp, vp, vp, sz, vp]
    lib.moe_demand_accumulate.restype = i
    lib.moe_experts_forward.argtypes = [ctypes.POINTER(ExpertsArgs), vp]
    lib.moe_experts_forward.restype = i
    lib.moe_experts_forward_noalloc.argtypes = [ctypes.POINTER(ExpertsArgs), vp]
    lib.moe_experts_forward_noalloc.restype = i
    lib.arena_load_slot.argtypes = [vp, sz, i, i, vp, sz, vp, vp]
    lib.arena_load_slot.restype = i
    lib.moe_hot_pick.argtypes = [vp, vp, i, i, i, vp, i, i, vp, ctypes.c_double, vp, vp, sz,
                                 vp]
    lib.moe_hot_pick.restype = i
    lib.moe_hot_install.argtypes = [vp, vp, i, i, i, vp, vp]
    lib.moe_hot_install.restype = i
    lib.moe_replan.argtypes = [vp, vp, i, i, i, i, vp, vp, vp, ctypes.POINTER(i)]
    lib.moe_replan.restype = i
    lib.moe_ring_plan.argtypes = [vp, vp, i, i, vp, i, i, i, vp, vp]
    lib.moe_ring_plan.restype = i
    lib.moe_ring_install.argtypes = [vp, vp, i, i, vp, i, i, vp]
    lib.moe_ring_install.restype = i
    lib.moe_history_save.argtypes = [ctypes.c_char_p, vp, i, i, ctypes.c_uint64]
    lib.moe_history_save.restype = i
    lib.moe_history_load.argtypes = [ctypes.c_char_p, vp, i, i, ctypes.POINTER(ctypes.c_uint64)]
    lib.moe_history_load.restype = i
    lib.moe_boot_plan.argtypes = [vp, i, i, i, i, vp]
    lib.moe_boot_plan.restype = i
    lib.moe_history_scale.argtypes = [vp, sz, ctypes.c_double, vp]
    lib.moe_history_scale.restype = i
    lib.moe_positions.argtypes = [vp, i, i, vp, vp, vp]
    lib.moe_positions.restype = i
    for name in ("moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward"):
        getattr(lib, name).argtypes = [ctypes.POINTER(RowsArgs), vp]
        getattr(lib, name).restype = i
    lib.moe_int8_row_bytes.argtypes = [i]
    lib.moe_int8_row_bytes.restype = sz
    lib.moe_int8_quantize.argtypes = [vp, i, i, sz, i, vp, sz, vp, vp]
    lib.moe_int8_quantize.restype = i
    lib.moe_int8_matmul.argtypes = [ctypes.POINTER(Int8MatmulArgs), vp]
    lib.moe_int8_matmul.restype = i
    lib.moe_int4_code_bytes.argtypes = [i, i]
    lib.moe_int4_code_bytes.restype = sz
    lib.moe_int4_scale_count.argtypes = [i, i, i]
    lib.moe_int4_scale_count.restype = sz
    lib.moe_int4_quantize.argtypes = [vp, i, i, sz, i, i, vp, vp, i, vp, vp]
    lib.moe_int4_quantize.restype = i
    lib.moe_int4_matmul.argtypes = [ctypes.POINTER(Int4MatmulArgs), vp]
    lib.moe_int4_matmul.restype = i
    lib.moe_grouped_matmul.argtypes = [ctypes.POINTER(GroupedMatmulArgs), vp]
    lib.moe_grouped_matmul.restype = i
    lib.moe_grouped_outer.argtypes = [ctypes.POINTER(GroupedOuterArgs), vp]
    lib.moe_grouped_outer.restype = i
    lib.moe_grouped_outer_ws_bytes.argtypes = [i, i, i, i, i]
    lib.moe_grouped_outer_ws_bytes.restype = sz
    lib.moe_swiglu_backward.argtypes = [i, i, i, vp, sz, vp, sz, vp, sz, vp]
    lib.moe_swiglu_backward.restype = i
    lib.moe_test_mxfp4_probe.argtypes = [i, vp, vp, vp, vp, vp, vp]
    lib.moe_test_mxfp4_probe.restype = i
    lib.moe_test_stream_read.argtypes = [vp, ctypes.c_size_t, vp, i, vp]
    lib.moe_test_stream_read.restype = i
    lib.moe_test_mfma_loop.argtypes = [i, i, vp, i, vp]
    lib.moe_test_mfma_loop.restype = i
    _lib = lib
    return lib


def _ptr(p) -> int | None:
    if p is None or isinstance(p, int):
        return p
    return p.data_ptr()


def fits(*sizes) -> bool:
    """Whether every size is one that a C int holds (ctypes would cut it to 32 bits)."""
    return max(sizes) <= MOE_INT_MAX and min(sizes) >= -MOE_INT_MAX


def _host(a) -> int | None:
    """Address of a host buffer: None, an int, or a C-contiguous numpy array."""
    if a is None or isinstance(a, int):
        return a
    if not a.flags["C_CONTIGUOUS"]:
        raise ValueError("host arrays must be C-contiguous")
    return int(a.ctypes.data)


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _event(e) -> int | None:
    if e is None:
        return None
    if isinstance(e, int):
        return e
    h = int(e.cuda_event)
    if h == 0:
        # torch creates the HIP event on its first record; a null handle would
        # make the library skip the record and a later wait on it a no-op
        raise ValueError("torch.cuda.Event has no HIP event yet: record it once before passing it")
    return h


def _events(evs):
    """Sequence of MOE_STAGE_EVENTS events -> (ctypes array, its address) or (None, None)."""
    if evs is None:
        return None, None
    if len(evs) != MOE_STAGE_EVENTS:
        raise ValueError(f"stage_events needs {MOE_STAGE_EVENTS} events")
    arr = (ctypes.c_void_p * MOE_STAGE_EVENTS)(*[_event(e) for e in evs])
    return arr, ctypes.addressof(arr)


load_lib = load


def status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


moe_status_string = status_string


def moe_mxfp4_row_bytes(K: int) -> int:
    return int(load().moe_mxfp4_row_bytes(int(K)))


def moe_act_row_bytes(K: int, act_format: int) -> int:
    return int(load().moe_act_row_bytes(int(K), int(act_format)))


def moe_slot_bytes(H: int, I: int) -> int:
    return int(load().moe_slot_bytes(int(H), int(I)))


def moe_slot_sections(H: int, I: int):
    out = (ctypes.c_size_t * 6)()
    st = load().moe_slot_sections(int(H), int(I), out)
    if st != MOE_OK:
        raise MoeError(st, "moe_slot_sections")
    return [int(v) for v in out]


def moe_workspace_bytes(op: int, T: int, H: int, E: int, k: int, I: int, S: int) -> int:
    return int(load().moe_workspace_bytes(op, T, H, E, k, I, S))


def moe_route(T, H, E, k, S, x, w_router, bias, expert_slot, topk_expert, topk_score,
              sel_expert, sel_weight, sel_slot, slot_offsets, perm, xq, ws, ws_bytes,
              stream=None, stage_events=None, hist_row=None, delta=None,
              reuse_logits=False, act_format=MOE_ACT_MXFP4) -> int:
    keep, evp = _events(stage_events)
    a = RouteArgs(int(T), int(H), int(E), int(k), int(S), _ptr(x), _ptr(w_router), _ptr(bias),
                  _ptr(expert_slot), _ptr(topk_expert), _ptr(topk_score), _ptr(sel_expert),
                  _ptr(sel_weight), _ptr(sel_slot), _ptr(slot_offsets), _ptr(perm), _ptr(xq),
                  _ptr(ws), int(ws_bytes), evp, _ptr(hist_row), _ptr(delta),
                  1 if reuse_logits else 0, int(act_format))
    return int(load().moe_route(ctypes.byref(a), _stream(stream)))


def moe_demand_accumulate(topk_expert, topk_score, T, k, E, hist_row, delta, ws, ws_bytes,
                          stream=None) -> int:
    return int(load().moe_demand_accumulate(_ptr(topk_expert), _ptr(topk_score), int(T), int(k),
                                            int(E), _ptr(hist_row), _ptr(delta), _ptr(ws),
                                            int(ws_bytes), _stream(stream)))


def moe_experts_forward(T, H, I, k, S, xq, arena, slot_stride, slot_offsets, perm, sel_slot,
                        sel_weight, out, ws, ws_bytes, stream=None, stage_events=None,
                        defer_slot=-1, defer_event=None, shared_expert=None,
                        act_format=MOE_ACT_MXFP4) -> int:
    keep, evp = _events(stage_events)
    a = ExpertsArgs(int(T), int(H), int(I), int(k), int(S), _ptr(xq), _ptr(arena),
                    int(slot_stride), _ptr(slot_offsets), _ptr(perm), _ptr(sel_slot),
                    _ptr(sel_weight), _ptr(out), _ptr(ws), int(ws_bytes), evp,
                    int(defer_slot), _event(defer_event), _ptr(shared_expert), int(act_format))
    return int(load().moe_experts_forward(ctypes.byref(a), _stream(stream)))


def moe_experts_forward_noalloc(T, H, I, k, S, xq, arena, slot_stride, slot_offsets, perm,
                                sel_slot, sel_weight, out, stream=None, stage_events=None,
                                defer_slot=-1, defer_event=None, ws=None, ws_bytes=0,
                                shared_expert=None, act_format=MOE_ACT_MXFP4) -> int:
    """moe_experts_forward with the library's own scratch (ws must stay None / 0)."""
    keep, evp = _events(stage_events)
    a = ExpertsArgs(int(T), int(H), int(I), int(k), int(S), _ptr(xq), _ptr(arena),
                    int(slot_stride), _ptr(slot_offsets), _ptr(perm), _ptr(sel_slot),
                    _ptr(sel_weight), _ptr(out), _ptr(ws), int(ws_bytes), evp,
                    int(defer_slot), _event(defer_event), _ptr(shared_expert), int(act_format))
    return int(load().moe_experts_forward_noalloc(ctypes.byref(a), _stream(stream)))


def arena_load_slot(arena, slot_stride, num_slots, slot, host_src, nbytes, side_stream=None,
                    done=None) -> int:
    return int(load().arena_load_slot(_ptr(arena), int(slot_stride), int(num_slots), int(slot),
                                      _ptr(host_src), int(nbytes), _stream(side_stream),
                                      _event(done)))


def moe_hot_pick(topk_expert, topk_score, T, k, E, expert_slot, S, n_arena, hist_row, threshold,
                 out, ws=None, ws_bytes=0, stream=None) -> int:
    return int(load().moe_hot_pick(_ptr(topk_expert), _ptr(topk_score), int(T), int(k), int(E),
                                   _ptr(expert_slot), int(S), int(n_arena), _ptr(hist_row),
                                   float(threshold), _ptr(out), _ptr(ws), int(ws_bytes),
                                   _stream(stream)))


def moe_hot_install(pick, expert_slot, E, S, n_arena, slot_out=None, stream=None) -> int:
    return int(load().moe_hot_install(_ptr(pick), _ptr(expert_slot), int(E), int(S),
                                      int(n_arena), _ptr(slot_out), _stream(stream)))


def moe_replan(hist, expert_slot, L, E, k, n_swap, evict, load, new_expert_slot, n_done) -> int:
    """Host function: hist, expert_slot, evict, load, new_expert_slot are host
    buffers (numpy arrays or addresses); n_done is a ctypes.c_int."""
    return int(load_lib().moe_replan(_host(hist), _host(expert_slot), int(L), int(E), int(k),
                                     int(n_swap), _host(evict), _host(load),
                                     _host(new_expert_slot), ctypes.byref(n_done)))


def moe_ring_plan(miss_weight, expert_slot, L, E, ring, R, ring_slot0, per_step, plan,
                  stream=None) -> int:
    return int(load().moe_ring_plan(_ptr(miss_weight), _ptr(expert_slot), int(L), int(E),
                                    _ptr(ring), int(R), int(ring_slot0), int(per_step),
                                    _ptr(plan), _stream(stream)))


def moe_ring_install(plan, expert_slot, L, E, ring, R, ring_slot0, stream=None) -> int:
    return int(load().moe_ring_install(_ptr(plan), _ptr(expert_slot), int(L), int(E), _ptr(ring),
                                       int(R), int(ring_slot0), _stream(stream)))


def moe_history_save(path: str, hist, L, E, tokens: int = 0) -> int:
    """Host function: hist is a host float64 [L][E] array."""
    return int(load_lib().moe_history_save(os.fsencode(path), _host(hist), int(L), int(E),
                                            ctypes.c_uint64(int(tokens))))


def moe_history_load(path: str, hist, L, E, tokens=None) -> int:
    """Host function: fills the host float64 [L][E] array `hist`; `tokens`, if
    given, is a ctypes.c_uint64 that receives the stored token count."""
    return int(load_lib().moe_history_load(os.fsencode(path), _host(hist), int(L), int(E),
                                            ctypes.byref(tokens) if tokens is not None else None))


def moe_boot_plan(hist, L, E, k, n_slots, expert_slot) -> int:
    """Host function: hist float64 [L][E] in, expert_slot int32 [L][E] out."""
    return int(load_lib().moe_boot_plan(_host(hist), int(L), int(E), int(k), int(n_slots),
                                         _host(expert_slot)))


def moe_history_scale(hist, n, factor, stream=None) -> int:
    return int(load().moe_history_scale(_ptr(hist), int(n), float(factor), _stream(stream)))


# Sizes that a C int does not hold are past every limit of these calls.
def moe_positions(perm, T, k, pos, perm_copy=None, stream=None) -> int:
    if not fits(T, k):
        return MOE_EUNSUPPORTED
    return int(load().moe_positions(_ptr(perm), int(T), int(k), _ptr(pos), _ptr(perm_copy),
                                    _stream(stream)))


def _rows_args(T, H, k, dtype, pos, src, src_stride, dst, dst_stride, weight, perm=None,
               other=None, other_stride=0, dweight=None):
    return ctypes.byref(RowsArgs(int(T), int(H), int(k), int(dtype), _ptr(perm), _ptr(pos),
                                 _ptr(weight), _ptr(src), int(src_stride), _ptr(dst),
                                 int(dst_stride), _ptr(other), int(other_stride),
                                 _ptr(dweight)))


def moe_dispatch(T, H, k, dtype, pos, src, src_stride, dst, dst_stride, weight=None, perm=None,
                 stream=None) -> int:
    if not fits(T, H, k, dtype):
        return MOE_EUNSUPPORTED
    return int(load().moe_dispatch(_rows_args(T, H, k, dtype, pos, src, src_stride, dst,
                                              dst_stride, weight, perm), _stream(stream)))


def moe_dispatch_backward(T, H, k, dtype, pos, src, src_stride, dst, dst_stride, weight=None,
                          other=None, other_stride=0, dweight=None, stream=None) -> int:
    if not fits(T, H, k, dtype):
        return MOE_EUNSUPPORTED
    return int(load().moe_dispatch_backward(
        _rows_args(T, H, k, dtype, pos, src, src_stride, dst, dst_stride, weight, None, other,
                   other_stride, dweight), _stream(stream)))


def moe_combine(T, H, k, dtype, pos, src, src_stride, dst, dst_stride, weight=None,
                stream=None) -> int:
    if not fits(T, H, k, dtype):
        return MOE_EUNSUPPORTED
    return int(load().moe_combine(_rows_args(T, H, k, dtype, pos, src, src_stride, dst,
                                             dst_stride, weight), _stream(stream)))


def moe_combine_backward(T, H, k, dtype, pos, src, src_stride, dst, dst_stride, weight=None,
                         perm=None, other=None, other_stride=0, dweight=None,
                         stream=None) -> int:
    if not fits(T, H, k, dtype):
        return MOE_EUNSUPPORTED
    return int(load().moe_combine_backward(
        _rows_args(T, H, k, dtype, pos, src, src_stride, dst, dst_stride, weight, perm, other,
                   other_stride, dweight), _stream(stream)))


def moe_int8_row_bytes(K: int) -> int:
    if not fits(K):
        return 0
    return int(load().moe_int8_row_bytes(int(K)))


def moe_int8_quantize(x, M, K, x_stride, dtype, q, q_stride, scale, stream=None) -> int:
    if not fits(M, K, dtype):
        return MOE_EUNSUPPORTED
    return int(load().moe_int8_quantize(_ptr(x), int(M), int(K), int(x_stride), int(dtype),
                                        _ptr(q), int(q_stride), _ptr(scale), _stream(stream)))


def moe_int8_matmul(M, N, K, G, swiglu, a_rows, a, a_stride, a_scale, index, index_div, offsets,
                    b, b_stride, b_group_stride, b_scale, b_scale_group_stride, out, out_stride,
                    out_dtype, stream=None) -> int:
    if not fits(M, N, K, G, a_rows, index_div, out_dtype):
        return MOE_EUNSUPPORTED
    args = Int8MatmulArgs(int(M), int(N), int(K), int(G), 1 if swiglu else 0, int(a_rows),
                          _ptr(a), int(a_stride), _ptr(a_scale), _ptr(index), int(index_div),
                          _ptr(offsets), _ptr(b), int(b_stride), int(b_group_stride),
                          _ptr(b_scale), int(b_scale_group_stride), _ptr(out), int(out_stride),
                          int(out_dtype))
    return int(load().moe_int8_matmul(ctypes.byref(args), _stream(stream)))


def moe_grouped_matmul(M, N, K, G, dtype, swiglu, b_across, zero_rest, a_rows, a, a_stride, index,
                       index_div, offsets, b, b_stride, b_group_stride, out, out_stride, pre=None,
                       pre_stride=0, out_dtype=None, pos=None, stream=None) -> int:
    out_dtype = dtype if out_dtype is None else out_dtype
    if not fits(M, N, K, G, dtype, swiglu, b_across, zero_rest, a_rows, index_div, out_dtype):
        return MOE_EUNSUPPORTED
    args = GroupedMatmulArgs(int(M), int(N), int(K), int(G), int(dtype), int(swiglu),
                             int(b_across), int(zero_rest), int(a_rows), _ptr(a), int(a_stride),
                             _ptr(index), int(index_div), _ptr(offsets), _ptr(b), int(b_stride),
                             int(b_group_stride), _ptr(out), int(out_stride), _ptr(pre),
                             int(pre_stride), int(out_dtype), _ptr(pos))
    return int(load().moe_grouped_matmul(ctypes.byref(args), _stream(stream)))


def moe_grouped_outer(M, L, R, G, dtype, left_rows, right_rows, left, left_stride, left_index,
                      left_div, right, right_stride, right_index, right_div, offsets, out,
                      out_stride, out_group_stride, ws=None, ws_bytes=0, pos=None,
                      stream=None) -> int:
    if not fits(M, L, R, G, dtype, left_rows, right_rows, left_div, right_div):
        return MOE_EUNSUPPORTED
    args = GroupedOuterArgs(int(M), int(L), int(R), int(G), int(dtype), int(left_rows),
                            int(right_rows), _ptr(left), int(left_stride), _ptr(left_index),
                            int(left_div), _ptr(right), int(right_stride), _ptr(right_index),
                            int(right_div), _ptr(offsets), _ptr(out), int(out_stride),
                            int(out_group_stride), _ptr(ws), int(ws_bytes), _ptr(pos))
    return int(load().moe_grouped_outer(ctypes.byref(args), _stream(stream)))


def moe_grouped_outer_ws_bytes(M: int, L: int, R: int, G: int, dtype: int) -> int:
    if not fits(M, L, R, G, dtype):
        return 0
    return int(load().moe_grouped_outer_ws_bytes(int(M), int(L), int(R), int(G), int(dtype)))


def moe_swiglu_backward(M, N, dtype, pre, pre_stride, dout, dout_stride, dpre, dpre_stride,
                        stream=None) -> int:
    if not fits(M, N, dtype):
        return MOE_EUNSUPPORTED
    return int(load().moe_swiglu_backward(int(M), int(N), int(dtype), _ptr(pre), int(pre_stride),
                                          _ptr(dout), int(dout_stride), _ptr(dpre),
                                          int(dpre_stride), _stream(stream)))


def moe_int4_code_bytes(N: int, K: int) -> int:
    if not fits(N, K):
        return 0
    return int(load().moe_int4_code_bytes(int(N), int(K)))


def moe_int4_scale_count(N: int, K: int, group: int) -> int:
    if not fits(N, K, group):
        return 0
    return int(load().moe_int4_scale_count(int(N), int(K), int(group)))


def moe_int4_quantize(w, N, K, w_stride, dtype, group, codes, scale, scale_dtype, zero=None,
                      stream=None) -> int:
    if not fits(N, K, dtype, group, scale_dtype):
        return MOE_EUNSUPPORTED
    return int(load().moe_int4_quantize(_ptr(w), int(N), int(K), int(w_stride), int(dtype),
                                        int(group), _ptr(codes), _ptr(scale), int(scale_dtype),
                                        _ptr(zero), _stream(stream)))


def moe_int4_matmul(M, N, K, G, swiglu, a_rows, a, a_stride, a_dtype, index, index_div, offsets,
                    group, codes, codes_group_stride, scale, scale_group_stride, scale_dtype,
                    zero, zero_group_stride, out, out_stride, out_dtype, stream=None) -> int:
    if not fits(M, N, K, G, swiglu, a_rows, a_dtype, index_div, group, scale_dtype, out_dtype):
        return MOE_EUNSUPPORTED
    args = Int4MatmulArgs(int(M), int(N), int(K), int(G), int(swiglu), int(a_rows), _ptr(a),
                          int(a_stride), int(a_dtype), _ptr(index), int(index_div),
                          _ptr(offsets), int(group), _ptr(codes), int(codes_group_stride),
                          _ptr(scale), int(scale_group_stride), int(scale_dtype), _ptr(zero),
                          int(zero_group_stride), _ptr(out), int(out_stride), int(out_dtype))
    return int(load().moe_int4_matmul(ctypes.byref(args), _stream(stream)))


def moe_test_mxfp4_probe(shape, a, a_scale, b, b_scale, d, stream=None) -> int:
    return int(load().moe_test_mxfp4_probe(int(shape), _ptr(a), _ptr(a_scale), _ptr(b),
                                           _ptr(b_scale), _ptr(d), _stream(stream)))


def check(status: int, what: str = "moe") -> None:
    if status != MOE_OK:
        raise MoeError(status, what)


def moe_test_stream_read(src, nbytes, sink, grid, stream=None) -> int:
    return int(load().moe_test_stream_read(_ptr(src), int(nbytes), _ptr(sink), int(grid),
                                           _stream(stream)))


def moe_test_mfma_loop(iters, sink, grid, stream=None, act_format=MOE_ACT_MXFP4) -> int:
    return int(load().moe_test_mfma_loop(int(iters), int(act_format), _ptr(sink), int(grid),
                                         _stream(stream)))
