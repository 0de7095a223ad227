"""Python binding of libmesh_attn.so, the single-GPU Mesh-Attention hot path for sm_103a.

Argument marshalling only: every step of the computation (tile map, greedy order, tile
attention, LSE merge) runs in the C++ planner and the CUDA kernels behind the C ABI declared
in include/mesh_attn.h.  The functions carry the same names as the C entry points; those of rotary
positions, differential attention, the paged cache and range-masked attention hand their tensors to _binding.so, an extension module loaded
by the first of them.  PyTorch
supplies device memory and streams; nothing here computes attention, and there is no CPU
fallback: if the library is missing, load_library() raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Dict, Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmesh_attn.so")

MESH_ATTN_OK = 0
MESH_ATTN_F32 = 0
MESH_ATTN_BF16 = 1
MESH_ATTN_STATUS_WORDS = 4
STATUS_NAMES = {
    0: "OK", 1: "ERR_INVALID_ARG", 2: "ERR_UNSUPPORTED", 3: "ERR_MISALIGNED", 4: "ERR_CUDA",
    5: "ERR_DEVICE_TIMEOUT", 6: "ERR_OUT_OF_RANGE", 7: "ERR_INTERNAL", 8: "ERR_NO_MEMORY",
    9: "ERR_WORKSPACE",
}

_lib: Optional[ctypes.CDLL] = None
_ext = None  # _binding.so: the calls of rotary positions and differential attention

c_i32, c_i64, c_sz, c_f32, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float, ctypes.c_void_p
P_i32 = ctypes.POINTER(c_i32)
P_i64 = ctypes.POINTER(c_i64)
P_sz = ctypes.POINTER(c_sz)


class PlanInfo(ctypes.Structure):
    _fields_ = [("S", c_i64), ("L", c_i64), ("P", c_i32), ("R", c_i32), ("causal", c_i32), ("kvr", c_i32),
                ("greedy", c_i32), ("n_slots", c_i32), ("n_steps", c_i32), ("layout", c_i32), ("tile_q", c_i32),
                ("tile_kv", c_i32), ("n_kv_entries", c_i64), ("n_live_blocks", c_i64), ("n_kv_slots", c_i32),
                ("reserved", c_i32)]


_SIGS = {
    "mesh_attn_plan_create": (c_i32, [c_i64, c_i32, c_i32, c_i32, c_i32, ctypes.POINTER(c_vp)]),
    "mesh_attn_plan_create_ring": (c_i32, [c_i64, c_i32, c_i32, ctypes.POINTER(c_vp)]),
    "mesh_attn_plan_destroy": (c_i32, [c_vp]),
    "mesh_attn_plan_get_info": (c_i32, [c_vp, ctypes.POINTER(PlanInfo)]),
    "mesh_attn_plan_tiles": (c_i32, [c_vp, P_i32, P_i32]),
    "mesh_attn_plan_slots": (c_i32, [c_vp, P_i32]),
    "mesh_attn_plan_order": (c_i32, [c_vp, P_i32, P_i32, P_i32, P_i32]),
    "mesh_attn_plan_volumes": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, P_i32, P_i64, P_i64]),
    "mesh_attn_plan_launch_order": (c_i32, [c_vp, P_i32]),
    "mesh_attn_partials_size": (c_i32, [c_vp, c_i32, c_i32, c_i32, P_sz, P_sz]),
    "mesh_attn_workspace_size": (c_i32, [c_vp, P_sz]),
    "mesh_attn_workspace_size_for": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, P_sz]),
    "mesh_attn_tile_fwd": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_f32, c_vp, c_vp,
                                   c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_tile_fwd_noalloc": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_f32, c_vp,
                                           c_vp, c_vp, c_vp]),
    "mesh_attn_merge": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_plan_kv_slots": (c_i32, [c_vp, P_i32, P_i32, P_i32, P_i32]),
    "mesh_attn_bwd_partials_size": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, P_sz, P_sz]),
    "mesh_attn_bwd_workspace_size": (c_i32, [c_vp, P_sz]),
    "mesh_attn_bwd_prep": (c_i32, [c_i32, c_i32, c_i32, c_i64, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "mesh_attn_tile_bwd": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                   c_f32, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_bwd_reduce": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                     c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_read_status": (c_i32, [c_vp, c_vp, P_i32]),
    "mesh_attn_status_string": (ctypes.c_char_p, [c_i32]),
    "mesh_attn_last_error": (ctypes.c_char_p, []),
    "mesh_attn_set_wait_limit_ns": (c_i32, [c_i64]),
    "mesh_attn_rope": (c_i32, [c_i32, c_i32, c_i64, c_i32, c_i32, c_vp, P_i64, c_vp, P_i64, c_i32, c_vp, P_i64, c_vp,
                               P_i64, c_i32, c_i32, c_i32, ctypes.POINTER(ctypes.c_double), P_i32, c_i32, c_i32, c_vp,
                               c_i32, P_i64, c_vp]),
    "mesh_attn_plan_tables_size": (c_i32, [c_vp, P_sz]),
    "mesh_attn_plan_tables_write": (c_i32, [c_vp, c_vp, c_sz]),
    "mesh_attn_diff_workspace_size": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, P_sz]),
    "mesh_attn_diff_fwd": (c_i32, [c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_i32, c_f32,
                                   c_vp, c_vp, c_vp, c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_diff_bwd": (c_i32, [c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_i32, c_vp,
                                   c_vp, c_vp, c_vp, c_f32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_diff_decode_workspace_size": (c_i32, [c_i32, c_i32, c_i32, c_i32, c_i64, P_sz]),
    "mesh_attn_diff_decode": (c_i32, [c_i32, c_i32, c_i32, c_i32, c_i32, c_i64, c_vp, c_vp, P_i64, c_vp, P_i64, c_vp, c_vp,
                                      c_i32, c_f32, c_vp, c_vp, c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_paged_append": (c_i32, [c_i32, c_i64, c_i32, c_i32, c_i32, c_i32, c_vp, P_i64, c_vp, P_i64, c_vp, P_i64, c_vp, P_i64,
                                       c_i32, c_i32, c_vp, P_i64, c_vp, P_i64, c_vp, c_i32, c_i64, c_vp, c_vp, c_i32, c_i32, c_i32,
                                       ctypes.POINTER(ctypes.c_double), P_i32, c_i32, c_vp, c_i32, P_i64, c_vp, c_vp]),
    "mesh_attn_paged_workspace_size": (c_i32, [c_i32, c_i64, c_i32, c_i32, c_i32, c_i32, c_i64, P_sz]),
    "mesh_attn_paged_attn": (c_i32, [c_i32, c_i64, c_i32, c_i32, c_i32, c_i32, c_vp, P_i64, c_i32, c_i32, c_vp, P_i64, c_vp, P_i64,
                                     c_vp, c_i32, c_i64, c_vp, c_vp, c_i64, c_f32, c_f32, c_vp, c_i64, c_vp, c_vp, c_vp, c_sz, c_vp,
                                     c_vp]),
    "mesh_attn_range_workspace_size": (c_i32, [c_i32, c_i32, c_i32, c_i32, c_i64, c_i32, c_i32, P_sz]),
    "mesh_attn_range_fwd": (c_i32, [c_i32, c_i32, c_i32, c_i32, c_i64, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp, c_f32, c_f32,
                                    c_vp, c_vp, c_vp, c_sz, c_vp, c_vp]),
    "mesh_attn_range_bwd": (c_i32, [c_i32, c_i32, c_i32, c_i32, c_i64, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp, c_vp, c_vp,
                                    c_vp, c_f32, c_f32, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp, c_vp]),
}


class MeshAttnError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmesh_attn.so (built by __graft_entry__.build()) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def load_binding():
    """Load _binding.so, which takes the tensors of rotary positions, differential attention and its decoding, the paged cache
    and range-masked attention.
    Those calls load it when they are first made; nothing else needs it."""
    global _ext
    if _ext is None:
        lib = load_library()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("_binding.so is missing, or of another PyTorch: build it (python -c 'import __graft_entry__ as "
                               "g; g.build()')") from e
        _binding.bind(*(ctypes.cast(getattr(lib, name), c_vp).value for name in (
            "mesh_attn_rope", "mesh_attn_diff_fwd", "mesh_attn_diff_bwd", "mesh_attn_diff_decode", "mesh_attn_paged_append",
            "mesh_attn_paged_attn", "mesh_attn_range_fwd", "mesh_attn_range_bwd")))
        _ext = _binding
    return _ext


def _check(code: int, where: str):
    if code != MESH_ATTN_OK:
        msg = _lib.mesh_attn_last_error().decode()
        raise MeshAttnError(code, where, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return MESH_ATTN_BF16
    if dt == torch.float32:
        return MESH_ATTN_F32
    raise TypeError(f"unsupported dtype {dt}: use torch.bfloat16 or torch.float32")


class Plan:
    """Owning handle of a mesh_attn_plan (host memory, immutable)."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        info = PlanInfo()
        _check(_lib.mesh_attn_plan_get_info(self._h, ctypes.byref(info)), "mesh_attn_plan_get_info")
        self.info = info
        self._tables: Dict[int, torch.Tensor] = {}
        self._tables_stream: Dict[int, int] = {}  # the stream that owns their memory
        self._native = (handle.value, info.S, self._tables, self._tables_stream)  # what _binding takes

    @property
    def handle(self):
        return self._h

    def tables(self, device=None) -> torch.Tensor:
        """The plan's constant tables on `device`, copied there on the first call (which waits for the copy,
        so that every stream may read them; make it before capturing a graph, and keep the plan as long as the
        graph) and shared by all later ones."""
        got = self._tables.get(device)  # by index, the usual call
        if got is not None:
            return got
        dev = torch.device("cuda" if device is None else device)
        index = dev.index if dev.index is not None else torch.cuda.current_device()
        got = self._tables.get(index)
        if got is None:
            n = c_sz()
            _check(_lib.mesh_attn_plan_tables_size(self._h, ctypes.byref(n)), "mesh_attn_plan_tables_size")
            host = torch.empty(n.value, dtype=torch.uint8)
            _check(_lib.mesh_attn_plan_tables_write(self._h, _ptr(host), n.value), "mesh_attn_plan_tables_write")
            got = host.to(torch.device("cuda", index))
            torch.cuda.current_stream(index).synchronize()
            self._tables_stream[index] = torch.cuda.current_stream(index).cuda_stream
            self._tables[index] = got
        return got

    def __getattr__(self, name):
        if name in ("S", "L", "P", "R", "causal", "kvr", "greedy", "n_slots", "n_steps", "n_kv_entries",
                    "n_live_blocks", "layout", "tile_q", "tile_kv", "n_kv_slots"):
            return getattr(self.__dict__["info"], name)
        raise AttributeError(name)

    def close(self):
        if self._h is not None and _lib is not None:
            _lib.mesh_attn_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _i32(n: int):
    return (c_i32 * max(n, 1))()


def mesh_attn_plan_create(S: int, P: int, causal: bool, kvr: bool = True, greedy: bool = True) -> Plan:
    load_library()
    h = c_vp()
    _check(_lib.mesh_attn_plan_create(S, P, int(causal), int(kvr), int(greedy), ctypes.byref(h)),
           "mesh_attn_plan_create")
    return Plan(h)


def mesh_attn_plan_create_ring(S: int, P: int, causal: bool) -> Plan:
    load_library()
    h = c_vp()
    _check(_lib.mesh_attn_plan_create_ring(S, P, int(causal), ctypes.byref(h)), "mesh_attn_plan_create_ring")
    return Plan(h)


def mesh_attn_plan_tiles(plan: Plan):
    a, b = plan.tile_q, plan.tile_kv
    q, kv = _i32(plan.P * a), _i32(plan.P * b)
    _check(_lib.mesh_attn_plan_tiles(plan.handle, q, kv), "mesh_attn_plan_tiles")
    return ([list(q[t * a:(t + 1) * a]) for t in range(plan.P)], [list(kv[t * b:(t + 1) * b]) for t in range(plan.P)])


def mesh_attn_plan_slots(plan: Plan):
    off = _i32(plan.P + 1)
    _check(_lib.mesh_attn_plan_slots(plan.handle, off), "mesh_attn_plan_slots")
    return list(off[:plan.P + 1])


def mesh_attn_plan_order(plan: Plan):
    n = plan.n_slots
    items, steps, kv_off, kv_list = _i32(3 * n), _i32(n), _i32(n + 1), _i32(plan.n_kv_entries)
    _check(_lib.mesh_attn_plan_order(plan.handle, items, steps, kv_off, kv_list), "mesh_attn_plan_order")
    off = list(kv_off[:n + 1])
    kvl = list(kv_list[:plan.n_kv_entries])
    return ([tuple(items[3 * i:3 * i + 3]) for i in range(n)], list(steps[:n]),
            [kvl[off[i]:off[i + 1]] for i in range(n)])


def mesh_attn_plan_launch_order(plan: Plan):
    """Indices into mesh_attn_plan_order's item list, in the order the kernels take the items."""
    n = plan.n_slots
    out = (c_i32 * max(n, 1))()
    _check(_lib.mesh_attn_plan_launch_order(plan.handle, out), "mesh_attn_plan_launch_order")
    return [out[i] for i in range(n)]


def mesh_attn_plan_volumes(plan: Plan, Hq: int, Hkv: int, d: int, dtype: torch.dtype = torch.bfloat16):
    counts = _i32(3 * plan.P)
    byts = (c_i64 * (3 * plan.P))()
    ring = c_i64()
    _check(_lib.mesh_attn_plan_volumes(plan.handle, Hq, Hkv, d, _dtype_code(dtype), counts, byts, ctypes.byref(ring)),
           "mesh_attn_plan_volumes")
    P = plan.P
    return ([tuple(counts[3 * v:3 * v + 3]) for v in range(P)], [tuple(byts[3 * v:3 * v + 3]) for v in range(P)],
            ring.value)


def mesh_attn_partials_size(plan: Plan, B: int, Hq: int, d: int) -> Tuple[int, int]:
    o, l = c_sz(), c_sz()
    _check(_lib.mesh_attn_partials_size(plan.handle, B, Hq, d, ctypes.byref(o), ctypes.byref(l)),
           "mesh_attn_partials_size")
    return o.value, l.value


def mesh_attn_workspace_size(plan: Plan) -> int:
    n = c_sz()
    _check(_lib.mesh_attn_workspace_size(plan.handle, ctypes.byref(n)), "mesh_attn_workspace_size")
    return n.value


def mesh_attn_workspace_size_for(plan: Plan, dtype: torch.dtype, B: int, Hq: int, Hkv: int, d: int) -> int:
    n = c_sz()
    _check(_lib.mesh_attn_workspace_size_for(plan.handle, _dtype_code(dtype), B, Hq, Hkv, d, ctypes.byref(n)),
           "mesh_attn_workspace_size_for")
    return n.value


def new_status(device=None) -> torch.Tensor:
    """A zeroed device status block (MESH_ATTN_STATUS_WORDS int32)."""
    return torch.zeros(MESH_ATTN_STATUS_WORDS, dtype=torch.int32, device=device or "cuda")


def new_workspace(plan: Plan, device=None, q: Optional[torch.Tensor] = None, k: Optional[torch.Tensor] = None
                  ) -> torch.Tensor:
    """Workspace for mesh_attn_tile_fwd and mesh_attn_merge; pass q and k (fp32 inputs need room
    for their bf16 pieces)."""
    if q is not None and k is not None:
        B, Hq, _, d = q.shape
        n = mesh_attn_workspace_size_for(plan, q.dtype, B, Hq, k.shape[1], d)
    else:
        n = mesh_attn_workspace_size(plan)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def new_partials(plan: Plan, B: int, Hq: int, d: int, device=None):
    no, nl = mesh_attn_partials_size(plan, B, Hq, d)
    dev = device or "cuda"
    return (torch.empty(max(no, 4), dtype=torch.float32, device=dev),
            torch.empty(max(nl, 4), dtype=torch.float32, device=dev))


def mesh_attn_tile_fwd(plan: Plan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float],
                       partial_o: torch.Tensor, partial_lse: torch.Tensor, workspace: torch.Tensor,
                       status: torch.Tensor, stream=None) -> None:
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    _check(_lib.mesh_attn_tile_fwd(plan.handle, _dtype_code(q.dtype), B, Hq, Hkv, d, _ptr(q), _ptr(k), _ptr(v),
                                   float(scale), _ptr(partial_o), _ptr(partial_lse), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(status),
                                   _stream_handle(stream)), "mesh_attn_tile_fwd")


def mesh_attn_tile_fwd_noalloc(plan: Plan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                               scale: Optional[float], partial_o: torch.Tensor, partial_lse: torch.Tensor,
                               status: torch.Tensor, stream=None) -> None:
    """mesh_attn_tile_fwd without a workspace: for callers that may not allocate device memory.
    The work list goes into the library's fixed scratch array; calls overlapping on the GPU race."""
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    _check(_lib.mesh_attn_tile_fwd_noalloc(plan.handle, _dtype_code(q.dtype), B, Hq, Hkv, d, _ptr(q), _ptr(k),
                                           _ptr(v), float(scale), _ptr(partial_o), _ptr(partial_lse), _ptr(status),
                                           _stream_handle(stream)), "mesh_attn_tile_fwd_noalloc")


def mesh_attn_merge(plan: Plan, B: int, Hq: int, d: int, partial_o: torch.Tensor, partial_lse: torch.Tensor,
                    O: torch.Tensor, LSE: torch.Tensor, workspace: torch.Tensor, status: torch.Tensor,
                    stream=None) -> None:
    _check(_lib.mesh_attn_merge(plan.handle, _dtype_code(O.dtype), B, Hq, d, _ptr(partial_o), _ptr(partial_lse),
                                _ptr(O), _ptr(LSE), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(status), _stream_handle(stream)), "mesh_attn_merge")


def mesh_attn_plan_kv_slots(plan: Plan):
    """Backward KV slots: (kv_slot_off [P+1], [(k, t, kv_slot)], [[Q partitions] per slot])."""
    n = plan.n_kv_slots
    off, items, q_off, q_list = _i32(plan.P + 1), _i32(3 * n), _i32(n + 1), _i32(plan.n_live_blocks)
    _check(_lib.mesh_attn_plan_kv_slots(plan.handle, off, items, q_off, q_list), "mesh_attn_plan_kv_slots")
    qo = list(q_off[:n + 1])
    ql = list(q_list[:plan.n_live_blocks])
    return (list(off[:plan.P + 1]), [tuple(items[3 * i:3 * i + 3]) for i in range(n)],
            [ql[qo[i]:qo[i + 1]] for i in range(n)])


def mesh_attn_bwd_partials_size(plan: Plan, B: int, Hq: int, Hkv: int, d: int) -> Tuple[int, int]:
    q, kv = c_sz(), c_sz()
    _check(_lib.mesh_attn_bwd_partials_size(plan.handle, B, Hq, Hkv, d, ctypes.byref(q), ctypes.byref(kv)),
           "mesh_attn_bwd_partials_size")
    return q.value, kv.value


def mesh_attn_bwd_workspace_size(plan: Plan) -> int:
    n = c_sz()
    _check(_lib.mesh_attn_bwd_workspace_size(plan.handle, ctypes.byref(n)), "mesh_attn_bwd_workspace_size")
    return n.value


def new_bwd_workspace(plan: Plan, device=None) -> torch.Tensor:
    return torch.empty(max(mesh_attn_bwd_workspace_size(plan), 16), dtype=torch.uint8, device=device or "cuda")


def new_bwd_partials(plan: Plan, B: int, Hq: int, Hkv: int, d: int, device=None):
    nq, nkv = mesh_attn_bwd_partials_size(plan, B, Hq, Hkv, d)
    dev = device or "cuda"
    return tuple(torch.empty(max(n, 4), dtype=torch.float32, device=dev) for n in (nq, nkv, nkv))


def mesh_attn_bwd_prep(O: torch.Tensor, dO: torch.Tensor, D: torch.Tensor, status: torch.Tensor,
                       stream=None) -> None:
    B, Hq, S, d = O.shape
    if O.dtype != dO.dtype or not O.is_contiguous() or not dO.is_contiguous():
        raise ValueError("O and dO must be contiguous and of one dtype")
    _check(_lib.mesh_attn_bwd_prep(_dtype_code(O.dtype), B, Hq, S, d, _ptr(O), _ptr(dO), _ptr(D), _ptr(status),
                                   _stream_handle(stream)), "mesh_attn_bwd_prep")


def mesh_attn_tile_bwd(plan: Plan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dO: torch.Tensor,
                       LSE: torch.Tensor, D: torch.Tensor, scale: Optional[float], dq_partial: torch.Tensor,
                       dk_partial: torch.Tensor, dv_partial: torch.Tensor, workspace: torch.Tensor,
                       status: torch.Tensor, stream=None) -> None:
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for t in (q, k, v, dO):
        if not t.is_contiguous():
            raise ValueError("q, k, v and dO must be contiguous")
    _check(_lib.mesh_attn_tile_bwd(plan.handle, _dtype_code(q.dtype), B, Hq, Hkv, d, _ptr(q), _ptr(k), _ptr(v),
                                   _ptr(dO), _ptr(LSE), _ptr(D), float(scale), _ptr(dq_partial), _ptr(dk_partial),
                                   _ptr(dv_partial), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _ptr(status), _stream_handle(stream)), "mesh_attn_tile_bwd")


def mesh_attn_bwd_reduce(plan: Plan, B: int, Hq: int, Hkv: int, d: int, dq_partial: torch.Tensor,
                         dk_partial: torch.Tensor, dv_partial: torch.Tensor, dQ: torch.Tensor, dK: torch.Tensor,
                         dV: torch.Tensor, workspace: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    if not (dQ.dtype == dK.dtype == dV.dtype):
        raise ValueError("dQ, dK and dV must share one dtype")
    _check(_lib.mesh_attn_bwd_reduce(plan.handle, _dtype_code(dQ.dtype), B, Hq, Hkv, d, _ptr(dq_partial),
                                     _ptr(dk_partial), _ptr(dv_partial), _ptr(dQ), _ptr(dK), _ptr(dV),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
                                     _stream_handle(stream)), "mesh_attn_bwd_reduce")


def mesh_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, O: torch.Tensor,
                            LSE: torch.Tensor, dO: torch.Tensor, P: int, causal: bool, kvr: bool = True,
                            greedy: bool = True, scale: Optional[float] = None, plan: Optional[Plan] = None,
                            return_partials: bool = False, check_status: bool = True):
    """Whole backward on the current stream: D = dO . O, tile backward, reduce.

    q [B,Hq,S,d], k/v [B,Hkv,S,d], O and dO [B,Hq,S,d] (one dtype, bf16 or fp32), LSE [B,Hq,S]
    fp32 from the forward.  Returns (dQ, dK, dV) in q's dtype; with return_partials also the
    fp32 partials (dq, dk, dv).
    """
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    plan = plan or mesh_attn_plan_create(S, P, causal, kvr, greedy)
    dq_p, dk_p, dv_p = new_bwd_partials(plan, B, Hq, Hkv, d, q.device)
    ws = new_bwd_workspace(plan, q.device)
    st = new_status(q.device)
    D = torch.empty(B, Hq, S, dtype=torch.float32, device=q.device)
    dQ, dK, dV = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    mesh_attn_bwd_prep(O, dO, D, st)
    mesh_attn_tile_bwd(plan, q, k, v, dO, LSE, D, scale, dq_p, dk_p, dv_p, ws, st)
    mesh_attn_bwd_reduce(plan, B, Hq, Hkv, d, dq_p, dk_p, dv_p, dQ, dK, dV, ws, st)
    if check_status:
        code = mesh_attn_read_status(st)
        if code != 0:
            raise MeshAttnError(code, "device", f"status block {st.tolist()}")
    if return_partials:
        return dQ, dK, dV, dq_p, dk_p, dv_p
    return dQ, dK, dV


def mesh_attn_read_status(status: torch.Tensor, stream=None) -> int:
    out = c_i32()
    _check(_lib.mesh_attn_read_status(_ptr(status), _stream_handle(stream), ctypes.byref(out)),
           "mesh_attn_read_status")
    return out.value


def mesh_attn_set_wait_limit_ns(ns: int) -> None:
    load_library()
    _check(_lib.mesh_attn_set_wait_limit_ns(int(ns)), "mesh_attn_set_wait_limit_ns")


def mesh_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, P: int, causal: bool, kvr: bool = True,
                   greedy: bool = True, scale: Optional[float] = None, plan: Optional[Plan] = None,
                   return_partials: bool = False, check_status: bool = True):
    """Whole hot path on the current stream: plan, tile forward, LSE merge.

    q [B,Hq,S,d], k/v [B,Hkv,S,d] CUDA tensors (bf16 or fp32).  Returns (O, LSE) with O in
    q's dtype and LSE fp32; with return_partials also (partial_o, partial_lse).
    """
    B, Hq, S, d = q.shape
    plan = plan or mesh_attn_plan_create(S, P, causal, kvr, greedy)
    po, pl = new_partials(plan, B, Hq, d, q.device)
    ws = new_workspace(plan, q.device, q, k)
    st = new_status(q.device)
    O = torch.empty_like(q)
    LSE = torch.empty(B, Hq, S, dtype=torch.float32, device=q.device)
    mesh_attn_tile_fwd(plan, q, k, v, scale, po, pl, ws, st)
    mesh_attn_merge(plan, B, Hq, d, po, pl, O, LSE, ws, st)
    if check_status:
        code = mesh_attn_read_status(st)
        if code != 0:
            raise MeshAttnError(code, "device", f"status block {st.tolist()}")
    if return_partials:
        return O, LSE, po, pl
    return O, LSE


def _dense_gradient(g: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels take it: contiguous, on a 16-byte boundary.  PyTorch hands on views of larger gradients (of a cat, say)
    that begin anywhere."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class MeshAttentionFunction(torch.autograd.Function):
    """torch.autograd binding of the two public calls: the forward runs mesh_attention and keeps
    q, k, v, O and LSE; the backward runs mesh_attention_backward with the incoming dO.  Gradients
    reach q, k and v; LSE is returned as a non-differentiable output (no gradient flows through
    it).  Argument marshalling only: every step runs in the library's kernels."""

    @staticmethod
    def forward(ctx, q, k, v, P, causal, kvr, greedy, scale):
        plan = mesh_attn_plan_create(q.shape[2], P, causal, kvr, greedy)
        O, LSE = mesh_attention(q, k, v, P, causal, kvr, greedy, scale, plan=plan)
        ctx.save_for_backward(q, k, v, O, LSE)
        ctx.plan = plan
        ctx.args = (P, causal, kvr, greedy, scale)
        ctx.mark_non_differentiable(LSE)
        return O, LSE

    @staticmethod
    def backward(ctx, dO, dLSE):
        q, k, v, O, LSE = ctx.saved_tensors
        P, causal, kvr, greedy, scale = ctx.args
        dQ, dK, dV = mesh_attention_backward(q, k, v, O, LSE, _dense_gradient(dO), P, causal, kvr, greedy, scale,
                                             plan=ctx.plan)
        return dQ, dK, dV, None, None, None, None, None


def mesh_attention_autograd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, P: int, causal: bool,
                            kvr: bool = True, greedy: bool = True, scale: Optional[float] = None):
    """mesh_attention with autograd: returns (O, LSE); O.backward(...) fills q.grad, k.grad and v.grad
    through the tile backward."""
    return MeshAttentionFunction.apply(q, k, v, P, causal, kvr, greedy, scale)


# ---------------------------------------------------------------- rotary positions

class MeshRope:
    """Rotary positions with several axes: which axis turns each pair of columns, and how fast.

    d         columns of a head, `groups` equal groups of them rotated alike (2 for the halves of a
              differential head)
    sections  pairs of each axis, e.g. (12, 10, 10) for time, height and width; their sum is at
              most d / groups / 2, the columns behind are copied
    style     "half": pairs (i, i + n); "adjacent": (2 i, 2 i + 1)
    freq      "global": base^(-i / n) over all n pairs, each axis taking its section of that ladder;
              "axial": base^(-j / n_a) within the section of each axis; or the frequencies
              themselves, one a pair, in radians a position
    axis_of_pair  the axis of each pair where the sections are interleaved
    """

    def __init__(self, d: int, sections: Sequence[int], base: float = 10000.0, groups: int = 1, style: str = "half",
                 freq="global", axis_of_pair: Optional[Sequence[int]] = None):
        sections = [int(n) for n in sections]
        if not sections or any(n < 0 for n in sections) or sum(sections) < 1:
            raise ValueError("sections must be one or more pair counts")
        n = sum(sections)
        if groups < 1 or d % groups or 2 * n > d // groups:
            raise ValueError(f"need groups >= 1, d % groups == 0 and 2 * sum(sections) <= d / groups; got d = {d}, "
                             f"groups = {groups}, sections = {sections}")
        if style not in ("half", "adjacent"):
            raise ValueError("style must be 'half' or 'adjacent'")
        axis = [a for a, m in enumerate(sections) for _ in range(m)]
        if axis_of_pair is not None:
            axis = [int(a) for a in axis_of_pair]
            if len(axis) != n or any(a < 0 or a >= len(sections) for a in axis):
                raise ValueError("axis_of_pair must give an axis of sections for each pair")
        if isinstance(freq, str):
            if not base > 0:
                raise ValueError("base must be > 0")
            if freq == "global":
                freq = [float(base) ** (-i / n) for i in range(n)]
            elif freq == "axial":
                at = [0] * len(sections)
                out = []
                for a in axis:
                    out.append(float(base) ** (-at[a] / axis.count(a)))
                    at[a] += 1
                freq = out
            else:
                raise ValueError("freq must be 'global', 'axial' or a sequence of frequencies")
        freq = [float(f) for f in freq]
        if len(freq) != n:
            raise ValueError("freq must give a frequency for each pair")
        self.d, self.groups, self.style, self.n_axes, self.n_pairs = int(d), int(groups), style, len(sections), n
        self.freq, self.axis = tuple(freq), tuple(axis)
        # what _binding takes: a header, the frequencies, the axes
        self._native = struct.pack(f"=6i{n}d{n}i", d, groups, n, len(sections), int(style == "adjacent"), 0, *freq, *axis)


def _handle_of(stream):
    return None if stream is None else stream.cuda_stream


def mesh_attn_rope(rope: MeshRope, q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
                   q_out: torch.Tensor, k_out: Optional[torch.Tensor], inverse: bool = False, stream=None) -> None:
    """q [B, Hq, S, d] and k [B, Hk, S, d] (or None) rotated into q_out and k_out; views with any batch,
    head and token strides.  positions: int32 or int64 [axes, S] or [axes, B, S] ([S] or [B, S]
    for one axis), any strides."""
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    _rope(rope, q, k, positions, q_out, k_out, inverse, stream)


def _rope(rope, q, k, positions, q_out, k_out, inverse, stream=None):
    out = (_ext or load_binding()).rope(rope._native, q, k, positions, q_out, k_out, 1 if inverse else 0, _handle_of(stream))
    if out.__class__ is int:
        _check(out, "mesh_attn_rope")
    return out


def mesh_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, rope: MeshRope):
    """q [B, Hq, S, d] and k [B, Hk, S, d] (or None) with their positions, as dense [B, H, S, d] tensors, which is what
    the attention calls take; q and k may be views, e.g. a projection's [B, S, H, d] transposed."""
    return _rope(rope, q, k, positions, None, None, False)


def mesh_rope_backward(dq: torch.Tensor, dk: Optional[torch.Tensor], positions: torch.Tensor, rope: MeshRope,
                       dq_out: Optional[torch.Tensor] = None, dk_out: Optional[torch.Tensor] = None):
    """The gradients of mesh_rope's q and k from those of its outputs, into dq_out and dk_out where given (any strides,
    e.g. the projection's layout), else into dense tensors."""
    return _rope(rope, dq, dk, positions, dq_out, dk_out, True)


def _memory_order(t: torch.Tensor):
    """t's axes from the slowest to the fastest in memory, the columns last."""
    return sorted(range(t.dim() - 1), key=lambda i: (-t.stride(i), i)) + [t.dim() - 1]


def _empty_in_order(like: torch.Tensor, order) -> torch.Tensor:
    out = torch.empty([like.shape[i] for i in order], dtype=like.dtype, device=like.device)
    return out.permute([order.index(i) for i in range(like.dim())])


class MeshRopeFunction(torch.autograd.Function):
    """torch.autograd binding of mesh_rope: the backward pass is the inverse rotation, written in
    the memory order that q and k have (a projection's [B, S, H, d] where they are views of one)."""

    @staticmethod
    def forward(ctx, q, k, positions, rope):
        ctx.save_for_backward(positions)
        ctx.rope = rope
        ctx.orders = (_memory_order(q), None if k is None else _memory_order(k))
        return mesh_rope(q, k, positions, rope)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        (positions,) = ctx.saved_tensors
        grads = [None if g is None else g if g.stride(-1) == 1 else g.contiguous() for g in (dq, dk)]
        outs = [None if g is None else _empty_in_order(g, o) for g, o in zip(grads, ctx.orders)]
        return (*mesh_rope_backward(*grads, positions, ctx.rope, *outs), None, None)


def mesh_rope_autograd(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, rope: MeshRope):
    """mesh_rope with autograd."""
    return MeshRopeFunction.apply(q, k, positions, rope)


# ---------------------------------------------------------------- differential attention

def mesh_attn_diff_workspace_size(plan: Plan, dtype: torch.dtype, B: int, Hq: int, Hkv: int, d: int,
                                  backward: bool = False) -> int:
    n = c_sz()
    _check(_lib.mesh_attn_diff_workspace_size(plan.handle, _dtype_code(dtype), B, Hq, Hkv, d, int(backward), ctypes.byref(n)),
           "mesh_attn_diff_workspace_size")
    return n.value


def new_diff_workspace(plan: Plan, q: torch.Tensor, k: torch.Tensor, backward: bool = False) -> torch.Tensor:
    """Workspace of mesh_attn_diff_fwd for tensors of q's and k's sizes; with backward, of both directions."""
    B, Hq, _, d = q.shape
    n = mesh_attn_diff_workspace_size(plan, q.dtype, B, Hq, k.shape[1], d, backward)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def _on_plan(name: str, plan: Plan, device, *args):
    """One of _binding's calls that read a plan's tables, which are made for the device where they are not there yet."""
    entry = getattr(_ext or load_binding(), name)
    out = entry(plan._native, *args)
    if out is None:
        plan.tables(device)
        out = entry(plan._native, *args)
    if out.__class__ is int:
        _check(out, "mesh_attn_" + name)
    return out


def mesh_attn_diff_fwd(plan: Plan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
                       scale: Optional[float], O: torch.Tensor, O2: Optional[torch.Tensor], LSE: torch.Tensor,
                       workspace: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    _on_plan("diff_fwd", plan, q.device, q, k, v, lam, scale, O, O2, LSE, 0, workspace, status,
             _handle_of(stream))


def mesh_attn_diff_bwd(plan: Plan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, O: torch.Tensor,
                       O2: torch.Tensor, LSE: torch.Tensor, dO: torch.Tensor, scale: Optional[float], dQ: torch.Tensor,
                       dK: torch.Tensor, dV: torch.Tensor, dlam: torch.Tensor, workspace: torch.Tensor,
                       status: torch.Tensor, stream=None) -> None:
    _on_plan("diff_bwd", plan, q.device, q, k, v, lam, O, O2, LSE, dO, scale, dQ, dK, dV, dlam, workspace,
             status, _handle_of(stream))


def _raise_status(status: torch.Tensor):
    code = mesh_attn_read_status(status, torch.cuda.current_stream(status.device))
    if code != 0:
        raise MeshAttnError(code, "device", f"status block {status.tolist()}")


def mesh_diff_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, P: int, causal: bool,
                        kvr: bool = True, greedy: bool = True, scale: Optional[float] = None,
                        plan: Optional[Plan] = None, workspace: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, check_status: bool = True, return_saved: bool = False):
    """Differential attention on the current stream: softmax(q1 k1^T s) v - lam softmax(q2 k2^T s) v with q = [q1 | q2] and
    k = [k1 | k2] by columns (s = 1 / sqrt(d / 2) unless given).

    q [B, Hq, S, d], k, v [B, Hkv, S, d], lam [Hq] or [1] (one value for all heads), all bf16 or all fp32.  Returns O (q's
    shape and dtype) and LSE (fp32 [B, Hq, 2, S]); with return_saved O, O2 and LSE, which
    mesh_diff_attention_backward takes.  P, kvr and greedy make the plan where none is given (P has to divide S); the plan's
    length and mask count here, its partitions do not.  A program that calls it every step keeps plan, workspace
    (new_diff_workspace) and status (new_status) and passes check_status=False, which leaves out the wait.
    """
    if plan is None or workspace is None or status is None:
        load_binding().diff_check(q, k, v, lam)
        plan = plan or mesh_attn_plan_create(q.shape[2], P, causal, kvr, greedy)
    ws = new_diff_workspace(plan, q, k) if workspace is None else workspace
    st = new_status(q.device) if status is None else status
    O, O2, LSE = _on_plan("diff_fwd", plan, q.device, q, k, v, lam, scale, None, None, None,
                          1 if return_saved else 0, ws, st, None)
    if check_status:
        _raise_status(st)
    return (O, O2, LSE) if return_saved else (O, LSE)


def mesh_diff_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, O: torch.Tensor,
                                 O2: torch.Tensor, LSE: torch.Tensor, dO: torch.Tensor, P: int, causal: bool,
                                 kvr: bool = True, greedy: bool = True, scale: Optional[float] = None,
                                 plan: Optional[Plan] = None, workspace: Optional[torch.Tensor] = None,
                                 status: Optional[torch.Tensor] = None, check_status: bool = True):
    """(dQ, dK, dV, dlam) from the forward's O, O2 and LSE and the gradient dO, on the current stream."""
    if plan is None or workspace is None or status is None:
        load_binding().diff_check(q, k, v, lam)
        plan = plan or mesh_attn_plan_create(q.shape[2], P, causal, kvr, greedy)
    ws = new_diff_workspace(plan, q, k, backward=True) if workspace is None else workspace
    st = new_status(q.device) if status is None else status
    grads = _on_plan("diff_bwd", plan, q.device, q, k, v, lam, O, O2, LSE, dO, scale, None, None, None,
                     None, ws, st, None)
    if check_status:
        _raise_status(st)
    return grads


class MeshDiffAttentionFunction(torch.autograd.Function):
    """torch.autograd binding of mesh_diff_attention: gradients reach q, k, v and lam; LSE is a non-differentiable output."""

    @staticmethod
    def forward(ctx, q, k, v, lam, P, causal, kvr, greedy, scale, plan, check_status, status):
        plan = plan or mesh_attn_plan_create(q.shape[2], P, causal, kvr, greedy)
        O, O2, LSE = mesh_diff_attention(q, k, v, lam, P, causal, kvr, greedy, scale, plan=plan, status=status,
                                         check_status=check_status, return_saved=True)
        ctx.save_for_backward(q, k, v, lam, O, O2, LSE)
        ctx.plan = plan
        ctx.args = (P, causal, kvr, greedy, scale)
        ctx.check_status, ctx.status = check_status, status
        ctx.mark_non_differentiable(LSE)
        return O, LSE

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO, dLSE):
        grads = mesh_diff_attention_backward(*ctx.saved_tensors, _dense_gradient(dO), *ctx.args, plan=ctx.plan, status=ctx.status,
                                             check_status=ctx.check_status)
        return (*grads, None, None, None, None, None, None, None, None)


def mesh_diff_attention_autograd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, P: int, causal: bool,
                                 kvr: bool = True, greedy: bool = True, scale: Optional[float] = None,
                                 plan: Optional[Plan] = None, check_status: bool = True,
                                 status: Optional[torch.Tensor] = None):
    """mesh_diff_attention with autograd: returns (O, LSE); O.backward(...) fills the gradients of q, k, v and lam.  With
    check_status=False a failure in either direction is recorded in `status` (new_status), for the program to read later."""
    return MeshDiffAttentionFunction.apply(q, k, v, lam, P, causal, kvr, greedy, scale, plan, check_status, status)


def new_diff_decode_workspace(B: int, Hq: int, Hkv: int, d: int, T: int, device=None) -> torch.Tensor:
    """Workspace of mesh_diff_decode for these sizes and smaller ones, zeroed as the first call wants it."""
    load_library()
    n = c_sz()
    _check(_lib.mesh_attn_diff_decode_workspace_size(B, Hq, Hkv, d, T, ctypes.byref(n)), "mesh_attn_diff_decode_workspace_size")
    return torch.zeros(max(n.value, 16), dtype=torch.uint8, device=device or "cuda")


def mesh_attn_diff_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor,
                          lam: torch.Tensor, scale: Optional[float], O: torch.Tensor, LSE: torch.Tensor,
                          workspace: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    _diff_decode(q, k_cache, v_cache, lens, lam, scale, O, LSE, workspace, status, stream)


def _diff_decode(q, k_cache, v_cache, lens, lam, scale, O, LSE, workspace, status, stream=None):
    out = (_ext or load_binding()).diff_decode(q, k_cache, v_cache, lens, lam, scale, O, LSE, workspace, status, _handle_of(stream))
    if out.__class__ is int:
        _check(out, "mesh_attn_diff_decode")
    return out


def mesh_diff_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor, lam: torch.Tensor,
                     scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, check_status: bool = True):
    """Differential attention of one new token a sequence, on the current stream: q [B, Hq, 1, d] against the first lens[b]
    (int32, on the device) tokens of k_cache, v_cache [B, Hkv, T, d], which may be views with other strides (16-byte
    multiples).  Returns O [B, Hq, 1, d] and LSE [B, Hq, 2, 1].  A serving loop keeps workspace
    (new_diff_decode_workspace) and status and passes check_status=False."""
    if workspace is None or status is None:
        load_binding().diff_check(q, k_cache, v_cache, lam)
    ws = workspace
    if ws is None:
        ws = new_diff_decode_workspace(q.shape[0], q.shape[1], k_cache.shape[1], q.shape[3], k_cache.shape[2], q.device)
    st = new_status(q.device) if status is None else status
    O, LSE = _diff_decode(q, k_cache, v_cache, lens, lam, scale, None, None, ws, st)
    if check_status:
        _raise_status(st)
    return O, LSE


# ---------------------------------------------------------------- a paged cache

def mesh_paged_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                      table: torch.Tensor, offsets: torch.Tensor, lens: torch.Tensor, rope: Optional[MeshRope] = None,
                      positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, check_status: bool = True) -> Optional[torch.Tensor]:
    """New tokens' keys and values into their sequences' pages, on the current stream: k turned by `rope` (copied
    without one), v copied.  Returns q turned likewise, as a dense tensor or in q_out, for mesh_paged_attention (None for no q).

    q [N, Hq, d], k, v [N, Hkv, d]: the new tokens of all sequences one sequence after another, views with any token and head
    strides, e.g. slices of one projection.  k_pages, v_pages [n_pages, Hkv, page, d], written in place; table int32 [B, pages]:
    sequence b's token i is row i % page of page table[b, i // page].  Sequence b's new tokens are rows offsets[b] to offsets[b + 1]
    (int32 [B + 1]) and the last of the lens[b] (int32 [B]) tokens it then has; rows from offsets[B] on are left as they
    are (in a q_out made by the call: not set).  positions: int32 or int64 [axes, N] ([N] for one axis) where they are not the
    tokens' places.  A token whose place or page does not exist is left out and recorded in `status`; a program that calls it every step
    keeps status (new_status) and passes check_status=False, which leaves out the wait."""
    st = new_status(k.device) if status is None else status
    out = (_ext or load_binding()).paged_append(None if rope is None else rope._native, q, k, v, k_pages, v_pages, table, offsets,
                                                lens, positions, q_out, st, None)
    if out.__class__ is int:
        _check(out, "mesh_attn_paged_append")
    if check_status:
        _raise_status(st)
    return out[0]


def new_paged_workspace(q: torch.Tensor, k_pages: torch.Tensor, table: torch.Tensor, max_new: int) -> torch.Tensor:
    """Workspace of mesh_paged_attention for batches of at most as many tokens and sequences and at most max_new new tokens of
    one, its head zeroed as the first call wants it."""
    load_library()
    n = c_sz()
    _check(_lib.mesh_attn_paged_workspace_size(_dtype_code(q.dtype), q.shape[0], table.shape[0], q.shape[1], k_pages.shape[1],
                                               q.shape[2], max_new, ctypes.byref(n)), "mesh_attn_paged_workspace_size")
    ws = torch.empty(max(n.value, 2048), dtype=torch.uint8, device=q.device)
    ws[:2048].zero_()
    return ws


def mesh_paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor, offsets: torch.Tensor,
                         lens: torch.Tensor, max_new: int, scale: Optional[float] = None, cap: float = 0.0,
                         slopes: Optional[torch.Tensor] = None, window: int = 0, O: Optional[torch.Tensor] = None,
                         LSE: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, check_status: bool = True):
    """Attention of the new tokens q [N, Hq, d] over their sequences' pages, on the current stream; the pages hold
    the new tokens' own keys and values already (mesh_paged_append, whose arguments these are).  Token i of a sequence sees its
    tokens j <= i, with window > 0 those with i - j < window; scores are scale q.k (1 / sqrt(d) unless given), capped to
    cap tanh(score / cap) with cap > 0 (1e-18 to 1e18), less slopes[h] (i - j) with slopes (fp32 [Hq]).

    One call serves decoding steps (max_new = 1), guessed tokens and chunks of prompts, also mixed: max_new bounds a
    sequence's new tokens.  Returns O [N, Hq, d] and LSE fp32 [N, Hq]; rows from offsets[B] on are not written.  q and the pages may
    be views with strides of multiples of 16 bytes; page a multiple of 16.  A serving loop keeps workspace (new_paged_workspace) and
    status and passes check_status=False; its status block is for its calls over pages alone, which go on behind an index out of range
    (code 6) where range-masked and plain attention do not.  A wait that ran out (code 5) takes its place."""
    ws = new_paged_workspace(q, k_pages, table, max_new) if workspace is None else workspace
    st = new_status(q.device) if status is None else status
    out = (_ext or load_binding()).paged_attn(q, k_pages, v_pages, table, offsets, lens, max_new, scale, cap, slopes, window, O, LSE,
                                              ws, st, None)
    if out.__class__ is int:
        _check(out, "mesh_attn_paged_attn")
    if check_status:
        _raise_status(st)
    return out


# ---------------------------------------------------------------- range-masked attention

def mesh_ranges(documents: Sequence[int], causal: bool = True, prefixes: Optional[Sequence[int]] = None, window: int = 0,
                length: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """lo and hi (int32 [S], on the host) of documents of these lengths packed one after another: each query sees its own document
    (causal: up to itself), the first prefixes[i] tokens of document i also one another, with window > 0 no key further
    back than window - 1.  `length` beyond their sum pads: rows behind see nothing and are not seen."""
    documents = [int(n) for n in documents]
    if any(n < 0 for n in documents):
        raise ValueError("documents must have lengths >= 0")
    if prefixes is not None and len(prefixes) != len(documents):
        raise ValueError("prefixes must give a length for each document")
    if window < 0:
        raise ValueError("window must be >= 0")
    S = sum(documents) if length is None else int(length)
    if S < sum(documents):
        raise ValueError(f"the documents have {sum(documents)} tokens, more than length = {S}")
    lo, hi = torch.zeros(S, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    at = 0
    for d, n in enumerate(documents):
        i = torch.arange(at, at + n, dtype=torch.int32)
        lo[at:at + n] = torch.clamp(i - (window - 1), min=at) if window else at
        hi[at:at + n] = i + 1 if causal else at + n
        if prefixes is not None and causal:
            hi[at:at + n] = torch.clamp(hi[at:at + n], min=at + max(0, min(int(prefixes[d]), n)))
        at += n
    return lo, hi


def new_range_workspace(q: torch.Tensor, k: torch.Tensor, backward: bool = False) -> torch.Tensor:
    """Workspace of mesh_range_attention for tensors of q's and k's sizes; with backward, of both directions."""
    load_library()
    B, Hq, S, d = q.shape
    n = c_sz()
    _check(_lib.mesh_attn_range_workspace_size(_dtype_code(q.dtype), B, Hq, k.shape[1], S, d, int(backward), ctypes.byref(n)),
           "mesh_attn_range_workspace_size")
    return torch.empty(max(n.value, 16), dtype=torch.uint8, device=q.device)


def mesh_range_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lo: torch.Tensor, hi: torch.Tensor,
                         scale: Optional[float] = None, cap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                         O: Optional[torch.Tensor] = None, LSE: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                         check_status: bool = True):
    """Attention where query i sees the keys lo[i] <= j < hi[i], on the current stream: packed documents, prefixes that
    see one another, windows, padding (mesh_ranges makes lo and hi).  q [B, Hq, S, d], k, v [B, Hkv, S, d], all bf16 or all
    fp32; lo, hi int32 [S] or [B, S] on the device, any values.  Scores are scale q.k (1 / sqrt(d) unless given), capped to
    cap tanh(score / cap) with cap > 0 (1e-18 to 1e18), less slopes[h] |i - j| with slopes (fp32 [Hq]).  Returns O (q's shape and dtype) and LSE
    (fp32 [B, Hq, S]); a query that sees nothing gets 0 and -inf.  A program that calls it every step keeps workspace
    (new_range_workspace) and status (new_status) and passes check_status=False, which leaves out the wait."""
    if workspace is None or status is None:
        load_binding().range_check(q, k, v, lo, hi, slopes)
    ws = new_range_workspace(q, k) if workspace is None else workspace
    st = new_status(q.device) if status is None else status
    out = (_ext or load_binding()).range_fwd(q, k, v, lo, hi, scale, cap, slopes, O, LSE, ws, st, None)
    if out.__class__ is int:
        _check(out, "mesh_attn_range_fwd")
    if check_status:
        _raise_status(st)
    return out


def mesh_range_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lo: torch.Tensor, hi: torch.Tensor,
                                  O: torch.Tensor, LSE: torch.Tensor, dO: torch.Tensor, scale: Optional[float] = None,
                                  cap: float = 0.0, slopes: Optional[torch.Tensor] = None, dQ: Optional[torch.Tensor] = None,
                                  dK: Optional[torch.Tensor] = None, dV: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                  check_status: bool = True):
    """(dQ, dK, dV) from the forward's O and LSE and the gradient dO, on the current stream."""
    if workspace is None or status is None:
        load_binding().range_check(q, k, v, lo, hi, slopes)
    ws = new_range_workspace(q, k, backward=True) if workspace is None else workspace
    st = new_status(q.device) if status is None else status
    out = (_ext or load_binding()).range_bwd(q, k, v, lo, hi, O, LSE, dO, scale, cap, slopes, dQ, dK, dV, ws, st, None)
    if out.__class__ is int:
        _check(out, "mesh_attn_range_bwd")
    if check_status:
        _raise_status(st)
    return out


class MeshRangeAttentionFunction(torch.autograd.Function):
    """torch.autograd binding of mesh_range_attention: gradients reach q, k and v; LSE is a non-differentiable output."""

    @staticmethod
    def forward(ctx, q, k, v, lo, hi, scale, cap, slopes, check_status, status):
        if ctx.needs_input_grad[7]:
            raise ValueError("slopes get no gradient: pass them detached")
        O, LSE = mesh_range_attention(q, k, v, lo, hi, scale, cap, slopes, status=status, check_status=check_status)
        ctx.save_for_backward(q, k, v, lo, hi, slopes, O, LSE)
        ctx.args = (scale, cap)
        ctx.check_status, ctx.status = check_status, status
        ctx.mark_non_differentiable(LSE)
        return O, LSE

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO, dLSE):
        q, k, v, lo, hi, slopes, O, LSE = ctx.saved_tensors
        grads = mesh_range_attention_backward(q, k, v, lo, hi, O, LSE, _dense_gradient(dO), *ctx.args, slopes, status=ctx.status,
                                              check_status=ctx.check_status)
        return (*grads, None, None, None, None, None, None, None)


def mesh_range_attention_autograd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lo: torch.Tensor, hi: torch.Tensor,
                                  scale: Optional[float] = None, cap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                                  check_status: bool = True, status: Optional[torch.Tensor] = None):
    """mesh_range_attention with autograd: returns (O, LSE); O.backward(...) fills the gradients of q, k and v.  With
    check_status=False a failure in either direction is recorded in `status` (new_status), for the program to read later.  Inside a
    captured graph take gradients with torch.autograd.grad, while no autograd graph made outside of it holds the same tensors."""
    return MeshRangeAttentionFunction.apply(q, k, v, lo, hi, scale, cap, slopes, check_status, status)
