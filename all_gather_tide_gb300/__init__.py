"""GB300 (sm_103a) layout-aware reduce-scatter and all-gather placement for FSDP2 groups.

A thin ctypes binding of ``libtide.so`` (C ABI in ``include/tide.h``).  Functions carry the C
names; they only marshal arguments (tensors -> device pointers, stream objects -> handles) and
turn negative statuses into :class:`TideError`.  Every step of the path runs in the library's
CUDA kernels or copy-engine calls; there is no Python or CPU fallback, and importing a function
fails loudly if the library has not been built.

"TIDE" is "The Endgame of FSDP Communication: Layout-Aware Collectives on Copy Engines, RDMA, and
NVSwitch" (arXiv 2610.38228): the reduce-scatter is its TIDE-RS (abstract; Fig. 2b), the
placement its TIDE-AG landing (abstract; Fig. 5b), the layout its Table 2.  Between the two, the
rest of a training step runs on the same shards: embedding lookup and gradient, the gradients' norm and
clipping, AdamW; and a layer of experts between the two: tokens to their experts and back, and products in
8-bit floating point with weights read from the shards and gradients written for the reduce-scatter.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtide.so")

TIDE_OK = 0
TIDE_EINVAL = -1
TIDE_EALIGN = -2
TIDE_ELAYOUT = -3
TIDE_ECUDA = -4
TIDE_ENOMEM = -5
TIDE_ERANGE = -6
TIDE_FLAG_VEC_STRICT = 0x1
TIDE_FLAG_CE_STRICT = 0x2
TIDE_FLAG_CE_2D = 0x4
TIDE_FLAG_OVERLAP = 0x8
TIDE_FLAG_CE_1D = 0x10
TIDE_RS_AUTO = 0
TIDE_RS_REGISTER = 1
TIDE_RS_BULK = 2
TIDE_RS_TMEM = 3
TIDE_AG_AUTO = 0
TIDE_AG_REGISTER = 1
TIDE_AG_BULK = 2
TIDE_DEBUG_STALL_PRODUCER = 0x1
TIDE_F32 = 0
TIDE_BF16 = 1
TIDE_I32 = 2
TIDE_I64 = 3
TIDE_SHORT_POSITIONS = 256
TIDE_SHORT_BATCHES = 64
TIDE_ADAMW_SKIP_NONFINITE = 0x1
TIDE_MAX_EXPERTS = 1024
TIDE_MAX_CHOICES = 32
TIDE_FP8_TRANSPOSED = 0x1
TIDE_FP8_ANY_SCALES = 0x2

_lib = None
_i64p = ctypes.POINTER(ctypes.c_int64)
_i32p = ctypes.POINTER(ctypes.c_int32)
_f32p = ctypes.POINTER(ctypes.c_float)
_vp = ctypes.c_void_p
_vpp = ctypes.POINTER(ctypes.c_void_p)


class _Fp8(ctypes.Structure):
    """tide_fp8_t"""

    _fields_ = [("codes", ctypes.c_void_p), ("stride", ctypes.c_int64), ("batch", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("scale_stride", ctypes.c_int64), ("scale_batch", ctypes.c_int64)]


_fp8p = ctypes.POINTER(_Fp8)

# name -> (restype, argtypes); every symbol declared in include/tide.h
SIGNATURES = {
    "tide_plan_layout": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, _i64p, _i64p, _i64p, _i64p, _i64p, _i64p, _i64p]),
    "tide_group_create": (ctypes.c_int, [_vpp, ctypes.c_int32, ctypes.c_int32, _i64p, _i64p, ctypes.c_uint32]),
    "tide_group_destroy": (ctypes.c_int, [_vp]),
    "tide_group_shard_elems": (ctypes.c_int, [_vp, _i64p]),
    "tide_group_unsharded_elems": (ctypes.c_int, [_vp, _i64p]),
    "tide_group_param_layout": (ctypes.c_int, [_vp, ctypes.c_int32, _i64p, _i64p]),
    "tide_group_valid_rows": (ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int32, _i64p]),
    "tide_group_set_ctas": (ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int32]),
    "tide_group_get_ctas": (ctypes.c_int, [_vp, _i32p, _i32p]),
    "tide_reduce_scatter": (ctypes.c_int, [_vp, _vpp, _vpp, _vp]),
    "tide_reduce_scatter_slots": (ctypes.c_int, [_vp, ctypes.c_int32, _vpp, _vp, _vp]),
    "tide_probe_mixed": (ctypes.c_int, [_vp, ctypes.c_int64, _vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, _vp, _vp]),
    "tide_stage_slices": (ctypes.c_int, [_vp, ctypes.c_int32, _vpp, _vpp, _vp]),
    "tide_all_gather": (ctypes.c_int, [_vp, _vpp, _vpp, _vp]),
    "tide_all_gather_ce": (ctypes.c_int, [_vp, _vpp, _vpp, _vp]),
    "tide_group_last_ce_copies": (ctypes.c_int, [_vp, _i64p, _i32p]),
    "tide_group_set_rs_variant": (ctypes.c_int, [_vp, ctypes.c_int32]),
    "tide_group_set_ag_variant": (ctypes.c_int, [_vp, ctypes.c_int32]),
    "tide_group_set_ce_lanes": (ctypes.c_int, [_vp, ctypes.c_int32]),
    "tide_group_set_ce_bands": (ctypes.c_int, [_vp, ctypes.c_int32]),
    "tide_group_ag_kernel": (ctypes.c_int, [_vp, _i32p]),
    "tide_group_rs_kernel": (ctypes.c_int, [_vp, _i32p]),
    "tide_group_set_wait_timeout": (ctypes.c_int, [_vp, ctypes.c_uint64]),
    "tide_group_device_status": (ctypes.c_int, [_vp, _i32p]),
    "tide_group_set_debug": (ctypes.c_int, [_vp, ctypes.c_uint32]),
    "tide_reduce_scatter_noalloc": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, _i64p, _i64p, _vpp, _vpp, _vp]),
    "tide_probe_hold": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64,
                                       _vp, _vp]),
    "tide_probe_bulk_read": (ctypes.c_int, [_vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp, _vp]),
    "tide_probe_ingest": (ctypes.c_int, [_vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp, _vp]),
    "tide_stage_into_slots": (ctypes.c_int, [_vp, _vpp, _vpp, ctypes.c_int64, _vpp, _vp]),
    "tide_embedding": (ctypes.c_int, [_vp, ctypes.c_int32, _vpp, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                      _vp, ctypes.c_int32, ctypes.c_int64, _vp]),
    "tide_embedding_grad_workspace": (ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int64, _i64p]),
    # n, ids, douts and dout_stride as addresses: the binding passes parts of one array
    "tide_embedding_grad": (ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int32, _vp, _vp, ctypes.c_int32, _vp, _vp,
                                           ctypes.c_int32, ctypes.c_float, ctypes.c_int32, _vpp, _vp, ctypes.c_int64,
                                           _vp]),
    "tide_tensors_create": (ctypes.c_int, [_vpp, ctypes.c_int32, _i64p, _i32p]),
    "tide_tensors_destroy": (ctypes.c_int, [_vp]),
    "tide_grad_norm": (ctypes.c_int, [_vp, _vpp, _vp, _vp, _vp]),
    "tide_clip_grads": (ctypes.c_int, [_vp, _vpp, _vp, ctypes.c_float, _vp]),
    "tide_clip_grad_norm": (ctypes.c_int, [_vp, _vpp, ctypes.c_float, _vp, _vp]),
    "tide_adamw": (ctypes.c_int, [_vp, _vpp, _vpp, _vpp, _vpp, _vpp, _f32p, ctypes.c_double, ctypes.c_double,
                                  ctypes.c_double, ctypes.c_double, ctypes.c_int64, _vp, ctypes.c_float, ctypes.c_uint32,
                                  _vp]),
    "tide_experts_create": (ctypes.c_int, [_vpp, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint32]),
    "tide_experts_destroy": (ctypes.c_int, [_vp]),
    "tide_experts_device_status": (ctypes.c_int, [_vp, _i32p]),
    "tide_experts_set_wait_timeout": (ctypes.c_int, [_vp, ctypes.c_uint64]),
    "tide_experts_set_debug": (ctypes.c_int, [_vp, ctypes.c_uint32]),
    "tide_experts_sort_workspace": (ctypes.c_int, [_vp, ctypes.c_int64, _i64p]),
    "tide_experts_sort": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, ctypes.c_int64, _vp, _vp, _vp, _vp, ctypes.c_int64, _vp]),
    "tide_experts_dispatch": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _vp, _vp,
                                             ctypes.c_int64, _vp]),
    "tide_experts_dispatch_fp8": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _vp, _fp8p,
                                                 _vp]),
    "tide_experts_combine": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _vp, _vp, _vp,
                                            ctypes.c_int64, _vp]),
    "tide_experts_combine_grad": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, ctypes.c_int64, _vp, ctypes.c_int64, ctypes.c_int64,
                                                 ctypes.c_int64, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp]),
    "tide_fp8_padded_rows": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int32, _i64p]),
    "tide_experts_quantize": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                             _vp, _vp, _fp8p, _fp8p, _vp]),
    "tide_all_gather_fp8": (ctypes.c_int, [_vp, ctypes.c_int32, _i32p, _vpp, _fp8p, _fp8p, _vp]),
    "tide_experts_matmul": (ctypes.c_int, [_vp, _fp8p, ctypes.c_int64, _vp, _fp8p, ctypes.c_uint32, ctypes.c_int64, ctypes.c_int64, _vp,
                                           ctypes.c_int32, ctypes.c_int64, _vp]),
    "tide_experts_weight_grad": (ctypes.c_int, [_vp, _fp8p, _fp8p, ctypes.c_int64, _vp, ctypes.c_uint32, ctypes.c_int64, ctypes.c_int64,
                                                _vpp, ctypes.c_int32, _vp]),
    "tide_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "tide_last_cuda_error": (ctypes.c_int, []),
    "tide_version": (ctypes.c_int, []),
}


class TideError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().tide_strerror(status).decode()
        if status == TIDE_ECUDA:
            msg += f" (cudaError {lib().tide_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [{status}]")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m all_gather_tide_gb300.build` "
                               "(or __graft_entry__.build()); there is no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != TIDE_OK:
        raise TideError(status, where)


def _ptr(x) -> int:
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _ptr_array(xs: Sequence) -> ctypes.Array:
    if isinstance(xs, ctypes.Array):  # already marshalled (see pointer_table)
        return xs
    return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def pointer_table(xs: Sequence) -> ctypes.Array:
    """Marshals tensors (or raw addresses) once into the pointer array the C calls take, for callers
    that pass the same buffers every step: a group with hundreds of parameters otherwise pays about
    a millisecond of Python per call to read R*P data pointers.  The tensors must stay alive and
    unmoved while the table is in use."""
    return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def float_table(xs: Sequence[float]) -> ctypes.Array:
    """Marshals per-tensor numbers (weight decays) once, as ``pointer_table`` does pointers."""
    return (ctypes.c_float * len(xs))(*xs)


_codes = {}


def _dtype_code(x) -> int:
    if not _codes:
        import torch

        _codes.update({torch.float32: TIDE_F32, torch.bfloat16: TIDE_BF16, torch.int32: TIDE_I32, torch.int64: TIDE_I64})
    code = _codes.get(x.dtype)
    if code is None:
        raise TideError(TIDE_EINVAL, f"a tensor of {x.dtype}")
    return code


_NAMES = {2: "bf16", 4: "fp32"}
_held = {}


def _held_as() -> dict:
    """Bytes of an element -> the types that hold it: fp32, or bf16, also as the 16-bit integers of its bits."""
    if not _held:
        import torch

        _held.update({4: (torch.float32,), 2: (torch.bfloat16, torch.int16, torch.uint16)})
    return _held


_gpus = 0  # that torch sees, once asked


def _current_device() -> int:
    import torch

    return torch.cuda.current_device()


def _elsewhere(*xs) -> bool:
    """Whether one of the GPU tensors lies on another GPU than the current one (which the C calls compare with the group's).
    Not asked again once there is found to be no other."""
    global _gpus
    if not _gpus:
        import torch

        _gpus = max(1, torch.cuda.device_count())
    if _gpus == 1:
        return False
    here = _current_device()
    return any(x.device.index not in (None, here) for x in xs)


_current_stream = None  # torch's functions for the current device and its current stream's handle


def _stream(stream) -> Optional[int]:
    if stream is None:
        global _current_stream
        if _current_stream is None:
            import torch

            _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        # the handle of torch.cuda.current_stream(), without building the stream object (3 us on Grace)
        device, handle = _current_stream
        return handle(device())
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _i64_array(xs: Sequence[int]):
    return (ctypes.c_int64 * len(xs))(*[int(x) for x in xs])


# ---- C-named functions ------------------------------------------------------------------------


def tide_version() -> int:
    return lib().tide_version()


def tide_strerror(status: int) -> str:
    return lib().tide_strerror(status).decode()


def tide_last_cuda_error() -> int:
    return lib().tide_last_cuda_error()


def tide_plan_layout(R: int, rows: Sequence[int], row_len: Sequence[int]):
    """Host-only planner: returns (m, s, o, S, U) as Python lists / ints."""
    P = len(rows)
    m, s, o = (ctypes.c_int64 * P)(), (ctypes.c_int64 * P)(), (ctypes.c_int64 * P)()
    S, U = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().tide_plan_layout(R, P, _i64_array(rows), _i64_array(row_len), m, s, o,
                                  ctypes.byref(S), ctypes.byref(U)), "tide_plan_layout")
    return list(m), list(s), list(o), S.value, U.value


def tide_group_create(R: int, rows: Sequence[int], row_len: Sequence[int], flags: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(lib().tide_group_create(ctypes.byref(h), R, len(rows), _i64_array(rows), _i64_array(row_len), flags),
           "tide_group_create")
    return h.value


def tide_group_destroy(g: int) -> None:
    _check(lib().tide_group_destroy(g), "tide_group_destroy")


def tide_group_shard_elems(g: int) -> int:
    v = ctypes.c_int64()
    _check(lib().tide_group_shard_elems(g, ctypes.byref(v)), "tide_group_shard_elems")
    return v.value


def tide_group_unsharded_elems(g: int) -> int:
    v = ctypes.c_int64()
    _check(lib().tide_group_unsharded_elems(g, ctypes.byref(v)), "tide_group_unsharded_elems")
    return v.value


def tide_group_param_layout(g: int, p: int) -> Tuple[int, int]:
    m, o = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().tide_group_param_layout(g, p, ctypes.byref(m), ctypes.byref(o)), "tide_group_param_layout")
    return m.value, o.value


def tide_group_valid_rows(g: int, d: int, p: int) -> int:
    v = ctypes.c_int64()
    _check(lib().tide_group_valid_rows(g, d, p, ctypes.byref(v)), "tide_group_valid_rows")
    return v.value


def tide_group_set_ctas(g: int, rs_ctas: int = 0, ag_ctas: int = 0) -> None:
    _check(lib().tide_group_set_ctas(g, rs_ctas, ag_ctas), "tide_group_set_ctas")


def tide_group_get_ctas(g: int) -> Tuple[int, int]:
    a, b = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().tide_group_get_ctas(g, ctypes.byref(a), ctypes.byref(b)), "tide_group_get_ctas")
    return a.value, b.value


def _flat_grads(grads):
    if isinstance(grads, ctypes.Array):
        return grads
    if len(grads) and isinstance(grads[0], (list, tuple)):
        return [x for row in grads for x in row]
    return list(grads)


def tide_reduce_scatter(g: int, grads, shards: Sequence, stream=None) -> None:
    """``grads``: R lists of P bf16 tensors (or a flat list indexed r*P+p, or raw pointers);
    ``shards``: R fp32 tensors of at least S elements."""
    _check(lib().tide_reduce_scatter(g, _ptr_array(_flat_grads(grads)), _ptr_array(shards), _stream(stream)),
           "tide_reduce_scatter")


def tide_stage_slices(g: int, d: int, grads, slots: Sequence, stream=None) -> None:
    """Copies slice d of every contributor's gradients into ``slots`` (R bf16 tensors of S elements)
    at the shard offsets, one copy-engine copy per (contributor, parameter)."""
    _check(lib().tide_stage_slices(g, d, _ptr_array(_flat_grads(grads)), _ptr_array(slots), _stream(stream)),
           "tide_stage_slices")


def tide_reduce_scatter_slots(g: int, d: int, slots: Sequence, shard, stream=None) -> None:
    """``slots``: R bf16 staging slots of S elements (slot r holds contributor r's slice d of every
    parameter at o_p); ``shard``: d's fp32 shard of S elements."""
    _check(lib().tide_reduce_scatter_slots(g, d, _ptr_array(slots), _ptr(shard), _stream(stream)),
           "tide_reduce_scatter_slots")


def tide_all_gather(g: int, shards: Sequence, params: Sequence, stream=None) -> None:
    _check(lib().tide_all_gather(g, _ptr_array(shards), _ptr_array(params), _stream(stream)), "tide_all_gather")


def tide_all_gather_ce(g: int, shards: Sequence, params: Sequence, stream=None) -> None:
    _check(lib().tide_all_gather_ce(g, _ptr_array(shards), _ptr_array(params), _stream(stream)),
           "tide_all_gather_ce")


def tide_group_set_rs_variant(g: int, variant: int) -> None:
    _check(lib().tide_group_set_rs_variant(g, variant), "tide_group_set_rs_variant")


def tide_group_set_ag_variant(g: int, variant: int) -> None:
    _check(lib().tide_group_set_ag_variant(g, variant), "tide_group_set_ag_variant")


def tide_group_ag_kernel(g: int) -> int:
    v = ctypes.c_int32()
    _check(lib().tide_group_ag_kernel(g, ctypes.byref(v)), "tide_group_ag_kernel")
    return v.value


def tide_group_rs_kernel(g: int) -> int:
    v = ctypes.c_int32()
    _check(lib().tide_group_rs_kernel(g, ctypes.byref(v)), "tide_group_rs_kernel")
    return v.value


def tide_group_set_ce_lanes(g: int, lanes: int) -> None:
    _check(lib().tide_group_set_ce_lanes(g, lanes), "tide_group_set_ce_lanes")


def tide_group_set_ce_bands(g: int, bands: int) -> None:
    _check(lib().tide_group_set_ce_bands(g, bands), "tide_group_set_ce_bands")


def tide_group_set_wait_timeout(g: int, timeout_ns: int) -> None:
    _check(lib().tide_group_set_wait_timeout(g, timeout_ns), "tide_group_set_wait_timeout")


def tide_group_device_status(g: int) -> int:
    v = ctypes.c_int32()
    _check(lib().tide_group_device_status(g, ctypes.byref(v)), "tide_group_device_status")
    return v.value


def tide_group_set_debug(g: int, flags: int) -> None:
    _check(lib().tide_group_set_debug(g, flags), "tide_group_set_debug")


def tide_reduce_scatter_noalloc(R: int, rows: Sequence[int], row_len: Sequence[int], grads, shards: Sequence,
                                stream=None) -> None:
    """Reduce-scatter without any allocation (for callers that cannot allocate device memory):
    the work tables go to the library's fixed device scratch array.  Same data layout as
    ``tide_reduce_scatter``; calls on different streams must not overlap."""
    _check(lib().tide_reduce_scatter_noalloc(R, len(rows), _i64_array(rows), _i64_array(row_len),
                                             _ptr_array(_flat_grads(grads)), _ptr_array(shards), _stream(stream)),
           "tide_reduce_scatter_noalloc")


def tide_stage_into_slots(g: int, grads, slots: Sequence, slot_elems: int, stream=None) -> List[int]:
    """Slot-Reuse staging: copies every rank's gradients into its slot (packed, no padding) and
    returns the R*P staged device addresses (flat, index r*P+p) for ``tide_reduce_scatter``."""
    flat = _flat_grads(grads)
    staged = (ctypes.c_void_p * len(flat))()
    _check(lib().tide_stage_into_slots(g, _ptr_array(flat), _ptr_array(slots), slot_elems, staged, _stream(stream)),
           "tide_stage_into_slots")
    return [int(x) for x in staged]


def tide_group_last_ce_copies(g: int) -> Tuple[int, bool]:
    n, u = ctypes.c_int64(), ctypes.c_int32()
    _check(lib().tide_group_last_ce_copies(g, ctypes.byref(n), ctypes.byref(u)), "tide_group_last_ce_copies")
    return n.value, bool(u.value)


def tide_probe_hold(ctas: int, threads: int, smem_bytes: int, cluster_size: int, hold_ns: int, records=None,
                    stream=None) -> None:
    """Resident probe CTAs (Fig. 4 spin kernels; Table 5 SM-id probe when ``records`` is given:
    a device uint64 tensor of 3*ctas entries receiving SM id, entry and exit ns per CTA)."""
    _check(lib().tide_probe_hold(ctas, threads, smem_bytes, cluster_size, hold_ns,
                                 _ptr(records) if records is not None else None, _stream(stream)), "tide_probe_hold")


def tide_probe_bulk_read(buf, nbytes: int, ctas: int, copy_bytes: int, stages: int, out, stream=None) -> None:
    """Bulk-copy read bandwidth probe; ``out`` is a device uint32/int32 tensor of 2 entries."""
    _check(lib().tide_probe_bulk_read(_ptr(buf), nbytes, ctas, copy_bytes, stages, _ptr(out), _stream(stream)),
           "tide_probe_bulk_read")


def tide_probe_ingest(buf, bulk_bytes: int, ldg_bytes: int, ctas: int, copy_bytes: int, stages: int,
                      consumer_warps: int, ldg_warps: int, out, stream=None) -> None:
    """Per-SM ingest probe (bulk copies read out of shared memory and/or 32-byte register loads);
    ``out`` is a device uint32/int32 tensor of 2 entries."""
    _check(lib().tide_probe_ingest(_ptr(buf), bulk_bytes, ldg_bytes, ctas, copy_bytes, stages, consumer_warps,
                                   ldg_warps, _ptr(out), _stream(stream)), "tide_probe_ingest")


def tide_probe_mixed(buf, bulk_bytes: int, st_buf, st_bytes: int, ctas: int, copy_bytes: int, stages: int,
                     consumer_warps: int, st_warps: int, out, stream=None, burst_rows: int = 0,
                     burst_vecs: int = 0) -> None:
    """Per-SM read/write sharing probe (bulk copies read out of shared memory while other warps
    write 32-byte vectors); ``out`` is a device int64 tensor of 3 entries (checksum, error flags,
    bytes written)."""
    _check(lib().tide_probe_mixed(_ptr(buf), bulk_bytes, _ptr(st_buf) if st_buf is not None else None, st_bytes,
                                  ctas, copy_bytes, stages, consumer_warps, st_warps, burst_rows, burst_vecs,
                                  _ptr(out), _stream(stream)),
           "tide_probe_mixed")


# ---- the sharded training step ------------------------------------------------------------------


def tide_embedding(g: int, p: int, shards: Sequence, ids, out, scale: float = 1.0, stream=None) -> None:
    """``shards``: R bf16 shards; ``ids``: contiguous int32 or int64 tensor of n ids; ``out``: bf16 or fp32
    tensor whose last dimension is the row and whose rows lie ``out.stride(-2)`` apart (n of them)."""
    _embedding(g, p, shards, ids, out, _row_stride(out), scale, stream)


def _embedding(g, p, shards, ids, out, stride, scale, stream) -> None:
    _check(lib().tide_embedding(g, p, _ptr_array(shards), ids.data_ptr(), _dtype_code(ids), ids.numel(), scale,
                                out.data_ptr(), _dtype_code(out), stride, _stream(stream)), "tide_embedding")


def _row_stride(x) -> int:
    """Elements between the rows of a tensor whose last dimension is contiguous."""
    return x.stride(-2) if x.dim() > 1 and x.shape[-2] > 1 else max(x.shape[-1], 1)


def tide_embedding_grad_workspace(g: int, p: int, n: int) -> int:
    v = ctypes.c_int64()
    _check(lib().tide_embedding_grad_workspace(g, p, n, ctypes.byref(v)), "tide_embedding_grad_workspace")
    return v.value


def tide_embedding_grad(g: int, p: int, ids: Sequence, douts: Sequence, shards: Sequence, workspace, scale: float = 1.0,
                        accumulate: bool = False, stream=None) -> None:
    """``ids`` and ``douts``: B tensors each (batch b: n_b ids, n_b rows); ``shards``: R fp32 shards;
    ``workspace``: contiguous tensor of ``tide_embedding_grad_workspace`` bytes, or None for a list that needs none
    (``TIDE_SHORT_POSITIONS`` positions in ``TIDE_SHORT_BATCHES`` batches at most)."""
    batches = [v for i, x in zip(ids, douts) for v in (i.numel(), i.data_ptr(), x.data_ptr(), _row_stride(x))]
    _embedding_grad(g, p, batches, ids[0], douts[0], shards, workspace, scale, accumulate, stream)


def _embedding_grad(g, p, batches, ids, dout, shards, workspace, scale, accumulate, stream) -> None:
    """``batches``: positions, address of the ids, address of the douts and their row stride, batch after batch; ``ids`` and
    ``dout``: one of each, for the types."""
    B = len(batches) // 4
    # the four arrays of the call in one
    a = (ctypes.c_int64 * (4 * B))(*batches[::4], *batches[1::4], *batches[2::4], *batches[3::4])
    at = ctypes.addressof(a)
    work, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check(lib().tide_embedding_grad(g, p, B, at, at + 8 * B, _dtype_code(ids), at + 16 * B, at + 24 * B, _dtype_code(dout),
                                     scale, accumulate, _ptr_array(shards), work, size, _stream(stream)), "tide_embedding_grad")


def tide_tensors_create(elems: Sequence[int], types=None) -> int:
    h = ctypes.c_void_p()
    K = len(elems)
    ty = None if types is None else (ctypes.c_int32 * K)(*types)
    _check(lib().tide_tensors_create(ctypes.byref(h), K, _i64_array(elems), ty), "tide_tensors_create")
    return h.value


def tide_tensors_destroy(t: int) -> None:
    _check(lib().tide_tensors_destroy(t), "tide_tensors_destroy")


def tide_grad_norm(t: int, grads: Sequence, norm, sumsq=None, stream=None) -> None:
    """``norm``: fp32 device tensor of one element; ``sumsq``: fp64 device tensor of one element or None."""
    _check(lib().tide_grad_norm(t, _ptr_array(grads), _ptr(norm), None if sumsq is None else _ptr(sumsq), _stream(stream)),
           "tide_grad_norm")


def tide_clip_grads(t: int, grads: Sequence, norm, max_norm: float, stream=None) -> None:
    _check(lib().tide_clip_grads(t, _ptr_array(grads), _ptr(norm), max_norm, _stream(stream)), "tide_clip_grads")


def tide_clip_grad_norm(t: int, grads: Sequence, max_norm: float, norm, stream=None) -> None:
    _check(lib().tide_clip_grad_norm(t, _ptr_array(grads), max_norm, _ptr(norm), _stream(stream)), "tide_clip_grad_norm")


def tide_adamw(t: int, params: Sequence, grads: Sequence, exp_avg: Sequence, exp_avg_sq: Sequence, shards=None, *, lr: float,
               betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay=None, step: int, norm=None,
               max_norm: float = 0.0, flags: int = 0, stream=None) -> None:
    """``weight_decay``: K values (a sequence, or a ``float_table``) or None; ``shards``: K bf16 tensors or None."""
    if weight_decay is not None and not isinstance(weight_decay, ctypes.Array):
        weight_decay = float_table(weight_decay)
    _check(lib().tide_adamw(t, _ptr_array(params), _ptr_array(grads), _ptr_array(exp_avg), _ptr_array(exp_avg_sq),
                            None if shards is None else _ptr_array(shards), weight_decay, lr, betas[0], betas[1], eps, step,
                            None if norm is None else _ptr(norm), max_norm, flags, _stream(stream)), "tide_adamw")


# ---- a layer of experts --------------------------------------------------------------------------


def tide_experts_create(E: int, k: int, flags: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(lib().tide_experts_create(ctypes.byref(h), E, k, flags), "tide_experts_create")
    return h.value


def tide_experts_destroy(x: int) -> None:
    _check(lib().tide_experts_destroy(x), "tide_experts_destroy")


def tide_experts_device_status(x: int) -> int:
    v = ctypes.c_int32()
    _check(lib().tide_experts_device_status(x, ctypes.byref(v)), "tide_experts_device_status")
    return v.value


def tide_experts_set_wait_timeout(x: int, timeout_ns: int) -> None:
    _check(lib().tide_experts_set_wait_timeout(x, timeout_ns), "tide_experts_set_wait_timeout")


def tide_experts_set_debug(x: int, flags: int) -> None:
    _check(lib().tide_experts_set_debug(x, flags), "tide_experts_set_debug")


def tide_experts_sort_workspace(x: int, T: int) -> int:
    v = ctypes.c_int64()
    _check(lib().tide_experts_sort_workspace(x, T, ctypes.byref(v)), "tide_experts_sort_workspace")
    return v.value


def _address(x) -> Optional[int]:
    return None if x is None else x.data_ptr()


def tide_experts_sort(x: int, ids, T: int, offsets, slots, tokens, workspace=None, stream=None) -> None:
    """``ids``: contiguous int32 or int64 tensor of T*k ids; ``offsets``, ``slots``, ``tokens``: int32 tensors; ``workspace``: contiguous
    tensor of ``tide_experts_sort_workspace`` bytes, or None where that is 0."""
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tide_experts_sort(x, ids.data_ptr(), _dtype_code(ids), T, offsets.data_ptr(), slots.data_ptr(), tokens.data_ptr(), _address(workspace), size,
                                   _stream(stream)), "tide_experts_sort")


def tide_experts_dispatch(x: int, src, slots, rows, stream=None) -> None:
    """``src``: T rows of bf16 or fp32; ``rows``: T*k of the same type; both 2-D, their rows contiguous."""
    _check(lib().tide_experts_dispatch(x, src.data_ptr(), _dtype_code(src), _row_stride(src), src.shape[0], src.shape[1], slots.data_ptr(), rows.data_ptr(),
                                       _row_stride(rows), _stream(stream)), "tide_experts_dispatch")


def tide_experts_dispatch_fp8(x: int, src, slots, rows, stream=None) -> None:
    """``rows``: an ``Fp8Rows``."""
    _check(lib().tide_experts_dispatch_fp8(x, src.data_ptr(), _dtype_code(src), _row_stride(src), src.shape[0], src.shape[1], slots.data_ptr(), rows.c,
                                           _stream(stream)), "tide_experts_dispatch_fp8")


def tide_experts_combine(x: int, rows, slots, weights, out, stream=None) -> None:
    """``weights``: T*k contiguous fp32, or None for 1."""
    _check(lib().tide_experts_combine(x, rows.data_ptr(), _dtype_code(rows), _row_stride(rows), out.shape[0], out.shape[1], slots.data_ptr(), _address(weights),
                                      out.data_ptr(), _row_stride(out), _stream(stream)), "tide_experts_combine")


def tide_experts_combine_grad(x: int, dout, rows, slots, weights, drows, dweights, stream=None) -> None:
    _check(lib().tide_experts_combine_grad(x, dout.data_ptr(), _dtype_code(dout), _row_stride(dout), rows.data_ptr(), _row_stride(rows), dout.shape[0],
                                           dout.shape[1], slots.data_ptr(), weights.data_ptr(), drows.data_ptr(), _row_stride(drows), dweights.data_ptr(),
                                           _stream(stream)), "tide_experts_combine_grad")


def tide_fp8_padded_rows(M: int, E: int) -> int:
    v = ctypes.c_int64()
    _check(lib().tide_fp8_padded_rows(M, E, ctypes.byref(v)), "tide_fp8_padded_rows")
    return v.value


def tide_experts_quantize(x: int, src, M: int, offsets, tokens=None, rows=None, columns=None, stream=None) -> None:
    """``rows``: an ``Fp8Rows`` or None; ``columns``: an ``Fp8Columns`` or None; ``tokens``: which row of ``src`` each is, or None."""
    _check(lib().tide_experts_quantize(x, src.data_ptr(), _dtype_code(src), _row_stride(src), src.shape[0], M, src.shape[1], _address(offsets), _address(tokens),
                                       None if rows is None else rows.c, None if columns is None else columns.c, _stream(stream)), "tide_experts_quantize")


def tide_all_gather_fp8(g: int, ps, shards: Sequence, w, stream=None) -> None:
    """``ps``: the parameters' indexes; ``w``: an ``Fp8Weights``."""
    if not isinstance(ps, ctypes.Array):
        ps = (ctypes.c_int32 * len(ps))(*ps)
    _check(lib().tide_all_gather_fp8(g, len(ps), ps, _ptr_array(shards), w.c, w.c_transposed, _stream(stream)), "tide_all_gather_fp8")


def tide_experts_matmul(x: int, a, offsets, w, out, flags: int = 0, stream=None) -> None:
    """``a``: an ``Fp8Rows``; ``w``: an ``Fp8Weights``; ``out``: bf16 or fp32 rows."""
    transposed = flags & TIDE_FP8_TRANSPOSED
    N, K = (w.K, w.N) if transposed else (w.N, w.K)
    codes = w.c_transposed if transposed else w.c
    _check(lib().tide_experts_matmul(x, a.c, a.M, _address(offsets), codes, flags, N, K, out.data_ptr(), _dtype_code(out), _row_stride(out), _stream(stream)),
           "tide_experts_matmul")


def tide_experts_weight_grad(x: int, dy, a, offsets, grads, grad_type: int = TIDE_BF16, flags: int = 0, stream=None) -> None:
    """``dy``, ``a``: ``Fp8Columns``; ``grads``: E tensors or the ``pointer_table`` of them."""
    _check(lib().tide_experts_weight_grad(x, dy.c, a.c, dy.M, _address(offsets), flags, dy.len, a.len, _ptr_array(grads), grad_type, _stream(stream)),
           "tide_experts_weight_grad")


def _refuse(where: str, what: str) -> None:
    raise TideError(TIDE_EINVAL, f"{where}: {what}")


# ---- convenience objects ----------------------------------------------------------------------


class Group:
    """Owns one ``tide_group_t``.  ``params`` is a list of ``(rows, row_len)`` pairs."""

    def __init__(self, R: int, params: Sequence[Tuple[int, int]], flags: int = 0):
        self.R = R
        self._table = ctypes.c_void_p * R  # the type of a pointer_table of R shards
        self.rows = [int(r) for r, _ in params]
        self.row_len = [int(l) for _, l in params]
        self.P = len(self.rows)
        self.handle = tide_group_create(R, self.rows, self.row_len, flags)
        self.S = tide_group_shard_elems(self.handle)
        self.U = tide_group_unsharded_elems(self.handle)

    def close(self) -> None:
        if self.handle:
            tide_group_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def param_layout(self, p: int) -> Tuple[int, int]:
        return tide_group_param_layout(self.handle, p)

    def valid_rows(self, d: int, p: int) -> int:
        return tide_group_valid_rows(self.handle, d, p)

    def set_ctas(self, rs_ctas: int = 0, ag_ctas: int = 0) -> None:
        tide_group_set_ctas(self.handle, rs_ctas, ag_ctas)

    def get_ctas(self) -> Tuple[int, int]:
        return tide_group_get_ctas(self.handle)

    def reduce_scatter(self, grads, shards, stream=None) -> None:
        tide_reduce_scatter(self.handle, grads, shards, stream)

    def stage_slices(self, d: int, grads, slots, stream=None) -> None:
        tide_stage_slices(self.handle, d, grads, slots, stream)

    def reduce_scatter_slots(self, d: int, slots, shard, stream=None) -> None:
        tide_reduce_scatter_slots(self.handle, d, slots, shard, stream)

    def all_gather(self, shards, params, stream=None) -> None:
        tide_all_gather(self.handle, shards, params, stream)

    def all_gather_ce(self, shards, params, stream=None) -> None:
        tide_all_gather_ce(self.handle, shards, params, stream)

    def last_ce_copies(self) -> Tuple[int, bool]:
        return tide_group_last_ce_copies(self.handle)

    def stage_into_slots(self, grads, slots, slot_elems: int, stream=None) -> List[int]:
        return tide_stage_into_slots(self.handle, grads, slots, slot_elems, stream)

    def set_rs_variant(self, variant: int) -> None:
        tide_group_set_rs_variant(self.handle, variant)

    def set_ag_variant(self, variant: int) -> None:
        tide_group_set_ag_variant(self.handle, variant)

    def ag_kernel(self) -> int:
        return tide_group_ag_kernel(self.handle)

    def rs_kernel(self) -> int:
        return tide_group_rs_kernel(self.handle)

    def set_ce_lanes(self, lanes: int) -> None:
        tide_group_set_ce_lanes(self.handle, lanes)

    def set_ce_bands(self, bands: int) -> None:
        tide_group_set_ce_bands(self.handle, bands)

    def set_wait_timeout(self, timeout_ns: int) -> None:
        tide_group_set_wait_timeout(self.handle, timeout_ns)

    def device_status(self) -> int:
        return tide_group_device_status(self.handle)

    def set_debug(self, flags: int) -> None:
        tide_group_set_debug(self.handle, flags)

    # ---- the sharded training step ----

    def embedding(self, p: int, shards: Sequence, ids, out, scale: float = 1.0, stream=None) -> None:
        """Rows ``ids`` of parameter p read from the R bf16 ``shards``, times ``scale``, into ``out``
        (``ids.numel()`` rows: ``[n, L]``, or contiguous ``[..., L]``)."""
        if type(shards) is not self._table:
            self._check_shards("embedding", shards, 2)
        stride = self._check_rows("embedding", p, ids, out)
        _embedding(self.handle, p, shards, ids, out, stride, scale, stream)

    def embedding_grad_workspace(self, p: int, n: int):
        """A device buffer that ``embedding_grad`` can work in for up to ``n`` positions."""
        import torch

        return torch.empty(tide_embedding_grad_workspace(self.handle, p, n), dtype=torch.uint8, device="cuda")

    def embedding_grad(self, p: int, ids: Sequence, douts: Sequence, shards: Sequence, scale: float = 1.0,
                       accumulate: bool = False, workspace=None, stream=None) -> None:
        """The lookup's gradient into the R fp32 ``shards``: ``ids`` and ``douts`` are lists of batches.
        Without a ``workspace`` one is allocated for the call, unless the list is short enough to need none."""
        where = "embedding_grad"
        if type(shards) is not self._table:
            self._check_shards(where, shards, 4)
        if not len(ids) == len(douts) > 0:
            _refuse(where, "one dout for each batch of ids, and one batch at least")
        kind, form, batches = ids[0].dtype, douts[0].dtype, []
        for i, x in zip(ids, douts):
            stride = self._check_rows(where, p, i, x)
            if i.dtype is not kind or x.dtype is not form:
                _refuse(where, "the batches differ in type")
            batches += i.numel(), i.data_ptr(), x.data_ptr(), stride
        self._check_workspace(where, workspace)
        if workspace is None and ((n := sum(batches[::4])) > TIDE_SHORT_POSITIONS or len(ids) > TIDE_SHORT_BATCHES):
            import torch

            workspace = self.embedding_grad_workspace(p, n)
            if stream is not None:
                s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
                s.wait_stream(torch.cuda.current_stream())
                workspace.record_stream(s)
        _embedding_grad(self.handle, p, batches, ids[0], douts[0], shards, workspace, scale, accumulate, stream)

    @staticmethod
    def _check_workspace(where: str, x) -> None:
        """Refuses all but a contiguous tensor on the GPU, or None."""
        if not (x is None or (not isinstance(x, int) and x.is_cuda and x.is_contiguous() and not (_gpus != 1 and _elsewhere(x)))):
            _refuse(where, "a workspace is a contiguous tensor on the GPU")

    def _check_shards(self, where: str, shards, size: int) -> None:
        """Refuses all but R shards (tensors are looked at; addresses and pointer tables are not)."""
        if len(shards) != self.R:
            _refuse(where, f"{self.R} shards are needed")
        if not isinstance(shards, ctypes.Array):
            types = _held_as()[size]
            for x in shards:
                if not isinstance(x, int) and not (x.is_cuda and x.dtype in types and x.numel() >= self.S and x.is_contiguous() and not (_gpus != 1 and _elsewhere(x))):
                    _refuse(where, f"a shard is {self.S} contiguous elements of {_NAMES[size]} on the GPU")

    def _check_rows(self, where: str, p: int, ids, rows) -> int:
        """Refuses ids and rows that do not fit parameter p; returns the rows' stride."""
        if not 0 <= p < self.P:
            _refuse(where, "no such parameter")
        n, length, shape = ids.numel(), self.row_len[p], rows.shape
        if not (ids.is_contiguous() and ids.is_cuda and rows.is_cuda) or (_gpus != 1 and _elsewhere(ids, rows)):
            _refuse(where, "contiguous ids, and rows, on the GPU are needed")
        if shape == (n, length):
            if rows.is_contiguous():
                return length
            stride, inner = rows.stride()
            if (length == 1 or inner == 1) and (n <= 1 or stride >= length):
                return stride if n > 1 else length
        elif len(shape) and shape[-1] == length and rows.numel() == n * length and rows.is_contiguous():
            return length
        _refuse(where, f"{n} rows of {length} elements, contiguous or a row stride apart, are needed")

    def all_gather_fp8(self, ps: Sequence[int], shards: Sequence, w: "Fp8Weights", stream=None) -> None:
        """All-gather placement in 8 bits: the parameters ``ps``, all of one shape, read from the R bf16 ``shards`` as the experts'
        matrices of ``w`` (and their transposes, where ``w`` has them)."""
        where = "all_gather_fp8"
        if type(shards) is not self._table:
            self._check_shards(where, shards, 2)
        if not isinstance(w, Fp8Weights) or len(ps) != w.E or (_gpus != 1 and _elsewhere(w.codes)):
            _refuse(where, "one parameter is needed for each matrix of an Fp8Weights on this GPU")
        for p in ps:
            if not 0 <= p < self.P or (self.rows[p], self.row_len[p]) != (w.N, w.K):
                _refuse(where, f"a parameter of {w.N} rows of {w.K} elements is needed")
        tide_all_gather_fp8(self.handle, ps, shards, w, stream)

    def pieces(self, buffers: Sequence) -> list:
        """The valid rows of every (rank, parameter) piece of R shard buffers, as R*P views in the order
        d*P + p: the tensors of a ``TensorList`` over the group's shards."""
        out = []
        for d in range(self.R):
            for p in range(self.P):
                o = self.param_layout(p)[1]
                out.append(buffers[d][o:o + self.valid_rows(d, p) * self.row_len[p]])
        return out


class TensorList:
    """Owns one ``tide_tensors_t``: K tensors of ``elems[k]`` elements whose gradients are of
    ``types[k]`` (``TIDE_F32``, the default, or ``TIDE_BF16``).  Its calls take K tensors each, or the
    ``pointer_table`` of them."""

    def __init__(self, elems: Sequence[int], types=None):
        self.elems = [int(n) for n in elems]
        self.K = len(self.elems)
        self._table = ctypes.c_void_p * self.K  # the type of a pointer_table of K tensors
        self.grad_bytes = [2 if t == TIDE_BF16 else 4 for t in types] if types is not None else [4] * self.K
        self.handle = None
        self.handle = tide_tensors_create(self.elems, types)

    def close(self) -> None:
        if self.handle:
            tide_tensors_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _tensors(self, where: str, xs, size: int = 0):
        """xs, once it has the list's count (and tensors its sizes); ``size``: bytes of an element, 0 for gradients."""
        if type(xs) is self._table:
            return xs
        if len(xs) != self.K:
            _refuse(where, f"{self.K} tensors are needed")
        if not isinstance(xs, ctypes.Array):
            types = _held_as()
            for n, b, x in zip(self.elems, self.grad_bytes, xs):
                if not isinstance(x, int) and not (x.numel() == n and x.is_cuda and x.is_contiguous() and x.dtype in types[size or b] and not (_gpus != 1 and _elsewhere(x))):
                    _refuse(where, f"a contiguous tensor of {n} elements of {_NAMES[size or b]} on the GPU is needed")
        return xs

    @staticmethod
    def _scalar(where: str, x, size: int = 4):
        """x, unless it is a tensor that cannot hold one number of `size` bytes on the GPU."""
        if not (x is None or isinstance(x, int)) and not (x.is_cuda and x.is_floating_point() and x.element_size() == size and x.numel() > 0 and not (_gpus != 1 and _elsewhere(x))):
            _refuse(where, f"a floating-point tensor of {size}-byte elements on the GPU is needed")
        return x

    def grad_norm(self, grads, norm, sumsq=None, stream=None) -> None:
        where = "grad_norm"
        tide_grad_norm(self.handle, self._tensors(where, grads), self._scalar(where, norm), self._scalar(where, sumsq, 8), stream)

    def clip_grads(self, grads, norm, max_norm: float, stream=None) -> None:
        where = "clip_grads"
        tide_clip_grads(self.handle, self._tensors(where, grads), self._scalar(where, norm), max_norm, stream)

    def clip_grad_norm(self, grads, max_norm: float, norm, stream=None) -> None:
        where = "clip_grad_norm"
        tide_clip_grad_norm(self.handle, self._tensors(where, grads), max_norm, self._scalar(where, norm), stream)

    def adamw(self, params, grads, exp_avg, exp_avg_sq, shards=None, *, weight_decay=None, stream=None, **hyper) -> None:
        """One step; ``lr``, ``betas``, ``eps``, ``step``, ``norm``, ``max_norm`` and ``flags`` as ``tide_adamw``.
        ``weight_decay``: one number for all tensors, K of them, or a ``float_table``."""
        where = "adamw"
        table = self._table
        if not (type(params) is type(grads) is type(exp_avg) is type(exp_avg_sq) is table and (shards is None or type(shards) is table)):
            self._tensors(where, grads)
            for xs in (params, exp_avg, exp_avg_sq):
                self._tensors(where, xs, 4)
            if shards is not None:
                self._tensors(where, shards, 2)
        self._scalar(where, hyper.get("norm"))
        if isinstance(weight_decay, (int, float)):
            weight_decay = [weight_decay] * self.K
        if weight_decay is not None and len(weight_decay) != self.K:
            _refuse(where, f"{self.K} weight decays are needed")
        tide_adamw(self.handle, params, grads, exp_avg, exp_avg_sq, shards, weight_decay=weight_decay, stream=stream, **hyper)


# ---- a layer of experts --------------------------------------------------------------------------


def _fp8_struct(codes, scales, batch: int = 0, scale_batch: int = 0):
    return _Fp8(codes.data_ptr(), codes.stride(-2), batch, scales.data_ptr(), scales.stride(-2), scale_batch)


def _up(n: int, to: int) -> int:
    return -(-n // to) * to


def _row_bytes(n: int) -> int:
    """The stride of rows of n codes: whole lines of 128 bytes, so that a block of a row lies in one (6002 rows of 1027 by 1003 columns
    take 16 us, rows of 1040 bytes 19)."""
    return _up(n, 128 if n > 128 else 16)


def _bytes_as_e4m3(*shape):
    import torch

    return torch.empty(*shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


class Fp8Rows:
    """M rows of ``len`` e4m3 ``codes`` and their fp32 ``scales``, one for each block of 128 columns: what
    ``dispatch_fp8`` and ``quantize`` write and ``matmul`` reads.  The value is ``codes[s, c] * scales[s, c // 128]``.  The calls
    use the memory that it was made with: other values are copied into these tensors (so of the other containers)."""""

    def __init__(self, M: int, len: int):
        import torch

        self.M, self.len = M, len
        self.codes = _bytes_as_e4m3(M, _row_bytes(len))[:, :len]
        self.scales = torch.empty(M, _up(-(-len // 128), 4), device="cuda")[:, :-(-len // 128)]
        self.c = _fp8_struct(self.codes, self.scales)


class Fp8Columns:
    """The transposed form of M rows of ``len`` columns in the order of E experts: ``len`` rows of ``codes`` in which each expert's
    rows begin at a multiple of 128, and the ``scales`` of their blocks of 128, [block, column]: what ``quantize`` writes and
    ``weight_grad`` reads."""

    def __init__(self, M: int, len: int, E: int):
        import torch

        self.M, self.len, self.E = M, len, E
        padded = max(128, tide_fp8_padded_rows(M, E))
        self.codes = _bytes_as_e4m3(len, padded)
        self.scales = torch.empty(padded // 128, _up(len, 4), device="cuda")[:, :len]
        self.c = _fp8_struct(self.codes, self.scales)


class Fp8Weights:
    """E matrices of N rows of K e4m3 ``codes`` ([E, N, K]) and their fp32 ``scales`` ([E, ceil(N / 128), ceil(K / 128)], one for each
    block of 128 x 128), and, with ``transposed``, the same codes transposed (``codes_transposed``, [E, K, N]) for products
    with the transposed matrices.  ``Group.all_gather_fp8`` writes them; a checkpoint's can be copied into them."""

    def __init__(self, E: int, N: int, K: int, transposed: bool = False):
        import torch

        codes = _bytes_as_e4m3(E, N, _row_bytes(K))[:, :, :K]
        scales = torch.empty(E, -(-N // 128), _up(-(-K // 128), 4), device="cuda")[:, :, :-(-K // 128)]
        self._hold(codes, scales, _bytes_as_e4m3(E, K, _row_bytes(N))[:, :, :N] if transposed else None)

    def _hold(self, codes, scales, codes_transposed) -> None:
        self.E, self.N, self.K = codes.shape
        self.codes, self.scales, self.codes_transposed = codes, scales, codes_transposed
        self.c = _fp8_struct(codes, scales, codes.stride(0), scales.stride(0))
        self.c_transposed = None
        if codes_transposed is not None:
            self.c_transposed = _fp8_struct(codes_transposed, scales, codes_transposed.stride(0), scales.stride(0))

    def part(self, first: int, rows: int) -> "Fp8Weights":
        """Rows ``first`` to ``first + rows`` of every matrix, in place: several parameters side by side in one product.  Both are
        multiples of 128, but the rows of the last part."""
        if first < 0 or rows < 1 or first % 128 or first + rows > self.N or (rows % 128 and first + rows != self.N):
            _refuse("part", "whole blocks of 128 rows are needed")
        end, w = first + rows, Fp8Weights.__new__(Fp8Weights)
        t = self.codes_transposed
        w._hold(self.codes[:, first:end], self.scales[:, first // 128:-(-end // 128)], None if t is None else t[:, :, first:end])
        return w


class Route:
    """The order of T tokens' pairs: ``offsets`` [E + 1], ``slots`` [T, k] and ``tokens`` [T*k], int32, as ``Experts.sort`` writes them.
    The calls use the memory that it was made with: another order is copied into these tensors."""""

    def __init__(self, experts: "Experts", T: int):
        import torch

        self.T, self.E, self.k = T, experts.E, experts.k
        self.M = T * experts.k
        self.offsets = torch.zeros(experts.E + 1, dtype=torch.int32, device="cuda")
        self.slots = torch.full((T, experts.k), -1, dtype=torch.int32, device="cuda")
        self.tokens = torch.full((self.M,), -1, dtype=torch.int32, device="cuda")
        size = tide_experts_sort_workspace(experts.handle, T)
        self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        # addresses, once: the buffers stay these
        self._at = self.offsets.data_ptr(), self.slots.data_ptr(), self.tokens.data_ptr(), _address(self.workspace), size


class Experts:
    """Owns one ``tide_experts_t``: E experts, k choices a token."""

    def __init__(self, E: int, k: int, flags: int = 0):
        self.E, self.k = E, k
        self._table = ctypes.c_void_p * E  # the type of a pointer_table of E gradients
        self._lib = lib()
        self.handle = None
        self.handle = tide_experts_create(E, k, flags)

    def close(self) -> None:
        if self.handle:
            tide_experts_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def device_status(self) -> int:
        return tide_experts_device_status(self.handle)

    def set_wait_timeout(self, timeout_ns: int) -> None:
        tide_experts_set_wait_timeout(self.handle, timeout_ns)

    def set_debug(self, flags: int) -> None:
        tide_experts_set_debug(self.handle, flags)

    def route(self, T: int) -> Route:
        """Buffers for the order of T tokens."""
        return Route(self, T)

    # ---- order, rows there and back ----

    def sort(self, ids, route: Route, stream=None) -> None:
        """The experts' order of the pairs with ``ids`` ([T, k], int32 or int64; negative: no expert) into ``route``."""
        where = "sort"
        self._check_route(where, route)
        if not (ids.is_cuda and ids.is_contiguous() and ids.numel() == route.M) or (_gpus != 1 and _elsewhere(ids)):
            _refuse(where, f"{route.M} contiguous ids on the GPU are needed")
        _check(self._lib.tide_experts_sort(self.handle, ids.data_ptr(), _dtype_code(ids), route.T, *route._at, _stream(stream)), where)

    def dispatch(self, x, route: Route, rows, stream=None) -> None:
        """The tokens' rows ``x`` ([T, D], bf16 or fp32) into ``rows`` ([T*k, D]) in the experts' order."""
        where = "dispatch"
        self._check_route(where, route)
        D, kind = x.shape[-1], _dtype_code(x)
        stride, to = self._check_rows(where, x, route.T, D, kind), self._check_rows(where, rows, route.M, D, kind)
        _check(self._lib.tide_experts_dispatch(self.handle, x.data_ptr(), kind, stride, route.T, D, route._at[1], rows.data_ptr(), to, _stream(stream)), where)

    def dispatch_fp8(self, x, route: Route, rows: Fp8Rows, stream=None) -> None:
        """The same into 8-bit ``rows``."""
        where = "dispatch_fp8"
        self._check_route(where, route)
        D, kind = x.shape[-1], _dtype_code(x)
        stride = self._check_rows(where, x, route.T, D, kind)
        self._check_fp8(where, rows, Fp8Rows, route.M, D)
        _check(self._lib.tide_experts_dispatch_fp8(self.handle, x.data_ptr(), kind, stride, route.T, D, route._at[1], rows.c, _stream(stream)), where)

    def combine(self, rows, route: Route, out, weights=None, stream=None) -> None:
        """The experts' ``rows`` ([T*k, D]) back at their tokens, ``out`` ([T, D]), summed with ``weights`` ([T, k] fp32; None: 1, the
        gradient of ``dispatch``)."""
        where = "combine"
        self._check_route(where, route)
        D, kind = rows.shape[-1], _dtype_code(rows)
        stride, to = self._check_rows(where, rows, route.M, D, kind), self._check_rows(where, out, route.T, D, kind)
        if weights is not None:
            self._check_weights(where, weights, route)
        _check(self._lib.tide_experts_combine(self.handle, rows.data_ptr(), kind, stride, route.T, D, route._at[1], _address(weights), out.data_ptr(), to,
                                              _stream(stream)), where)

    def combine_grad(self, dout, rows, route: Route, weights, drows, dweights, stream=None) -> None:
        """The gradients of ``combine`` with ``weights``, into ``drows`` and ``dweights``."""
        where = "combine_grad"
        self._check_route(where, route)
        D, kind = dout.shape[-1], _dtype_code(dout)
        stride, of, to = (self._check_rows(where, x, n, D, kind) for x, n in ((dout, route.T), (rows, route.M), (drows, route.M)))
        self._check_weights(where, weights, route)
        self._check_weights(where, dweights, route)
        _check(self._lib.tide_experts_combine_grad(self.handle, dout.data_ptr(), kind, stride, rows.data_ptr(), of, route.T, D, route._at[1], weights.data_ptr(),
                                                   drows.data_ptr(), to, dweights.data_ptr(), _stream(stream)), where)

    # ---- products in 8 bits ----

    def quantize(self, x, route: Optional[Route], rows: Optional[Fp8Rows] = None, columns: Optional[Fp8Columns] = None, gather: bool = False,
                 stream=None) -> None:
        """Rows in the experts' order in 8 bits: ``x`` ([T*k, D]), or with ``gather`` the tokens' rows ``x`` ([T, D]), as they are
        and/or transposed.  ``route`` may be None where one expert has all rows."""
        where = "quantize"
        if x.dim() != 2:
            _refuse(where, "rows are needed")
        n, D = x.shape
        M, offsets = self._all_rows(where, route, n)
        if gather and route is None:
            _refuse(where, "gathering needs a route")
        kind = _dtype_code(x)
        stride = self._check_rows(where, x, route.T if gather else M, D, kind)
        if rows is not None:
            self._check_fp8(where, rows, Fp8Rows, M, D)
        if columns is not None:
            self._check_fp8(where, columns, Fp8Columns, M, D)
        _check(self._lib.tide_experts_quantize(self.handle, x.data_ptr(), kind, stride, n, M, D, offsets, route._at[2] if gather else None,
                                               None if rows is None else rows.c, None if columns is None else columns.c, _stream(stream)), where)

    def matmul(self, a: Fp8Rows, w: Fp8Weights, route: Optional[Route], out, transposed: bool = False, any_scales: bool = False, stream=None) -> None:
        """Every expert's rows of ``a`` times its matrix of ``w``: ``out[s] = w[e] @ a[s]`` ([T*k, N], bf16 or fp32), or with ``transposed``
        ``w[e].T @ a[s]`` ([T*k, K]).  ``any_scales``: scales may be other numbers than powers of two (a checkpoint's)."""
        where = "matmul"
        if not isinstance(w, Fp8Weights) or w.E != self.E or (transposed and w.c_transposed is None) or (_gpus != 1 and _elsewhere(w.codes)):
            _refuse(where, f"the Fp8Weights of {self.E} experts on this GPU are needed, with transposed codes for a transposed product")
        N, K, codes = (w.K, w.N, w.c_transposed) if transposed else (w.N, w.K, w.c)
        M, offsets = self._all_rows(where, route, a.M if isinstance(a, Fp8Rows) else 0)
        self._check_fp8(where, a, Fp8Rows, M, K)
        kind = _dtype_code(out)
        to = self._check_rows(where, out, M, N, kind)
        flags = (TIDE_FP8_TRANSPOSED if transposed else 0) | (TIDE_FP8_ANY_SCALES if any_scales else 0)
        _check(self._lib.tide_experts_matmul(self.handle, a.c, M, offsets, codes, flags, N, K, out.data_ptr(), kind, to, _stream(stream)), where)

    def weight_grad(self, dy: Fp8Columns, a: Fp8Columns, route: Optional[Route], grads, grad_type: int = TIDE_BF16, any_scales: bool = False, stream=None) -> None:
        """The gradient of every expert's matrix, ``dy[e].T @ a[e]``, into ``grads``: E contiguous tensors of N*K elements, bf16 or
        fp32, one tensor [E, N, K], or the ``pointer_table`` of E tensors of ``grad_type``.  ``any_scales`` as ``matmul``'s."""
        where = "weight_grad"
        M, offsets = self._all_rows(where, route, dy.M if isinstance(dy, Fp8Columns) else 0)
        for x in (dy, a):
            self._check_fp8(where, x, Fp8Columns, M, x.len if isinstance(x, Fp8Columns) else 0)
        n = dy.len * a.len
        if type(grads) is not self._table:
            if isinstance(grads, (list, tuple)):
                if len(grads) != self.E:
                    _refuse(where, f"{self.E} gradients are needed")
                grad_type = _dtype_code(grads[0])
                for g in grads:
                    if not (g.is_cuda and g.dtype is grads[0].dtype and g.is_contiguous() and g.numel() == n) or (_gpus != 1 and _elsewhere(g)):
                        _refuse(where, f"contiguous gradients of {dy.len} x {a.len} elements of one type on the GPU are needed")
                grads = _ptr_array(grads)
            else:
                if isinstance(grads, ctypes.Array) or not (grads.is_cuda and grads.is_contiguous() and grads.numel() == self.E * n) or (_gpus != 1 and _elsewhere(grads)):
                    _refuse(where, f"a contiguous gradient of {self.E} x {dy.len} x {a.len} elements on the GPU is needed")
                grad_type = _dtype_code(grads)
                first, each = grads.data_ptr(), n * grads.element_size()
                grads = self._table(*range(first, first + self.E * each, each))
            if grad_type not in (TIDE_F32, TIDE_BF16):
                _refuse(where, "gradients are bf16 or fp32")
        _check(self._lib.tide_experts_weight_grad(self.handle, dy.c, a.c, M, offsets, TIDE_FP8_ANY_SCALES if any_scales else 0, dy.len, a.len, grads, grad_type,
                                                  _stream(stream)), where)

    # ---- checks ----

    def _check_route(self, where: str, route) -> None:
        if not isinstance(route, Route) or route.E != self.E or route.k != self.k or (_gpus != 1 and _elsewhere(route.offsets)):
            _refuse(where, f"a route of {self.E} experts and {self.k} choices on this GPU is needed")

    def _all_rows(self, where: str, route, M: int):
        """The rows of a product, and the address of their offsets: the route's, or without one all M of one expert."""
        if route is not None:
            self._check_route(where, route)
            return route.M, route._at[0]
        if self.E != 1:
            _refuse(where, "several experts need a route")
        return M, None

    @staticmethod
    def _check_rows(where: str, x, n: int, length: int, kind: int) -> int:
        """Refuses all but n rows of `length` contiguous elements on the GPU that do not overlap, of bf16 or fp32 as `kind` says; returns their
        stride."""
        if not (x.is_cuda and x.shape == (n, length) and length > 0) or (_gpus != 1 and _elsewhere(x)):
            _refuse(where, f"{n} rows of {length} elements on the GPU are needed")
        if kind > TIDE_BF16 or _dtype_code(x) != kind:
            _refuse(where, "rows are bf16 or fp32, and of one type in a call")
        if x.is_contiguous():
            return length
        stride, inner = x.stride()
        if not ((length == 1 or inner == 1) and (n <= 1 or stride >= length)):
            _refuse(where, "rows are contiguous, or a row stride apart")
        return stride if n > 1 else length

    @staticmethod
    def _check_weights(where: str, x, route: Route) -> None:
        if not (x.is_cuda and _dtype_code(x) == TIDE_F32 and x.is_contiguous() and x.numel() == route.M) or (_gpus != 1 and _elsewhere(x)):
            _refuse(where, f"{route.M} contiguous fp32 weights on the GPU are needed")

    def _check_fp8(self, where: str, x, kind, M: int, length: int) -> None:
        if not isinstance(x, kind) or x.M != M or x.len != length or (kind is Fp8Columns and x.E != self.E) or (_gpus != 1 and _elsewhere(x.codes)):
            _refuse(where, f"{kind.__name__} of {M} rows of {length} elements on this GPU are needed")
