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
clipping, AdamW.
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

_lib = None
_i64p = ctypes.POINTER(ctypes.c_int64)
_i32p = ctypes.POINTER(ctypes.c_int32)
_f32p = ctypes.POINTER(ctypes.c_float)
_vp = ctypes.c_void_p
_vpp = ctypes.POINTER(ctypes.c_void_p)

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
