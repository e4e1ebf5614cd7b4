"""Argument checks of the sharded training step's entry points that fail before any CUDA call, and
the layout helpers of the binding (no GPU needed)."""
import ctypes

import pytest
import torch

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def tide():
    from all_gather_tide_gb300 import build

    build.build()
    import all_gather_tide_gb300 as t

    t.lib()
    return t


def _i64(xs):
    return (ctypes.c_int64 * max(1, len(xs)))(*xs)


def _ptrs(n, value=256):
    return (ctypes.c_void_p * n)(*[value] * n)


def test_null_handles_are_refused(tide):
    L = tide.lib()
    a, v = _ptrs(1), ctypes.c_int64()
    E = tide.TIDE_EINVAL
    assert L.tide_embedding(None, 0, a, 256, tide.TIDE_I64, 1, 1.0, 256, tide.TIDE_F32, 8, None) == E
    assert L.tide_embedding_grad_workspace(None, 0, 1, ctypes.byref(v)) == E
    assert L.tide_embedding_grad(None, 0, 1, _i64([1]), a, tide.TIDE_I64, a, _i64([8]), tide.TIDE_F32, 1.0, 0, a, 256, 4096, None) == E
    assert L.tide_grad_norm(None, a, 256, None, None) == E
    assert L.tide_clip_grads(None, a, 256, 1.0, None) == E
    assert L.tide_clip_grad_norm(None, a, 1.0, 256, None) == E
    assert L.tide_adamw(None, a, a, a, a, a, None, 1e-3, 0.9, 0.99, 1e-8, 1, None, 0.0, 0, None) == E
    assert L.tide_tensors_destroy(None) == tide.TIDE_OK


def test_tensor_list_refusals(tide):
    L = tide.lib()
    h = ctypes.c_void_p()

    def create(elems, types=None, out=True, K=None):
        ty = None if types is None else (ctypes.c_int32 * len(types))(*types)
        return L.tide_tensors_create(ctypes.byref(h) if out else None, len(elems) if K is None else K, _i64(elems), ty)

    assert create([4], out=False) == tide.TIDE_EINVAL
    assert create([], K=0) == tide.TIDE_EINVAL
    assert create([4, -1]) == tide.TIDE_EINVAL
    assert create([4], [tide.TIDE_I32]) == tide.TIDE_EINVAL
    assert create([1 << 43]) == tide.TIDE_ERANGE
    assert create([1 << 42, 1]) == tide.TIDE_ERANGE
    assert create([1], K=(1 << 22) // 8 + 1) == tide.TIDE_ERANGE
    assert L.tide_tensors_create(ctypes.byref(h), 1, None, None) == tide.TIDE_EINVAL
    assert h.value is None


def test_binding_marshals_types_and_strides(tide):
    assert [tide._dtype_code(torch.empty(1, dtype=d)) for d in (torch.float32, torch.bfloat16, torch.int32, torch.int64)] == [0, 1, 2, 3]
    with pytest.raises(tide.TideError) as e:
        tide._dtype_code(torch.empty(1, dtype=torch.float16))
    assert e.value.status == tide.TIDE_EINVAL
    assert tide._row_stride(torch.empty(5, 7)) == 7
    assert tide._row_stride(torch.empty(5, 9)[:, :7]) == 9
    assert tide._row_stride(torch.empty(1, 7)) == 7
    assert tide._row_stride(torch.empty(7)) == 7
    assert tide._row_stride(torch.empty(2, 3, 7)) == 7
    assert list(tide.float_table([0.5, 2.0])) == [0.5, 2.0]


class _Shape:
    """The layout part of a Group, for the checks that need no device."""

    def __init__(self, tide, R, params):
        self.R, self.P = R, len(params)
        self.rows, self.row_len = [r for r, _ in params], [l for _, l in params]
        self.m, _, self.o, self.S, _ = tide.tide_plan_layout(R, self.rows, self.row_len)

    def param_layout(self, p):
        return self.m[p], self.o[p]

    def valid_rows(self, d, p):
        return max(0, min(self.m[p], self.rows[p] - d * self.m[p]))


def test_pieces_are_the_valid_rows(tide):
    g = _Shape(tide, 4, [(5, 3), (7, 4), (2, 6)])
    buffers = [torch.arange(g.S) + 1000 * d for d in range(4)]
    views = tide.Group.pieces(g, buffers)
    assert len(views) == 12
    for d in range(4):
        for p in range(3):
            n = g.valid_rows(d, p) * g.row_len[p]
            want = torch.arange(n) + g.o[p] + 1000 * d
            assert torch.equal(views[d * 3 + p], want)
    assert sum(v.numel() for v in views) == 5 * 3 + 7 * 4 + 2 * 6


class _OnGpu:
    """A CPU tensor that says it lies on the GPU, for checks that look no further."""

    def __init__(self, x):
        self.x = x

    def __getattr__(self, name):
        return True if name == "is_cuda" else getattr(self.x, name)


@pytest.mark.parametrize("ids, rows", [
    (torch.zeros(6, dtype=torch.int64)[::2], torch.empty(3, 4)),  # ids with gaps
    (torch.zeros(3, dtype=torch.int64), torch.empty(3, 5)),  # another row length
    (torch.zeros(3, dtype=torch.int64), torch.empty(2, 4)),  # too few rows
    (torch.zeros(3, dtype=torch.int64), torch.empty(4, 3).t()),  # rows that are not contiguous
    (torch.zeros(3, dtype=torch.int64), torch.empty(1, 4).expand(3, 4)),  # rows in one place
])
def test_rows_that_do_not_fit_are_refused(tide, ids, rows):
    g = _Shape(tide, 2, [(7, 4)])
    check = lambda i, x: tide.Group._check_rows(g, "embedding", 0, _OnGpu(i), _OnGpu(x))
    with pytest.raises(tide.TideError) as e:
        check(ids, rows)
    assert e.value.status == tide.TIDE_EINVAL
    assert check(torch.zeros(3, dtype=torch.int64), torch.empty(3, 6)[:, :4]) == 6
    assert check(torch.zeros(2, 3, dtype=torch.int64), torch.empty(2, 3, 4)) == 4
    assert check(torch.zeros(1, dtype=torch.int64), torch.empty(1, 4)) == 4


def test_tensors_of_the_host_are_refused(tide):
    g = _Shape(tide, 2, [(7, 4)])
    i, x = torch.zeros(3, dtype=torch.int64), torch.empty(3, 4)
    refused = [lambda: tide.Group._check_rows(g, "embedding", 0, i, _OnGpu(x)), lambda: tide.Group._check_rows(g, "embedding", 0, _OnGpu(i), x),
               lambda: tide.Group._check_shards(g, "embedding", [torch.empty(g.S)] * 2, 4),
               lambda: tide.Group._check_shards(g, "embedding", [_OnGpu(torch.empty(g.S))] * 2, 2),  # the element size of the other kind
               lambda: tide.Group._check_shards(g, "embedding", [_OnGpu(torch.empty(g.S - 1))] * 2, 4),
               lambda: tide.TensorList._scalar("grad_norm", torch.empty(1)),
               lambda: tide.TensorList._scalar("grad_norm", _OnGpu(torch.empty(1, dtype=torch.int32)))]
    for f in refused:
        with pytest.raises(tide.TideError) as e:
            f()
        assert e.value.status == tide.TIDE_EINVAL
    tide.Group._check_shards(g, "embedding", [_OnGpu(torch.empty(g.S))] * 2, 4)
    tide.Group._check_shards(g, "embedding", tide.pointer_table([1, 2]), 4)


def test_a_workspace_of_the_host_or_with_gaps_is_refused(tide):
    for bad in (torch.empty(4096, dtype=torch.uint8), _OnGpu(torch.empty(8192, dtype=torch.uint8)[::2]), 4096):
        with pytest.raises(tide.TideError) as e:
            tide.Group._check_workspace("embedding_grad", bad)
        assert e.value.status == tide.TIDE_EINVAL
    for good in (None, _OnGpu(torch.empty(4096, dtype=torch.uint8)), _OnGpu(torch.empty(64, 16))):
        tide.Group._check_workspace("embedding_grad", good)


@pytest.mark.parametrize("size, right, wrong", [(2, (torch.bfloat16, torch.int16, torch.uint16), (torch.float16,)), (4, (torch.float32,), (torch.int32, torch.uint32))], ids=str)
def test_tensors_of_another_type_of_the_same_size_are_refused(tide, size, right, wrong):
    g = _Shape(tide, 2, [(7, 4)])

    class List:  # what _tensors looks at of a TensorList
        elems, K, grad_bytes, _table = [5, 3], 2, [size, size], ctypes.c_void_p * 2

    def calls(dtype):
        a, b = (_OnGpu(torch.zeros(n, dtype=dtype)) for n in List.elems)
        return (lambda: tide.Group._check_shards(g, "embedding", [_OnGpu(torch.zeros(g.S, dtype=dtype))] * 2, size),
                lambda: tide.TensorList._tensors(List, "adamw", [a, b], size), lambda: tide.TensorList._tensors(List, "grad_norm", [a, b]))

    for dtype in right:
        for f in calls(dtype):
            f()
    for dtype in wrong:
        for f in calls(dtype):
            with pytest.raises(tide.TideError) as e:
                f()
            assert e.value.status == tide.TIDE_EINVAL


class _OnAnotherGpu(_OnGpu):
    def __getattr__(self, name):
        return torch.device("cuda", 1) if name == "device" else super().__getattr__(name)


def test_tensors_of_another_gpu_are_refused(tide, monkeypatch):
    """Where there are several, all of a call's lie on the current one, which is the group's."""
    g, here, there = _Shape(tide, 2, [(7, 4)]), _OnGpu, _OnAnotherGpu
    ids, x, shard, work = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 4), torch.zeros(g.S), torch.zeros(64)

    class List:
        elems, K, grad_bytes, _table = [5], 1, [4], ctypes.c_void_p

    calls = [lambda a, b: tide.Group._check_rows(g, "embedding", 0, a(ids), b(x)), lambda a, b: tide.Group._check_shards(g, "embedding", [a(shard), b(shard)], 4),
             lambda a, b: tide.Group._check_workspace("embedding_grad", (b if a is here else a)(work)),
             lambda a, b: tide.TensorList._tensors(List, "grad_norm", [(b if a is here else a)(torch.zeros(5))]),
             lambda a, b: tide.TensorList._scalar("grad_norm", (b if a is here else a)(torch.zeros(1)))]
    monkeypatch.setattr(tide, "_gpus", 2)
    monkeypatch.setattr(tide, "_current_device", lambda: 0)
    for f in calls:
        f(here, here)
        for a, b in ((here, there), (there, here)):
            with pytest.raises(tide.TideError) as e:
                f(a, b)
            assert e.value.status == tide.TIDE_EINVAL
    monkeypatch.setattr(tide, "_current_device", lambda: 1)
    calls[0](there, there)
