"""A layer of experts without a GPU: argument checks that fail before any CUDA call, and the binding's own."""
import ctypes

import pytest
import torch

from test_step_abi import _OnAnotherGpu, _OnGpu


@pytest.fixture(scope="module")
def tide():
    from all_gather_tide_gb300 import build

    build.build()
    import all_gather_tide_gb300 as t

    t.lib()
    return t


def test_null_handles_are_refused(tide):
    L, E, v, s = tide.lib(), tide.TIDE_EINVAL, ctypes.c_int64(), ctypes.c_int32()
    m, a = tide._Fp8(256, 16, 0, 256, 4, 0), (ctypes.c_void_p * 1)(256)
    ps = (ctypes.c_int32 * 1)(0)
    assert L.tide_experts_device_status(None, ctypes.byref(s)) == E
    assert L.tide_experts_set_wait_timeout(None, 0) == E
    assert L.tide_experts_set_debug(None, 0) == E
    assert L.tide_experts_sort_workspace(None, 1, ctypes.byref(v)) == E
    assert L.tide_experts_sort(None, 256, tide.TIDE_I64, 1, 256, 256, 256, None, 0, None) == E
    assert L.tide_experts_dispatch(None, 256, tide.TIDE_BF16, 8, 1, 8, 256, 256, 8, None) == E
    assert L.tide_experts_dispatch_fp8(None, 256, tide.TIDE_BF16, 8, 1, 8, 256, m, None) == E
    assert L.tide_experts_combine(None, 256, tide.TIDE_BF16, 8, 1, 8, 256, None, 256, 8, None) == E
    assert L.tide_experts_combine_grad(None, 256, tide.TIDE_BF16, 8, 256, 8, 1, 8, 256, 256, 256, 8, 256, None) == E
    assert L.tide_experts_quantize(None, 256, tide.TIDE_BF16, 8, 1, 1, 8, None, None, m, None, None) == E
    assert L.tide_experts_matmul(None, m, 1, None, m, 0, 8, 8, 256, tide.TIDE_BF16, 8, None) == E
    assert L.tide_experts_weight_grad(None, m, m, 1, None, 0, 8, 8, a, tide.TIDE_BF16, None) == E
    assert L.tide_all_gather_fp8(None, 1, ps, a, m, None, None) == E
    assert L.tide_experts_destroy(None) == tide.TIDE_OK


def test_creation_refusals(tide):
    L, h = tide.lib(), ctypes.c_void_p(5)
    for E, k, flags in ((0, 1, 0), (tide.TIDE_MAX_EXPERTS + 1, 1, 0), (4, 0, 0), (4, tide.TIDE_MAX_CHOICES + 1, 0), (4, 2, tide.TIDE_FLAG_VEC_STRICT), (4, 2, 0x40)):
        h.value = 5
        assert L.tide_experts_create(ctypes.byref(h), E, k, flags) == tide.TIDE_EINVAL
        assert h.value is None
    assert L.tide_experts_create(None, 4, 2, 0) == tide.TIDE_EINVAL


@pytest.mark.parametrize("E", [1, 3, 128, 1024])
@pytest.mark.parametrize("M", [0, 1, 2, 127, 128, 129, 5000])
def test_padded_rows_hold_every_split(tide, M, E):
    """The largest number of blocks of any split of M rows among E experts: as many experts as can have one row over a whole block."""
    v = ctypes.c_int64()
    assert tide.lib().tide_fp8_padded_rows(M, E, ctypes.byref(v)) == tide.TIDE_OK
    most = 0
    for used in range(1, min(M, E) + 1):  # `used` experts with at least one row; all but one with a single row, or one over
        most = max(most, used + (M - used) // 128)
    assert v.value == 128 * most


def test_padded_rows_refusals(tide):
    L, v = tide.lib(), ctypes.c_int64()
    assert L.tide_fp8_padded_rows(1, 1, None) == tide.TIDE_EINVAL
    for M, E in ((-1, 1), (1, 0), (1, tide.TIDE_MAX_EXPERTS + 1)):
        assert L.tide_fp8_padded_rows(M, E, ctypes.byref(v)) == tide.TIDE_EINVAL
    assert L.tide_fp8_padded_rows((1 << 31) - (1 << 18) + 1, 1, ctypes.byref(v)) == tide.TIDE_ERANGE
    assert L.tide_fp8_padded_rows((1 << 31) - (1 << 18), 1024, ctypes.byref(v)) == tide.TIDE_OK and v.value < 1 << 31


# ---- the binding's checks, with tensors that say they lie on the GPU ------------------------------


class _Lib:
    """Takes every call."""

    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture
def layer(tide, monkeypatch):
    """An Experts, a Route and 8-bit buffers whose tensors lie on the host."""
    monkeypatch.setattr(tide, "_gpus", 1)
    monkeypatch.setattr(tide, "_stream", lambda s: 0)
    for name in ("empty", "zeros", "full"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _real=real, **k: _real(*a, **{x: y for x, y in k.items() if x != "device"}))
    ex = tide.Experts.__new__(tide.Experts)
    ex.E, ex.k, ex.handle, ex._table, ex._lib = 5, 2, None, ctypes.c_void_p * 5, _Lib()
    monkeypatch.setattr(tide, "tide_experts_sort_workspace", lambda h, T: 0)
    return ex, tide.Route(ex, 3)


def _refused(tide, f):
    with pytest.raises(tide.TideError) as e:
        f()
    assert e.value.status == tide.TIDE_EINVAL


def test_what_does_not_fit_is_refused(tide, layer):
    ex, r = layer
    g = _OnGpu
    rows, x, out = (g(torch.zeros(n, 8)) for n in (6, 3, 3))
    bf = g(torch.zeros(6, 8, dtype=torch.bfloat16))
    half = g(torch.zeros(6, 8, dtype=torch.float16))
    w = g(torch.zeros(3, 2))
    ids = g(torch.zeros(3, 2, dtype=torch.int64))
    other = tide.Experts.__new__(tide.Experts)
    other.E, other.k, other.handle = 5, 3, None
    alien = tide.Route(other, 2)
    ex.sort(ids, r), ex.dispatch(x, r, rows), ex.combine(rows, r, out), ex.combine(rows, r, out, w), ex.combine_grad(x, rows, r, w, rows, w)
    for f in (lambda: ex.sort(ids, alien), lambda: ex.sort(ids, None), lambda: ex.sort(torch.zeros(3, 2, dtype=torch.int64), r),
              lambda: ex.sort(g(torch.zeros(3, 3, dtype=torch.int64)), r), lambda: ex.sort(g(torch.zeros(2, 3, dtype=torch.int64).t()), r),
              lambda: ex.dispatch(x, r, bf), lambda: ex.dispatch(x, r, x), lambda: ex.dispatch(rows, r, rows), lambda: ex.dispatch(torch.zeros(3, 8), r, rows),
              lambda: ex.dispatch(g(torch.zeros(8, 3).t()), r, rows), lambda: ex.dispatch(g(torch.zeros(1, 8).expand(3, 8)), r, rows),
              lambda: ex.combine(half, r, out), lambda: ex.combine(rows, r, rows), lambda: ex.combine(rows, r, out, g(torch.zeros(3, 3))),
              lambda: ex.combine(rows, r, out, g(torch.zeros(3, 2, dtype=torch.bfloat16))), lambda: ex.combine(rows, r, out, g(torch.zeros(2, 3).t())),
              lambda: ex.combine_grad(x, rows, r, w, rows, g(torch.zeros(3, 1))), lambda: ex.combine_grad(x, bf, r, w, rows, w)):
        _refused(tide, f)


def test_8_bit_operands_that_do_not_fit_are_refused(tide, layer):
    ex, r = layer
    g = _OnGpu
    q, c, w = tide.Fp8Rows(6, 40), tide.Fp8Columns(6, 40, 5), tide.Fp8Weights(5, 24, 40)
    x, y, rows = g(torch.zeros(3, 40)), g(torch.zeros(6, 24)), g(torch.zeros(6, 40))
    ex.dispatch_fp8(x, r, q), ex.quantize(rows, r, rows=q, columns=c), ex.quantize(x, r, columns=c, gather=True), ex.matmul(q, w, r, y)
    dy = tide.Fp8Columns(6, 24, 5)
    grads = [g(torch.zeros(24 * 40, dtype=torch.bfloat16)) for _ in range(5)]
    ex.weight_grad(dy, c, r, grads), ex.weight_grad(dy, c, r, g(torch.zeros(5, 24, 40))), ex.weight_grad(dy, c, r, tide.pointer_table([1] * 5))
    for f in (lambda: ex.dispatch_fp8(x, r, tide.Fp8Rows(6, 41)), lambda: ex.dispatch_fp8(x, r, tide.Fp8Rows(5, 40)), lambda: ex.dispatch_fp8(x, r, c),
              lambda: ex.quantize(rows, r, rows=c), lambda: ex.quantize(rows, r, columns=tide.Fp8Columns(6, 40, 4)), lambda: ex.quantize(x, r, rows=q),
              lambda: ex.quantize(rows, None, rows=q), lambda: ex.quantize(rows, r, rows=q, gather=True),
              lambda: ex.matmul(q, tide.Fp8Weights(4, 24, 40), r, y), lambda: ex.matmul(q, w, r, rows), lambda: ex.matmul(q, w, r, rows, transposed=True),
              lambda: ex.matmul(c, w, r, y), lambda: ex.matmul(tide.Fp8Rows(6, 39), w, r, y), lambda: ex.matmul(q, q, r, y),
              lambda: ex.weight_grad(dy, c, r, grads[:4]), lambda: ex.weight_grad(dy, c, r, grads[:4] + [g(torch.zeros(24 * 40))]), lambda: ex.weight_grad(dy, q, r, grads),
              lambda: ex.weight_grad(dy, c, r, g(torch.zeros(5, 24, 41))), lambda: ex.weight_grad(dy, c, r, tide.pointer_table([1] * 4)),
              lambda: ex.weight_grad(dy, c, r, g(torch.zeros(5, 24, 40, dtype=torch.int32)))):
        _refused(tide, f)


def test_containers_lie_as_the_calls_need_them(tide, layer):
    for M, n in ((1, 1), (7, 40), (129, 1027)):
        q, c, w = tide.Fp8Rows(M, n), tide.Fp8Columns(M, n, 3), tide.Fp8Weights(3, M, n, transposed=True)
        assert q.codes.shape == (M, n) and q.c.stride % 16 == 0 and q.c.stride >= n and q.scales.shape == (M, -(-n // 128)) and q.c.scale_stride % 4 == 0
        assert c.codes.shape[0] == n and c.codes.shape[1] % 128 == 0 and c.scales.shape == (c.codes.shape[1] // 128, n) and c.c.scale_stride % 4 == 0
        assert w.codes.shape == (3, M, n) and w.codes_transposed.shape == (3, n, M) and w.c.batch % 16 == 0 and w.c_transposed.batch % 16 == 0
        assert w.scales.shape == (3, -(-M // 128), -(-n // 128)) and w.c.scale_batch == w.scales.stride(0)
    w = tide.Fp8Weights(2, 300, 200, transposed=True)
    p = w.part(128, 172)
    assert (p.E, p.N, p.K) == (2, 172, 200) and p.c.codes == w.c.codes + 128 * w.c.stride and p.c.scales == w.c.scales + 4 * w.c.scale_stride
    assert p.c_transposed.codes == w.c_transposed.codes + 128 and p.c.batch == w.c.batch


def test_tensors_of_another_gpu_are_refused(tide, layer, monkeypatch):
    ex, r = layer
    monkeypatch.setattr(tide, "_gpus", 2)
    monkeypatch.setattr(tide, "_current_device", lambda: 0)
    x, rows = torch.zeros(3, 8), torch.zeros(6, 8)
    monkeypatch.setattr(ex, "_check_route", lambda *a: None)  # its buffers lie on the host here
    ex.dispatch(_OnGpu(x), r, _OnGpu(rows))
    for a, b in ((_OnGpu, _OnAnotherGpu), (_OnAnotherGpu, _OnGpu)):
        _refused(tide, lambda: ex.dispatch(a(x), r, b(rows)))
    _refused(tide, lambda: ex.sort(_OnAnotherGpu(torch.zeros(6, dtype=torch.int64)), r))
    _refused(tide, lambda: ex.combine(_OnGpu(rows), r, _OnGpu(x), _OnAnotherGpu(torch.zeros(3, 2))))
