"""Products of 8-bit matrices where CTAs hand parts of a tile to one another, and at the edges of their checks, on the GPU.

Where codes and scales are small powers of two and whole numbers, every sum is a whole number below 2^24, which fp32 holds: results are compared bit for
bit.
"""
import pytest
import torch

from test_gpu_experts import tide  # noqa: F401
from test_gpu_step import gen

pytestmark = pytest.mark.gpu


def small_fp8(g, x, most):
    """Codes 0, +-1 and +-2, and scales 2^0 to 2^most, each drawn by itself; their values in 64 bits."""
    table = torch.tensor([0x00, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8)  # e4m3's
    x.codes.view(torch.uint8).copy_(table[torch.randint(0, 5, tuple(x.codes.shape), generator=g)])
    x.scales.copy_(torch.exp2(torch.randint(0, most + 1, tuple(x.scales.shape), generator=g).float()))


def row_values(x):
    return x.codes.float().double() * x.scales.double().repeat_interleave(128, 1)[:, :x.len]


def weight_values(w):
    return w.codes.float().double() * w.scales.double().repeat_interleave(128, 1)[:, :w.N].repeat_interleave(128, 2)[:, :, :w.K]


def column_values(x):
    return x.codes.float().double() * x.scales.double().t().repeat_interleave(128, 1)


def routed_evenly(tide, E, each):
    """E experts with `each` rows each, in order."""
    ex = tide.Experts(E, 1)
    route = ex.route(E * each)
    ex.sort(torch.arange(E).repeat_interleave(each).view(-1, 1).cuda(), route)
    return ex, route


class Traffic:
    """Copies on another stream meanwhile, so that the CTAs of a pair are not always equally far."""

    def __init__(self):
        self.stream, self.a = torch.cuda.Stream(), torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        self.b = torch.empty_like(self.a)

    def more(self):
        with torch.cuda.stream(self.stream):
            for _ in range(4):
                self.b.copy_(self.a)


# ---- tiles of two CTAs -----------------------------------------------------------------------------


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E, each, N, K", [(3, 7000, 1024, 1300), (8, 2600, 768, 2048), (1, 20000, 1500, 700)])
def test_products_of_pairs_use_every_blocks_own_scales(tide, E, each, N, K, kind):
    """Each CTA of a pair writes the exponents of its rows, and the first one's products use both's: of a row, a column and a block each."""
    g = gen(N + K)
    ex, route = routed_evenly(tide, E, each)
    A, W = tide.Fp8Rows(E * each, K), tide.Fp8Weights(E, N, K, transposed=True)
    D = tide.Fp8Rows(E * each, N)
    small_fp8(g, A, 3), small_fp8(g, W, 2), small_fp8(g, D, 3)
    W.codes_transposed.view(torch.uint8).copy_(W.codes.view(torch.uint8).transpose(1, 2))
    w, a, d = weight_values(W), row_values(A).view(E, each, K), row_values(D).view(E, each, N)
    traffic = Traffic()
    for transposed, x, want in ((False, A, a @ w.transpose(1, 2)), (True, D, d @ w)):
        assert float(want.abs().max()) < 1 << 24
        want = want.flatten(0, 1).to(kind)
        out = torch.empty_like(want)
        for _ in range(10):
            out.fill_(55.0)
            traffic.more()
            ex.matmul(x, W, route, out, transposed=transposed)
            assert torch.equal(out, want)
    assert ex.device_status() == 0


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E, each, N, K", [(32, 1100, 768, 1024), (5, 3000, 1024, 2048)])
def test_gradients_of_pairs_use_every_blocks_own_scales(tide, E, each, N, K, kind):
    g = gen(N + K + 1)
    ex, route = routed_evenly(tide, E, each)
    dy, a = tide.Fp8Columns(E * each, N, E), tide.Fp8Columns(E * each, K, E)
    small_fp8(g, dy, 2), small_fp8(g, a, 2)
    per = -(-each // 128) * 128
    for x in (dy, a):
        for e in range(E):
            x.codes.view(torch.uint8)[:, e * per + each:(e + 1) * per] = 0
    p, q = (column_values(x)[:, :E * per].view(-1, E, per).transpose(0, 1) for x in (dy, a))
    want = p @ q.transpose(1, 2)
    assert float(want.abs().max()) < 1 << 24
    want, traffic = want.to(kind), Traffic()
    out = torch.empty_like(want)
    for _ in range(10):
        out.fill_(55.0)
        traffic.more()
        ex.weight_grad(dy, a, route, out)
        assert torch.equal(out, want)
    assert ex.device_status() == 0


# ---- any scales ------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("each, N, K", [(128, 128, 384), (100, 331, 515), (300, 203, 397)])
def test_gradients_with_any_scales_of_tiles_with_an_odd_number_of_blocks(tide, each, N, K, kind):
    """The lanes hand their columns' scales round in two buffers; a tile that ends after one or three blocks goes over to the next with lanes unequally far, where
    rows' ends leave by elements. Every CTA takes many such tiles."""
    E = 200
    g = gen(each + N)
    ex, route = routed_evenly(tide, E, each)
    dy, a = tide.Fp8Columns(E * each, N, E), tide.Fp8Columns(E * each, K, E)
    small_fp8(g, dy, 4), small_fp8(g, a, 4)
    dy.scales.mul_(3), a.scales.mul_(5)  # no powers of two, and whole numbers
    per = -(-each // 128) * 128
    for x in (dy, a):
        for e in range(E):
            x.codes.view(torch.uint8)[:, e * per + each:(e + 1) * per] = 0
    p, q = (column_values(x)[:, :E * per].view(-1, E, per).transpose(0, 1) for x in (dy, a))
    want = p @ q.transpose(1, 2)
    assert float(want.abs().max()) < 1 << 24
    want, traffic = want.to(kind), Traffic()
    out = torch.empty_like(want)
    for _ in range(10):
        out.fill_(55.0)
        traffic.more()
        ex.weight_grad(dy, a, route, out, any_scales=True)
        assert torch.equal(out, want)
    assert ex.device_status() == 0
