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


# ---- scales that are no powers of two ------------------------------------------------------------------


def odd_scales(tide, x):
    """The same with scales that cannot be read four at a time."""
    whole = torch.empty(*x.scales.shape[:-1], x.scales.shape[-1] // 4 * 4 + 5, device="cuda")
    x.scales = whole[..., 1:1 + x.scales.shape[-1]]
    x.c = tide._fp8_struct(x.codes, x.scales, *((x.codes.stride(0), x.scales.stride(0)) if x.codes.dim() == 3 else ()))
    return x


BAD = (1.5, 0.0, -2.0, 2.0 ** -130)


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("each, N, K", [(70, 330, 300), (9000, 1100, 700)])
def test_products_tell_of_every_scale_that_is_no_power_of_two(tide, each, N, K, odd):
    """In both tile shapes, for the first and the last row, one of the second CTA's, the first and the last block, of both operands and both products."""
    E = 3
    ex, route = routed_evenly(tide, E + 1, each)  # and an expert of which no row is taken
    route.offsets[E + 1] = route.offsets[E]
    M = (E + 1) * each
    A, D, W = tide.Fp8Rows(M, K), tide.Fp8Rows(M, N), tide.Fp8Weights(E + 1, N, K, transposed=True)
    if odd:
        A, D, W = odd_scales(tide, A), odd_scales(tide, D), odd_scales(tide, W)
        W.c_transposed = tide._fp8_struct(W.codes_transposed, W.scales, W.codes_transposed.stride(0), W.scales.stride(0))
    for x in (A, D, W):
        x.codes.view(torch.uint8).fill_(0x38)
        x.scales.fill_(2.0)
    W.codes_transposed.view(torch.uint8).fill_(0x38)
    A.scales[E * each:], D.scales[E * each:], W.scales[E] = 1.5, 1.5, 1.5  # of no row's product
    out = {False: torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), True: torch.empty(M, K, dtype=torch.bfloat16, device="cuda")}
    blocks = {A: -(-K // 128), D: -(-N // 128)}
    for transposed, x in ((False, A), (True, D)):
        def status():
            ex.matmul(x, W, route, out[transposed], transposed=transposed)
            return ex.device_status()

        assert status() == 0
        rows = sorted({0, 40, min(200, each - 1), each - 1, each, E * each - 1})
        places = [(x, (r, b)) for r in rows for b in (0, blocks[x] - 1)]
        places += [(W, (e, n, c)) for e in (0, E - 1) for n in (0, -(-N // 128) - 1) for c in (0, -(-K // 128) - 1)]
        for i, (y, place) in enumerate(places):
            y.scales[place] = BAD[i % len(BAD)]
            assert status() == 2, (transposed, place)
            y.scales[place] = 2.0
        assert status() == 0


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("each, N, K", [(300, 331, 260), (1500, 1100, 2100)])
def test_gradients_tell_of_every_scale_that_is_no_power_of_two(tide, each, N, K, odd):
    E = 10
    ex, route = routed_evenly(tide, E, each)
    M, per = E * each, -(-each // 128)
    dy, a = tide.Fp8Columns(M, N, E), tide.Fp8Columns(M, K, E)
    if odd:
        dy, a = odd_scales(tide, dy), odd_scales(tide, a)
    for x in (dy, a):
        x.codes.view(torch.uint8).fill_(0)
        x.scales.fill_(2.0)
        x.scales[E * per:] = 1.5  # behind the last expert's blocks
    grads = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")

    def status():
        ex.weight_grad(dy, a, route, grads)
        return ex.device_status()

    assert status() == 0
    for x in (dy, a):
        for i, (block, n) in enumerate([(b, n) for b in (0, per - 1, per, E * per - 1) for n in (0, 1, 130, 200, x.len - 2, x.len - 1)]):
            x.scales[block, n] = BAD[i % len(BAD)]
            assert status() == 2, (block, n)
            x.scales[block, n] = 2.0
    assert status() == 0


@pytest.mark.parametrize("scale, counts_as", [(1.5, 1.0), (-2.0, 2.0), (-3.9, 2.0), (0.0, 2.0 ** -127), (2.0 ** -130, 2.0 ** -127), (2.0 ** -127, 2.0 ** -127), (2.0 ** -126, 2.0 ** -126),
                                              (2.0 ** 127, 2.0 ** 127), (float("inf"), float("nan")), (float("nan"), float("nan"))])
@pytest.mark.parametrize("M, N", [(9, 130), (20000, 1024)])
def test_what_a_scale_counts_as(tide, M, N, scale, counts_as):
    """One block of codes 1 for each row: 32 of them are there, so a result is 32 times both scales. The other operand's scale keeps it in range."""
    K, other = 32, 2.0 ** 100 if counts_as < 1 else 2.0 ** -60
    ex, A, W = tide.Experts(1, 1), tide.Fp8Rows(M, K), tide.Fp8Weights(1, N, K)
    out = torch.empty(M, N, device="cuda")
    for x in (A, W):
        x.codes.view(torch.uint8).fill_(0x38)
    for mine, theirs in ((A, W), (W, A)):
        mine.scales.fill_(scale), theirs.scales.fill_(other)
        ex.matmul(A, W, None, out)
        want = torch.full_like(out, 32.0 * counts_as * other)
        assert torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(want, 7.0)) and bool((out.isnan() == want.isnan()).all())
        told = counts_as == counts_as and (scale != counts_as or scale < 2.0 ** -126)
        assert ex.device_status() == (2 if told else 0)


# ---- no rows, far rows ---------------------------------------------------------------------------------


def test_no_tokens(tide):
    """Every call with T = 0: nothing is read or written but the order's offsets and the gradients, which are zeros."""
    E, k, N, K = 5, 2, 96, 160
    ex, G = tide.Experts(E, k), tide.Group(2, [(N, K)] * E)
    route = ex.route(0)
    assert route.workspace is None
    empty = lambda rows, n: torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    x, y, out = empty(0, K), empty(0, N), empty(0, N)
    weights, dweights = torch.empty(0, k, device="cuda"), torch.empty(0, k, device="cuda")
    W, x8, dy8 = tide.Fp8Weights(E, N, K, transposed=True), tide.Fp8Rows(0, K), tide.Fp8Rows(0, N)
    xt8, dyt8 = tide.Fp8Columns(0, K, E), tide.Fp8Columns(0, N, E)
    G.all_gather_fp8(range(E), [torch.ones(G.S, device="cuda").bfloat16() for _ in range(2)], W)
    route.offsets.fill_(7)
    for buf in (xt8, dyt8):
        buf.codes.view(torch.uint8).fill_(0x7F), buf.scales.fill_(float("nan"))
    grads = [torch.full((N, K), 55.0, device="cuda") for _ in range(E)]
    for any_scales in (False, True):
        ex.sort(torch.empty(0, k, dtype=torch.int64, device="cuda"), route)
        ex.dispatch(x, route, empty(0, K))
        ex.dispatch_fp8(x, route, x8)
        ex.matmul(x8, W, route, y, any_scales=any_scales)
        ex.combine(y, route, out, weights)
        ex.combine_grad(out, y, route, weights, empty(0, N), dweights)
        ex.quantize(y, route, rows=dy8, columns=dyt8)
        ex.matmul(dy8, W, route, empty(0, K), transposed=True, any_scales=any_scales)
        ex.quantize(x, route, columns=xt8, gather=True)
        ex.weight_grad(dyt8, xt8, route, grads, any_scales=any_scales)
        assert not any(bool(g.any()) for g in grads) and not bool(route.offsets.any()) and ex.device_status() == 0
        for g in grads:
            g.fill_(55.0)


def test_gradients_of_offsets_past_32_bits(tide):
    """The rows, their gradients and the transposed rows lie past 2^32 bytes. Whole numbers: every sum is exact."""
    T, k, E, D, N = 300_000, 8, 4, 2048, 256
    M = T * k
    g = torch.Generator(device="cuda").manual_seed(3)
    whole = lambda *shape: torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).bfloat16()
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    ex = tide.Experts(E, k)
    route = ex.route(T)
    ex.sort(ids, route)
    rows, dout, weights = whole(M, D), whole(T, D), torch.randint(1, 4, (T, k), generator=g, device="cuda").float()
    drows, dweights = torch.empty(M, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, k, device="cuda")
    ex.combine_grad(dout, rows, route, weights, drows, dweights)
    assert rows.numel() * 2 > 1 << 33
    slots = route.slots.long()
    for j in range(k):
        for a in range(0, T, 30_000):
            b = min(T, a + 30_000)
            s, d = slots[a:b, j], dout[a:b].float()
            assert torch.equal(drows[s].float(), d * weights[a:b, j, None]) and torch.equal(dweights[a:b, j], (rows[s].float() * d).sum(1))
    # the weights' gradient: rows of 2048 columns and of 256, transposed
    del rows, drows
    dy = whole(M, N)
    xt, dt = tide.Fp8Columns(M, D, E), tide.Fp8Columns(M, N, E)
    ex.quantize(dout, route, columns=xt, gather=True)
    ex.quantize(dy, route, columns=dt)
    assert xt.codes.numel() > 1 << 32
    grads = torch.empty(E, N, D, device="cuda")
    offsets, tokens = route.offsets.tolist(), route.tokens.long()
    for any_scales in (False, True):
        ex.weight_grad(dt, xt, route, grads, any_scales=any_scales)
        for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
            want = torch.zeros(N, D, dtype=torch.float64, device="cuda")
            for i in range(a, b, 1 << 17):
                c = min(b, i + (1 << 17))
                want += (dy[i:c].float().t() @ dout[tokens[i:c]].float()).double()  # whole numbers below 2^24
            assert float(want.abs().max()) < 1 << 24 and torch.equal(grads[e].double(), want), e
    assert ex.device_status() == 0


# ---- the same by handle, and by several threads ------------------------------------------------------------


def test_calls_by_handle_give_the_same_bits(tide):
    """The functions of the C names against the methods of Experts."""
    E, k, T, N, K = 6, 3, 700, 200, 264
    g = gen(8)
    ex, route = tide.Experts(E, k), None
    route, other = ex.route(T), ex.route(T)
    ids, x = torch.randint(-1, E, (T, k), generator=g).cuda(), torch.randn(T, K, generator=g).bfloat16().cuda()
    weights, dout = torch.rand(T, k, generator=g).cuda(), torch.randn(T, N, generator=g).bfloat16().cuda()
    W = tide.Fp8Weights(E, N, K, transposed=True)
    small_fp8(g, W, 2)
    W.codes_transposed.view(torch.uint8).copy_(W.codes.view(torch.uint8).transpose(1, 2))
    M, h = T * k, ex.handle

    def run(r, sort, dispatch, dispatch_fp8, matmul, combine, combine_grad, quantize, weight_grad):
        rows, y, dy, dxr = (torch.zeros(M, n, dtype=torch.bfloat16, device="cuda") for n in (K, N, N, K))
        out, dweights, grads = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, k, device="cuda"), torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
        x8, dy8, xt8, dyt8 = tide.Fp8Rows(M, K), tide.Fp8Rows(M, N), tide.Fp8Columns(M, K, E), tide.Fp8Columns(M, N, E)
        sort(ids, r), dispatch(x, r, rows), dispatch_fp8(x, r, x8), matmul(x8, r, y, False), combine(y, r, weights, out)
        combine_grad(dout, y, r, weights, dy, dweights), quantize(dy, r, dy8, dyt8, False), matmul(dy8, r, dxr, True), quantize(x, r, None, xt8, True)
        weight_grad(dyt8, xt8, r, grads)
        return [r.offsets, r.slots, r.tokens, rows, y, out, dy, dweights, dxr, grads]

    T_ = tide.TIDE_FP8_TRANSPOSED
    by_object = run(route, ex.sort, ex.dispatch, ex.dispatch_fp8, lambda a, r, y, t: ex.matmul(a, W, r, y, transposed=t), lambda y, r, w, o: ex.combine(y, r, o, w), ex.combine_grad,
                    lambda v, r, q, c, gather: ex.quantize(v, r, rows=q, columns=c, gather=gather), ex.weight_grad)
    by_handle = run(other, lambda i, r: tide.tide_experts_sort(h, i, T, r.offsets, r.slots, r.tokens, r.workspace), lambda v, r, y: tide.tide_experts_dispatch(h, v, r.slots, y),
                    lambda v, r, q: tide.tide_experts_dispatch_fp8(h, v, r.slots, q), lambda a, r, y, t: tide.tide_experts_matmul(h, a, r.offsets, W, y, T_ if t else 0),
                    lambda y, r, w, o: tide.tide_experts_combine(h, y, r.slots, w, o), lambda d, y, r, w, dy, dw: tide.tide_experts_combine_grad(h, d, y, r.slots, w, dy, dw),
                    lambda v, r, q, c, gather: tide.tide_experts_quantize(h, v, M, r.offsets, r.tokens if gather else None, q, c),
                    lambda d, a, r, gr: tide.tide_experts_weight_grad(h, d, a, r.offsets, [gr[e] for e in range(E)]))
    assert all(torch.equal(p, q) for p, q in zip(by_object, by_handle)) and ex.device_status() == 0


def test_two_host_threads_at_once(tide):
    """One object, two host threads, a stream and buffers each."""
    import threading

    from test_gpu_experts import Layer

    a, b = Layer(tide, 2000, 4, 8, 384, 512, 2, 1), Layer(tide, 700, 4, 8, 384, 512, 2, 2)
    b.ex, b.route = a.ex, a.ex.route(700)
    torch.cuda.synchronize()
    failed = []

    def work(layer):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                layer.step(stream)
            stream.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(x,)) for x in (a, b)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    a.check()
    b.check()
