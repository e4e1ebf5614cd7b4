"""A layer of experts on the GPU, against plain implementations in 64 bits.

Order, copies, codes and scales are compared bit for bit.  Sums of n products in fp32 (u = 2^-24) are off by at most
(n + 1) u times the sum of the products' magnitudes, and the result by half a step of its type more.  In a product of
8-bit matrices the products are exact and added by the tensor cores, 32 at a time, taken to lose at most 2u of the magnitudes
so far with each step of 32 and of the block's with each product; blocks' sums that are scaled apart have at most three
roundings each and are added in fp32: (128 + blocks + 3) * 2u of the sum of all magnitudes bounds both up to 33 blocks.  Buffers have guard bands around them.
"""
import ctypes

import pytest
import torch

from test_gpu_step import TYPES, U, Guarded, gen

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step, relative to the value


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import all_gather_tide_gb300 as t

    t.lib()
    return t


# ---- plain forms ---------------------------------------------------------------------------------


def order_of(ids, E):
    """offsets, slots, tokens of [T, k] CPU ids, pair by pair."""
    T, k = ids.shape
    flat = [int(i) for i in ids.flatten()]
    rows = [i for e in range(E) for i in [j for j, x in enumerate(flat) if x == e]] if len(flat) * E <= 100000 else None
    if rows is None:
        x = ids.flatten().long()
        held = (x >= 0) & (x < E)
        rows = torch.argsort(torch.where(held, x, E), stable=True)[:int(held.sum())].tolist()
    offsets = torch.tensor([sum(1 for x in flat if 0 <= x < e) for e in range(E + 1)] if len(flat) * E <= 100000 else
                           [0] + torch.bincount(ids.flatten()[(ids.flatten() >= 0) & (ids.flatten() < E)].long(), minlength=E).cumsum(0).tolist())
    slots, tokens = torch.full((T * k,), -1), torch.full((T * k,), -1)
    r = torch.tensor(rows, dtype=torch.long)
    slots[r] = torch.arange(len(rows))
    tokens[:len(rows)] = r // k
    return offsets, slots.view(T, k), tokens


def draw_ids(g, T, k, E, masked=0.1):
    ids = torch.randint(0, E, (T, k), generator=g)
    ids = torch.minimum(ids, torch.randint(0, E, (T, k), generator=g))  # low experts are more popular; choices may repeat
    ids[torch.rand(T, k, generator=g) < masked] = -1
    return ids


def e4m3(x, dims):
    """Codes (as values) and scales of x in 64 bits, one power of two for each block over `dims`, by comparison with every candidate."""
    amax = x.abs().amax(dims, keepdim=True)
    bad = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(bad | (amax == 0), torch.ones_like(amax), amax))
    p = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 120)
    scale = torch.where(amax == 0, 1.0, torch.ldexp(torch.ones_like(amax), p))
    scale = torch.where(bad, float("nan"), scale)
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(bad, float("nan"), torch.round(y / step) * step), scale


def in_rows(x):
    """[n, len] -> codes [n, len], scales [n, blocks]"""
    parts = [e4m3(x[:, c:c + 128].double(), (1,)) for c in range(0, x.shape[1], 128)]
    return torch.cat([c for c, _ in parts], 1), torch.cat([s for _, s in parts], 1)


def in_blocks(w):
    """[N, K] -> codes, scales [N / 128, K / 128]"""
    rows = []
    for n in range(0, w.shape[0], 128):
        parts = [e4m3(w[n:n + 128, c:c + 128].double(), (0, 1)) for c in range(0, w.shape[1], 128)]
        rows.append((torch.cat([c for c, _ in parts], 1), torch.cat([s for _, s in parts], 1)))
    return torch.cat([c for c, _ in rows]), torch.cat([s for _, s in rows])


def values(codes, scales):
    """Codes times the scales of their blocks of 128 in the last dimension."""
    return codes * scales.repeat_interleave(128, -1)[..., :codes.shape[-1]]


def same(a, b):
    """Equal, NaN where NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def routed(tide, E, k, ids, kind="i64", flags=0):
    ex = tide.Experts(E, k, flags)
    route = ex.route(ids.shape[0])
    ex.sort(ids.to(TYPES[kind]).cuda(), route)
    return ex, route


# ---- order ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("E", [1, 2, 31, 128, 1000, 1024])
@pytest.mark.parametrize("T, k", [(0, 2), (1, 1), (1, 8), (3, 5), (77, 3), (400, 32), (2048, 2), (2049, 2), (20011, 1), (40000, 8)])
def test_sort(tide, T, k, E):
    for masked, kind in ((0.0, "i64"), (0.3, "i32"), (1.0, "i64")):
        ids = draw_ids(gen(T + E), T, k, E, masked)
        offsets, slots, tokens = order_of(ids, E)
        ex = tide.Experts(E, k)
        route = ex.route(T)
        for x in (route.offsets, route.slots, route.tokens):
            x.fill_(-7)
        ex.sort(ids.to(TYPES[kind]).cuda(), route)
        assert torch.equal(route.offsets.cpu().long(), offsets)
        assert torch.equal(route.slots.cpu().long(), slots)
        assert torch.equal(route.tokens.cpu().long(), tokens)
        assert ex.device_status() == 0


@pytest.mark.parametrize("T", [5, 5000])
def test_sort_ids_past_the_experts(tide, T):
    ids = torch.full((T, 2), 3)
    ids[T // 2] = torch.tensor([4, 1 << 40])
    ids[0] = torch.tensor([-(1 << 40), 0])
    ex, route = routed(tide, 4, 2, ids)
    assert torch.equal(route.slots.cpu().long(), order_of(ids, 4)[1])
    assert ex.device_status() == 64 and ex.device_status() == 0


def test_sort_on_few_ctas(tide):
    ids = draw_ids(gen(1), 9000, 4, 60)
    ex, route = routed(tide, 60, 4, ids, flags=tide.TIDE_FLAG_OVERLAP)
    want = order_of(ids, 60)
    for x, y in zip((route.offsets, route.slots, route.tokens), want):
        assert torch.equal(x.cpu().long(), y)


# ---- rows there and back --------------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 3, 8, 100, 256, 1027, 2048, 4100])
def test_rows_there_and_back(tide, D, kind):
    g = gen(D)
    for T, k, E, shift, pad, masked in ((1, 1, 1, 0, 0, 0.0), (40, 8, 7, 0, 0, 0.1), (33, 3, 50, 1, 3, 0.5), (130, 32, 9, 2, 2, 0.05), (5, 2, 3, 4, 4, 1.0)):
        ids = draw_ids(g, T, k, E, masked)
        ex, route = routed(tide, E, k, ids)
        slots, held = route.slots.cpu().long(), int(route.offsets[-1])
        at = slots >= 0
        x = torch.randn(T, D + pad, generator=g).to(TYPES[kind])
        dx = Guarded(x, shift)
        rows = Guarded(torch.full((T * k, D + pad), 55.0).to(TYPES[kind]), shift)
        ex.dispatch(dx.view[:, :D], route, rows.view[:, :D])
        want = torch.full((T * k, D + pad), 55.0).to(TYPES[kind])
        want[slots[at], :D] = x[:, :D].repeat_interleave(k, 0).view(T, k, D)[at]
        got = rows.cpu()
        assert torch.equal(got, want)

        # back: rows that no pair has hold NaN, which must not enter
        y = torch.randn(T * k, D + pad, generator=g).to(TYPES[kind])
        y[held:] = float("nan")
        w = torch.randn(T, k, generator=g)
        dy, dw = Guarded(y, shift), Guarded(w)
        for weights in (None, dw):
            out = Guarded(torch.full((T, D + pad), 55.0).to(TYPES[kind]), shift)
            ex.combine(dy.view[:, :D], route, out.view[:, :D], None if weights is None else dw.view)
            f = torch.where(at, w.double() if weights is not None else 1.0, 0.0)
            parts = torch.where(at[:, :, None], y[slots.clamp(min=0), :D].double(), 0.0) * f[:, :, None]
            total, size = parts.sum(1), parts.abs().sum(1)
            got = out.cpu()
            err = (got[:, :D].double() - total).abs()
            assert bool((err <= (k + 1) * U * size * 1.01 + HALF[kind] * total.abs() * 1.01 + 1e-40).all())
            assert bool((got[:, D:] == 55).all())

        # the gradients
        dout = torch.randn(T, D + pad, generator=g).to(TYPES[kind])
        ddout, drows, dweights = Guarded(dout, shift), Guarded(torch.full((T * k, D + pad), 55.0).to(TYPES[kind]), shift), Guarded(torch.full((T, k), 55.0))
        ex.combine_grad(ddout.view[:, :D], dy.view[:, :D], route, dw.view, drows.view[:, :D], dweights.view)
        want = torch.full((T * k, D + pad), 55.0).to(TYPES[kind])
        product = dout[:, None, :D].float() * w[:, :, None]  # fp32, as the call forms it
        want[slots[at], :D] = product.to(TYPES[kind])[at]
        assert torch.equal(drows.cpu(), want)
        parts = torch.where(at[:, :, None], y[slots.clamp(min=0), :D].double(), 0.0) * dout[:, None, :D].double()
        err = (dweights.cpu().double() - parts.sum(2)).abs()
        assert bool((err <= (D + 1) * U * parts.abs().sum(2) * 1.01 + 1e-40).all())
        assert bool((dweights.cpu()[~at] == 0).all())


def test_gradients_by_differences(tide):
    """combine's gradients against differences of its own outputs, whose quotient is exact for a bilinear form but for roundings."""
    T, k, E, D = 6, 3, 4, 40
    g = gen(5)
    ids = draw_ids(g, T, k, E, 0.2)
    ex, route = routed(tide, E, k, ids)
    y, w, dout = torch.randn(T * k, D, generator=g).cuda(), torch.randn(T, k, generator=g).cuda(), torch.randn(T, D, generator=g).cuda()
    drows, dweights, out = torch.zeros(T * k, D, device="cuda"), torch.zeros(T, k, device="cuda"), torch.zeros(T, D, device="cuda")
    ex.combine_grad(dout, y, route, w, drows, dweights)

    def loss(y, w):
        ex.combine(y, route, out, w)
        return float((out.double() * dout.double()).sum())

    # each output is off by (k + 1) u of its products' magnitudes, at most 4 * 4 * 5 in all for |normal| <= 5; the loss sums T * D of them times |dout| <= 5
    slack = 2 * (k + 1) * U * 3 * 25 * 5 * T * D
    for i in range(T):
        for j in range(k):
            a, b = w.clone(), w.clone()
            a[i, j] += 0.5
            b[i, j] -= 0.5
            assert abs(loss(y, a) - loss(y, b) - float(dweights[i, j])) <= slack + (D + 1) * U * 25 * D
    for s in range(0, int(route.offsets[-1]), 3):
        for c in range(0, D, 7):
            a, b = y.clone(), y.clone()
            a[s, c] += 0.5
            b[s, c] -= 0.5
            assert abs(loss(a, w) - loss(b, w) - float(drows[s, c])) <= slack


def test_slots_outside_the_rows_count_as_none(tide):
    ex = tide.Experts(3, 2)
    route = ex.route(4)
    slots = torch.tensor([[0, 8], [-5, 1], [1 << 30, -(1 << 31)], [7, 2]], dtype=torch.int32)
    route.slots.copy_(slots)
    x = torch.arange(4 * 6, dtype=torch.float32).view(4, 6)
    rows = Guarded(torch.full((8, 6), 55.0))
    ex.dispatch(x.cuda(), route, rows.view)
    want = torch.full((8, 6), 55.0)
    want[0], want[1], want[7], want[2] = x[0], x[1], x[3], x[3]
    assert torch.equal(rows.cpu(), want)
    out = torch.full((4, 6), 9.0, device="cuda")
    ex.combine(rows.view, route, out)
    assert torch.equal(out.cpu(), torch.stack([x[0], x[1], torch.zeros(6), 2 * x[3]]))


# ---- 8-bit matrices --------------------------------------------------------------------------------


def strange(x):
    """Blocks of zeros, tiny and huge values, exact ties, NaN and infinity among ordinary ones."""
    n, c = x.shape
    x[0, :128] = 0.0
    if n > 1:
        x[1] *= 2.0 ** -120
    if n > 2:
        x[2] *= 2.0 ** 100
    if n > 3:
        x[3] = torch.where(torch.arange(c) % 2 == 0, 448.0, 17.0)  # 17 lies between 16 and 18
    if n > 4:
        x[4, c // 2] = float("nan")
    if n > 5:
        x[5, c // 3] = float("inf")
    if n > 6:
        x[6] = 2.0 ** -133
    if n > 7:
        x[7] = torch.where(torch.arange(c) % 2 == 0, 449.0, -448.0)
    return x


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 8, 100, 128, 136, 513, 1027, 2048])
def test_rows_in_8_bits(tide, D, kind):
    g = gen(D)
    for T, k, E, shift, pad in ((1, 1, 1, 0, 0), (41, 3, 7, 0, 0), (30, 2, 5, 1, 3), (300, 4, 6, 8, 8)):
        ids = draw_ids(g, T, k, E)
        ex, route = routed(tide, E, k, ids)
        M, held, offsets = T * k, int(route.offsets[-1]), route.offsets.cpu().tolist()
        x = strange(torch.randn(T, D + pad, generator=g)).to(TYPES[kind])
        dx = Guarded(x, shift)
        codes, scales = in_rows(x[:, :D])
        tokens = route.tokens.cpu().long()[:held]

        def check(q):
            assert same(q.codes.float().cpu()[:held].double(), codes[tokens]) and same(q.scales.cpu()[:held].double(), scales[tokens])

        q = tide.Fp8Rows(M, D)
        ex.dispatch_fp8(dx.view[:, :D], route, q)
        check(q)
        # the same by way of rows in the experts' order, and by gathering
        rows = Guarded(torch.full((M, D + pad), float("nan")).to(TYPES[kind]), shift)
        ex.dispatch(dx.view[:, :D], route, rows.view[:, :D])
        blocks = [-(-(b - a) // 128) for a, b in zip(offsets, offsets[1:])]
        for source, gather in ((rows.view[:, :D], False), (dx.view[:, :D], True)):
            q, qt = tide.Fp8Rows(M, D), tide.Fp8Columns(M, D, E)
            q.codes.view(torch.uint8).fill_(0x55)
            qt.codes.view(torch.uint8).fill_(0x55)
            ex.quantize(source, route, rows=q, columns=qt, gather=gather)
            check(q)
            assert bool((q.codes.view(torch.uint8)[held:] == 0x55).all())
            both = [q, qt]
            got, got_scales = qt.codes.float().cpu().double(), qt.scales.cpu().double()
            for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
                at = sum(blocks[:e])
                part = torch.zeros(D, blocks[e] * 128, dtype=torch.float64)
                part[:, :b - a] = x[tokens[a:b], :D].double().t()
                if b > a:
                    c, s = in_rows(part)
                    assert same(got[:, at * 128:(at + blocks[e]) * 128], c) and same(got_scales[at:at + blocks[e]], s.t())
            assert bool((qt.codes.view(torch.uint8)[:, sum(blocks) * 128:] == 0x55).all())
            # each alone
            q, qt = tide.Fp8Rows(M, D), tide.Fp8Columns(M, D, E)
            ex.quantize(source, route, rows=q, gather=gather)
            ex.quantize(source, route, columns=qt, gather=gather)
            check(q)
            n = sum(blocks)
            assert torch.equal(qt.codes.view(torch.uint8)[:, :n * 128], both[1].codes.view(torch.uint8)[:, :n * 128])
            assert same(qt.scales[:n].cpu(), both[1].scales[:n].cpu())


@pytest.mark.parametrize("R, N, K, before, E", [(1, 1, 1, 0, 1), (2, 128, 128, 0, 3), (3, 331, 525, 5, 4), (8, 768, 256, 8, 2), (4, 130, 1027, 0, 2), (8, 3, 200, 1, 5), (70, 200, 64, 0, 2)])
def test_all_gather_fp8(tide, R, N, K, before, E):
    g = gen(N)
    params = ([(before, 1)] if before else []) + [(N, K)] * E
    G = tide.Group(R, params)
    m = -(-N // R)
    shards = [Guarded(torch.full((G.S,), float("nan")).bfloat16(), 0) for _ in range(R)]
    first = 1 if before else 0
    w = [strange(torch.randn(N, K, generator=g)).bfloat16() if e == 1 else torch.randn(N, K, generator=g).bfloat16() for e in range(E)]
    for e in range(E):
        o = G.param_layout(first + e)[1]
        for d in range(R):
            part = w[e][d * m:(d + 1) * m].reshape(-1)
            shards[d].view[o:o + part.numel()].copy_(part)
    for transposed in (False, True):
        W = tide.Fp8Weights(E, N, K, transposed)
        ps = list(range(first, first + E))[::-1]  # any order
        G.all_gather_fp8(ps, [s.view for s in shards], W)
        for i, p in enumerate(ps):
            codes, scales = in_blocks(w[p - first])
            assert same(W.codes[i].float().cpu().double(), codes) and same(W.scales[i].cpu().double(), scales)
            if transposed:
                assert same(W.codes_transposed[i].float().cpu().double(), codes.t())


def test_parts_of_weights_side_by_side(tide):
    N, K, E = 256, 320, 3
    g = gen(0)
    G = tide.Group(2, [(N, K)] * (2 * E))
    shards = torch.randn(2, G.S, generator=g).bfloat16().cuda()
    both, one, two = tide.Fp8Weights(E, 2 * N, K, True), tide.Fp8Weights(E, N, K, True), tide.Fp8Weights(E, N, K, True)
    for q, i in ((both.part(0, N), 0), (both.part(N, N), 1), (one, 0), (two, 1)):
        G.all_gather_fp8(range(i, 2 * E, 2), list(shards), q)
    assert torch.equal(both.codes.view(torch.uint8), torch.cat([one.codes, two.codes], 1).view(torch.uint8))
    assert torch.equal(both.scales, torch.cat([one.scales, two.scales], 1))
    assert torch.equal(both.codes_transposed.view(torch.uint8), torch.cat([one.codes_transposed, two.codes_transposed], 2).view(torch.uint8))
    for first, rows in ((64, 128), (0, 100), (128, 512), (-128, 128)):
        with pytest.raises(tide.TideError):
            both.part(first, rows)


# ---- products --------------------------------------------------------------------------------------


def random_fp8(g, x, any_scales):
    """Fills codes with finite values of all sizes and scales with powers of two, or numbers that are none."""
    bits = torch.randint(0, 256, tuple(x.codes.shape), generator=g).to(torch.uint8)
    bits[(bits & 0x7F) == 0x7F] = 0x3A
    x.codes.view(torch.uint8).copy_(bits)
    r = torch.randn(tuple(x.scales.shape), generator=g)
    x.scales.copy_(torch.exp(r) if any_scales else torch.exp2(torch.round(2 * r)))


def bound(blocks, size):
    return (128 + blocks + 3) * 2 * U * size


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T, k, E, N, K", [(1, 1, 1, 1, 1), (1, 8, 16, 200, 300), (37, 2, 5, 128, 128), (300, 3, 4, 331, 525), (200, 4, 6, 513, 129), (1000, 2, 3, 260, 1040),
                                           (5000, 4, 9, 768, 384), (3000, 8, 20, 1003, 200), (3000, 8, 4, 512, 2600)])
@pytest.mark.parametrize("any_scales", [False, True])
def test_products(tide, T, k, E, N, K, kind, any_scales):
    g = gen(N + K)
    ids = draw_ids(g, T, k, E, 0.1)
    ex, route = routed(tide, E, k, ids)
    M, held, offsets = T * k, int(route.offsets[-1]), route.offsets.cpu().tolist()
    W = tide.Fp8Weights(E, N, K, transposed=True)
    random_fp8(g, W, any_scales)
    W.codes_transposed.view(torch.uint8).copy_(W.codes.view(torch.uint8).transpose(1, 2))
    w = W.codes.cpu().float().double() * W.scales.cpu().double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    for transposed, n, c in ((False, N, K), (True, K, N)):
        A = tide.Fp8Rows(M, c)
        random_fp8(g, A, any_scales)
        A.codes.view(torch.uint8)[held:] = 0x7F  # NaN in the rows that no pair has
        A.scales[held:] = float("nan")
        a = values(A.codes.cpu().float().double(), A.scales.cpu().double())[:held]
        for shift, pad in ((0, 0), (3, 5)):
            out = Guarded(torch.full((M, n + pad), 55.0).to(TYPES[kind]), shift)
            ex.matmul(A, W, route, out.view[:, :n], transposed=transposed, any_scales=any_scales)
            got = out.cpu()
            assert bool((got[held:] == 55).all()) and bool((got[:, n:] == 55).all())
            for e, (x, y) in enumerate(zip(offsets, offsets[1:])):
                m = w[e] if transposed else w[e].t()
                want, size = a[x:y] @ m, a[x:y].abs() @ m.abs()
                err = (got[x:y, :n].double() - want).abs()
                assert bool((err <= bound(-(-c // 128), size) + HALF[kind] * want.abs() * 1.01).all()), (transposed, e, float((err / (size + 1e-30)).max()))
    assert ex.device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T, k, E, N, K", [(1, 1, 1, 1, 1), (1, 4, 16, 200, 300), (37, 2, 5, 128, 128), (300, 3, 4, 331, 525), (1000, 2, 3, 260, 1040), (3000, 4, 9, 768, 384),
                                           (900, 4, 16, 900, 1100), (6000, 4, 16, 1280, 512)])
@pytest.mark.parametrize("any_scales", [False, True])
def test_weight_gradients(tide, T, k, E, N, K, kind, any_scales):
    g = gen(N + K + 1)
    ids = draw_ids(g, T, k, E, 0.1)
    ids[ids == 1] = 0  # an expert without rows
    ex, route = routed(tide, E, k, ids)
    M, offsets = T * k, route.offsets.cpu().tolist()
    dy, a = tide.Fp8Columns(M, N, E), tide.Fp8Columns(M, K, E)
    grads = [Guarded(torch.full((N * K,), 55.0).to(TYPES[kind]), 3 * e) for e in range(E)]
    random_fp8(g, dy, any_scales)
    random_fp8(g, a, any_scales)
    blocks = [-(-(y - x) // 128) for x, y in zip(offsets, offsets[1:])]
    at = 0
    for e, b in enumerate(blocks):  # zeros behind each expert's rows, NaN behind the last
        dy.codes.view(torch.uint8)[:, at * 128 + offsets[e + 1] - offsets[e]:(at + b) * 128] = 0
        at += b
    for x in (dy, a):
        x.codes.view(torch.uint8)[:, at * 128:] = 0x7F
        x.scales[at:] = float("nan")
    ex.weight_grad(dy, a, route, [x.view for x in grads], any_scales=any_scales)
    at = 0
    for e, b in enumerate(blocks):
        p, q = (values(x.codes.cpu().float().double()[:, at * 128:(at + b) * 128], x.scales.cpu().double()[at:at + b].t()) for x in (dy, a))
        want, size = p @ q.t(), p.abs() @ q.abs().t()
        err = (grads[e].cpu().view(N, K).double() - want).abs()
        assert bool((err <= bound(b, size) + HALF[kind] * want.abs() * 1.01).all()), (e, float((err / (size + 1e-30)).max()))
        at += b
    assert ex.device_status() == 0
    # one tensor of all gradients gets the same bits
    whole = torch.full((E, N, K), 55.0, device="cuda").to(TYPES[kind])
    ex.weight_grad(dy, a, route, whole, any_scales=any_scales)
    assert all(torch.equal(whole[e].cpu().flatten(), grads[e].cpu()) for e in range(E))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T, N", [(3, 1), (150, 331), (150, 515), (20000, 1003), (20000, 769)])
def test_products_leave_what_lies_beside_their_rows(tide, T, N, kind):
    """Results whose rows are aligned and not a multiple of 16 bytes long, in both tile shapes; an expert's last rows end inside a tile."""
    E, k, K = 3, 2, 96
    g = gen(N)
    ex, route = routed(tide, E, k, draw_ids(g, T, k, E, 0.1))
    held, offsets = int(route.offsets[-1]), route.offsets.cpu().tolist()
    A, W = tide.Fp8Rows(T * k, K), tide.Fp8Weights(E, N, K)
    random_fp8(g, A, False)
    random_fp8(g, W, False)
    out = torch.full((T * k, -(-N // 8) * 8 + 8), 55.0, device="cuda").to(TYPES[kind])
    ex.matmul(A, W, route, out[:, :N])
    got = out.cpu()
    assert bool((got[held:] == 55).all()) and bool((got[:, N:] == 55).all())
    a, w = values(A.codes.cpu().float().double(), A.scales.cpu().double()), W.codes.cpu().float().double() * W.scales.cpu().double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    for e, (x, y) in enumerate(zip(offsets, offsets[1:])):
        want, size = a[x:y] @ w[e].t(), a[x:y].abs() @ w[e].abs().t()
        assert bool(((got[x:y, :N].double() - want).abs() <= bound(1, size) + HALF[kind] * want.abs() * 1.01).all()), e


@pytest.mark.parametrize("any_scales", [False, True])
@pytest.mark.parametrize("T", [100, 20000])
def test_products_of_rows_with_nan_behind_their_ends(tide, T, any_scales):
    """The bytes between a row's end and the next multiple of 16 are not a part of it."""
    E, N, K = 2, 259, 397
    g = gen(T)
    ex, route = routed(tide, E, 1, draw_ids(g, T, 1, E, 0.0))
    A, W = tide.Fp8Rows(T, K), tide.Fp8Weights(E, N, K)
    for x in (A, W):
        whole = x.codes.view(torch.uint8).as_strided((x.codes[..., 0].numel(), x.codes.stride(-2)), (x.codes.stride(-2), 1))
        whole.fill_(0x7F)
        random_fp8(g, x, any_scales)
        assert K < whole.shape[1] and bool((whole[:, K:] == 0x7F).all())
    out = torch.empty(T, N, device="cuda")
    ex.matmul(A, W, route, out, any_scales=any_scales)
    offsets = route.offsets.cpu().tolist()
    a, w = values(A.codes.cpu().float().double(), A.scales.cpu().double()), W.codes.cpu().float().double() * W.scales.cpu().double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    for e, (x, y) in enumerate(zip(offsets, offsets[1:])):
        want, size = a[x:y] @ w[e].t(), a[x:y].abs() @ w[e].abs().t()
        assert bool(((out[x:y].cpu().double() - want).abs() <= bound(4, size) + HALF["f32"] * want.abs()).all()), e


def test_a_product_of_all_rows_without_a_route(tide):
    """One expert: a plain linear layer's product and gradients."""
    g = gen(3)
    M, N, K = 400, 192, 320
    x, dy, w = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(M, N, generator=g).bfloat16().cuda(), torch.randn(N, K, generator=g).bfloat16().cuda()
    ex, G = tide.Experts(1, 1), tide.Group(1, [(N, K)])
    W, X, D, XT, DT = tide.Fp8Weights(1, N, K, True), tide.Fp8Rows(M, K), tide.Fp8Rows(M, N), tide.Fp8Columns(M, K, 1), tide.Fp8Columns(M, N, 1)
    G.all_gather_fp8([0], [w.view(-1)], W)
    ex.quantize(x, None, rows=X, columns=XT)
    ex.quantize(dy, None, rows=D, columns=DT)
    y, dx, dw = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda")
    ex.matmul(X, W, None, y)
    ex.matmul(D, W, None, dx, transposed=True)
    ex.weight_grad(DT, XT, None, [dw])
    w8 = in_blocks(w.cpu())
    w8 = w8[0] * w8[1].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    x8, d8 = values(*in_rows(x.cpu())), values(*in_rows(dy.cpu()))
    xt8, dt8 = values(*in_rows(x.cpu().t())), values(*in_rows(dy.cpu().t()))
    for got, p, q in ((y, x8, w8.t()), (dx, d8, w8), (dw, dt8, xt8.t())):
        assert bool(((got.cpu().double() - p @ q).abs() <= bound(4, p.abs() @ q.abs()) + U * (p @ q).abs()).all())


def test_scales_that_are_no_powers_of_two_are_told_of(tide):
    for bad in (1.5, 0.0, -2.0):
        ex, W, A, out = tide.Experts(1, 1), tide.Fp8Weights(1, 130, 200), tide.Fp8Rows(9, 200), torch.empty(9, 130, device="cuda")
        random_fp8(gen(0), W, False)
        random_fp8(gen(1), A, False)
        ex.matmul(A, W, None, out)
        assert ex.device_status() == 0
        A.scales[8, 1] = bad
        ex.matmul(A, W, None, out)
        assert ex.device_status() == 2
        A.scales[8, 1] = 1.0
        W.scales[0, 1, 0] = bad
        ex.matmul(A, W, None, out)
        assert ex.device_status() == 2 and ex.device_status() == 0


def test_a_nan_scale_makes_its_rows_nan_alone(tide):
    ex, W, A, out = tide.Experts(1, 1), tide.Fp8Weights(1, 300, 400), tide.Fp8Rows(200, 400), torch.empty(200, 300, device="cuda")
    for any_scales in (False, True):
        random_fp8(gen(0), W, False)
        random_fp8(gen(1), A, False)
        A.scales[70, 2] = float("nan")
        W.scales[0, 1, 3] = float("nan")
        ex.matmul(A, W, None, out, any_scales=any_scales)
        want = torch.zeros(200, 300, dtype=torch.bool)
        want[70] = True
        want[:, 128:256] = True
        assert torch.equal(torch.isnan(out).cpu(), want) and ex.device_status() == 0


# ---- a run of them together -------------------------------------------------------------------------


class Layer:
    """y = sum over choices of weights * (W_e x): every call of a training step, and its plain form in 64 bits, with the same roundings to 8
    bits and to bf16 where rows are handed over."""

    def __init__(self, tide, T, k, E, N, K, R, seed, flags=0):
        g = gen(seed)
        self.T, self.k, self.E, self.N, self.K = T, k, E, N, K
        self.ids = draw_ids(g, T, k, E, 0.1)
        self.x, self.weights, self.dout = torch.randn(T, K, generator=g).bfloat16(), torch.rand(T, k, generator=g), torch.randn(T, N, generator=g).bfloat16()
        self.w = (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16()
        self.group = tide.Group(R, [(N, K)] * E, flags)
        m = -(-N // R)
        full = torch.zeros(E, R * m, K, dtype=torch.bfloat16)
        full[:, :N] = self.w
        self.shards = [full[:, d * m:(d + 1) * m].reshape(-1).cuda() for d in range(R)]
        self.ex = tide.Experts(E, k, flags)
        self.route = self.ex.route(T)
        M, dev = T * k, "cuda"
        self.dev = [x.cuda() for x in (self.ids, self.x, self.weights, self.dout)]
        self.W = tide.Fp8Weights(E, N, K, transposed=True)
        self.x8, self.xt8, self.dy8, self.dyt8 = tide.Fp8Rows(M, K), tide.Fp8Columns(M, K, E), tide.Fp8Rows(M, N), tide.Fp8Columns(M, N, E)
        self.y, self.dy, self.dxr = (torch.zeros(M, n, dtype=torch.bfloat16, device=dev) for n in (N, N, K))
        self.out, self.dx = torch.zeros(T, N, dtype=torch.bfloat16, device=dev), torch.zeros(T, K, dtype=torch.bfloat16, device=dev)
        self.dweights = torch.zeros(T, k, device=dev)
        self.grads = [torch.zeros(N * K, dtype=torch.bfloat16, device=dev) for _ in range(E)]

    def results(self):
        return [self.out, self.dx, self.dweights, self.y, self.dy, *self.grads]

    def step(self, stream=None):
        ex, r = self.ex, self.route
        ids, x, weights, dout = self.dev
        self.group.all_gather_fp8(range(self.E), self.shards, self.W, stream=stream)
        ex.sort(ids, r, stream=stream)
        ex.dispatch_fp8(x, r, self.x8, stream=stream)
        ex.matmul(self.x8, self.W, r, self.y, stream=stream)
        ex.combine(self.y, r, self.out, weights, stream=stream)
        ex.combine_grad(dout, self.y, r, weights, self.dy, self.dweights, stream=stream)
        ex.quantize(self.dy, r, rows=self.dy8, columns=self.dyt8, stream=stream)
        ex.matmul(self.dy8, self.W, r, self.dxr, transposed=True, stream=stream)
        ex.combine(self.dxr, r, self.dx, stream=stream)
        ex.quantize(x, r, columns=self.xt8, gather=True, stream=stream)
        ex.weight_grad(self.dyt8, self.xt8, r, self.grads, stream=stream)

    def check(self):
        """Each result against the plain form of the call that made it, from that call's own inputs."""
        T, k, E, N, K = self.T, self.k, self.E, self.N, self.K
        offsets, slots, tokens = order_of(self.ids, E)
        at, s = slots >= 0, slots.clamp(min=0)
        half = HALF["bf16"] * 1.01
        x8, y, dy, dxr = values(*in_rows(self.x)), self.y.cpu(), self.dy.cpu(), self.dxr.cpu()
        dy8 = values(*in_rows(dy))
        for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
            c, sc = in_blocks(self.w[e])
            w = c * sc.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
            rows = x8[tokens[a:b]]
            for got, p, q in ((y[a:b], rows, w.t()), (dxr[a:b], dy8[a:b], w),
                              (self.grads[e].cpu().view(N, K), values(*in_rows(dy[a:b].t())) if b > a else torch.zeros(N, 0).double(),
                               values(*in_rows(self.x[tokens[a:b]].t())).t() if b > a else torch.zeros(0, K).double())):
                want, size = p @ q, p.abs() @ q.abs()
                assert bool(((got.double() - want).abs() <= bound(-(-p.shape[1] // 128), size) + half * want.abs()).all())
        parts = torch.where(at[:, :, None], y[s].double(), 0.0)
        weighted = parts * self.weights.double()[:, :, None]
        for got, p in ((self.out, weighted), (self.dx, torch.where(at[:, :, None], dxr[s].double(), 0.0))):
            assert bool(((got.cpu().double() - p.sum(1)).abs() <= (k + 1) * U * p.abs().sum(1) + half * p.sum(1).abs()).all())
        want = torch.where(at[:, :, None], self.dout[:, None].float() * self.weights[:, :, None], 0.0).bfloat16()
        assert torch.equal(dy[slots[at]], want[at])
        p = parts * self.dout.double()[:, None]
        assert bool(((self.dweights.cpu().double() - p.sum(2)).abs() <= (N + 1) * U * p.abs().sum(2)).all())
        assert self.ex.device_status() == 0


@pytest.mark.parametrize("T, k, E, N, K, R, flags", [(1, 2, 4, 64, 96, 2, 0), (300, 3, 7, 331, 200, 3, 0), (2500, 8, 16, 640, 512, 8, 0), (700, 2, 5, 256, 384, 4, 8)])
def test_a_layer_and_its_gradients(tide, T, k, E, N, K, R, flags):
    layer = Layer(tide, T, k, E, N, K, R, T, flags)
    layer.step()
    layer.check()


@pytest.mark.parametrize("T, k", [(40, 32), (9000, 2)])
def test_a_layer_of_the_most_experts(tide, T, k):
    layer = Layer(tide, T, k, 1024, 72, 136, 2, k)
    layer.step()
    layer.check()


def test_the_longest_wait_limit(tide):
    layer = Layer(tide, 300, 3, 7, 200, 264, 2, 11)
    layer.ex.set_wait_timeout(2 ** 64 - 1)
    for _ in range(20):
        layer.step()
    layer.check()


def test_a_layer_on_another_stream(tide):
    """Work on a stream of its own, behind a long kernel there, with nothing of it on the current stream; by object and by handle."""
    for handle in (False, True):
        layer = Layer(tide, 300, 3, 7, 200, 264, 2, 3)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        layer.step(side.cuda_stream if handle else side)
        side.synchronize()
        layer.check()


def test_two_layers_at_once(tide):
    """One object of experts on two streams, each with its own buffers."""
    a, b = Layer(tide, 2000, 4, 8, 384, 512, 2, 1), Layer(tide, 2000, 4, 8, 384, 512, 2, 2)
    b.ex, b.route = a.ex, a.ex.route(2000)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        a.step(streams[0])
        b.step(streams[1])
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_a_layer_captured_and_replayed(tide):
    """Two graphs of two layers, replayed with other tokens than they were captured with."""
    layers = [Layer(tide, 9000, 4, 9, 200, 264, 3, 5), Layer(tide, 40, 2, 4, 136, 72, 2, 6)]
    graphs = []
    for layer in layers:
        layer.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.step()
        graphs.append(g)
    for seed in (7, 8):
        for layer in layers:
            g = gen(seed)
            layer.ids = draw_ids(g, layer.T, layer.k, layer.E, 0.3)
            layer.x, layer.dout = torch.randn(layer.T, layer.K, generator=g).bfloat16(), torch.randn(layer.T, layer.N, generator=g).bfloat16()
            for to, x in zip(layer.dev, (layer.ids, layer.x, layer.weights, layer.dout)):
                to.copy_(x)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for layer in layers:
            layer.check()


def test_equal_calls_give_equal_bits(tide):
    layer = Layer(tide, 3000, 4, 12, 520, 384, 4, 9)
    layer.step()
    first = [x.clone() for x in layer.results()]
    for x in layer.results():
        x.fill_(7)
    held = int(layer.route.offsets[-1])
    layer.step()
    for x, y in zip(layer.results(), first):
        if x is layer.y or x is layer.dy:
            x, y = x[:held], y[:held]
        assert torch.equal(x, y)


# ---- far offsets, expired waits, refusals -------------------------------------------------------------


def test_offsets_past_32_bits(tide):
    """Rows whose bytes lie past 2^32 in every buffer: a sample of rows against the plain form."""
    T, k, E, D, N = 300_000, 8, 4, 2048, 1040
    M = T * k
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    x = torch.randn(T, D, generator=g, device="cuda", dtype=torch.float32).bfloat16()
    ex = tide.Experts(E, k)
    route = ex.route(T)
    ex.sort(ids, route)
    rows, q = torch.empty(M, D, dtype=torch.bfloat16, device="cuda"), tide.Fp8Rows(M, D)
    ex.dispatch(x, route, rows)
    ex.dispatch_fp8(x, route, q)
    W = tide.Fp8Weights(E, N, D)
    random_fp8(gen(1), W, False)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ex.matmul(q, W, route, out)
    assert rows.numel() * 2 > 1 << 32 and q.codes.numel() > 1 << 32 and out.numel() * 2 > 1 << 32
    some = torch.cat([torch.arange(0, 64), torch.randint(0, M, (256,), generator=gen(2)), torch.arange(M - 64, M)]).cuda()
    tokens, offsets = route.tokens[some].long(), route.offsets.cpu()
    assert torch.equal(rows[some], x[tokens])
    codes, scales = in_rows(x[tokens].cpu())
    assert same(q.codes.view(torch.uint8)[some].view(torch.float8_e4m3fn).float().cpu().double(), codes) and same(q.scales[some].cpu().double(), scales)
    w = W.codes.cpu().float().double() * W.scales.cpu().double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :D]
    a, e = values(codes, scales), torch.bucketize(some.cpu(), offsets[1:], right=True)
    want, size = torch.einsum("sc,snc->sn", a, w[e]), torch.einsum("sc,snc->sn", a.abs(), w[e].abs())
    assert bool(((out[some].cpu().double() - want).abs() <= bound(D // 128, size) + HALF["bf16"] * 1.01 * want.abs()).all())
    # and back, out of the far rows
    back = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    ex.combine(rows, route, back)
    total = x.double() * k
    assert bool(((back.double() - total).abs() <= (k + 1) * U * total.abs() + HALF["bf16"] * 1.01 * total.abs()).all())
    # transposed: the last columns lie past 2^32 too
    del rows, out, back
    c = tide.Fp8Columns(M, D, E)
    ex.quantize(x, route, columns=c, gather=True)
    assert c.codes.numel() > 1 << 32
    last = int(offsets[-2]) + (M - int(offsets[-2]) - 1) // 128 * 128  # the last block's first row
    n, at = M - last, sum(-(-(b - a) // 128) for a, b in zip(offsets.tolist(), offsets.tolist()[1:])) - 1
    part = torch.zeros(D, 128, dtype=torch.float64)
    part[:, :n] = x[route.tokens[last:].long()].cpu().double().t()
    codes, scales = in_rows(part)
    assert same(c.codes[:, at * 128:(at + 1) * 128].float().cpu().double(), codes) and same(c.scales[at].cpu().double(), scales[:, 0])


@pytest.mark.parametrize("any_scales", [False, True])
def test_offsets_that_nobody_sorted(tide, any_scales):
    """Descending offsets are no rows: nothing is written, and gradients are zeros. Offsets outside the rows count as their bounds."""
    E, M, N, K = 3, 600, 384, 256
    ex = tide.Experts(E, 1)
    route = ex.route(M)
    g = gen(1)
    A, W, D, X = tide.Fp8Rows(M, K), tide.Fp8Weights(E, N, K), tide.Fp8Columns(M, N, E), tide.Fp8Columns(M, K, E)
    for x in (A, W, D, X):
        random_fp8(g, x, any_scales)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    big = 2 ** 31 - 1
    for offsets in ([0, 300, 200, 600], [0, big, 0, big], [5, 4, 4, 4]):
        route.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        out, grads = torch.full((M, N), 55.0, device="cuda"), torch.full((E, N, K), 55.0, device="cuda")
        q, c = tide.Fp8Rows(M, K), tide.Fp8Columns(M, K, E)
        for b in (q.codes.view(torch.uint8), c.codes.view(torch.uint8), q.scales, c.scales):
            b.fill_(55)
        ex.matmul(A, W, route, out, any_scales=any_scales)
        ex.weight_grad(D, X, route, grads, any_scales=any_scales)
        ex.quantize(x, route, rows=q, columns=c)
        assert bool((out == 55).all()) and not bool(grads.any())
        assert all(bool((b == 55).all()) for b in (q.codes.view(torch.uint8), c.codes.view(torch.uint8), q.scales, c.scales))
    results = []
    for offsets in ([-big, 0, 200, big], [0, 0, 200, 600]):
        route.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        out, grads, q = torch.full((M, N), 55.0, device="cuda"), torch.full((E, N, K), 55.0, device="cuda"), tide.Fp8Rows(M, K)
        ex.matmul(A, W, route, out, any_scales=any_scales)
        ex.weight_grad(D, X, route, grads, any_scales=any_scales)
        ex.quantize(x, route, rows=q)
        results.append((out, grads, q.codes.view(torch.uint8).clone(), q.scales.clone()))
    assert all(torch.equal(p, q) for p, q in zip(*results)) and ex.device_status() == 0


@pytest.mark.parametrize("T", [40, 20000])
def test_a_wait_that_runs_out_is_told_of(tide, T):
    """Products that load nothing: every wait gives up after a millisecond, the kernel returns, and the next call works. Both tile shapes, and
    sums in registers."""
    E, N, K = 4, 512, 768
    ex = tide.Experts(E, 2)
    route = ex.route(T)
    ex.sort(torch.randint(0, E, (T, 2), generator=gen(0)).cuda(), route)
    A, W, C, D = tide.Fp8Rows(2 * T, K), tide.Fp8Weights(E, N, K), tide.Fp8Columns(2 * T, K, E), tide.Fp8Columns(2 * T, N, E)
    for i, x in enumerate((A, W, C, D)):
        random_fp8(gen(i), x, False)
    out, grads = torch.zeros(2 * T, N, device="cuda"), torch.zeros(E, N, K, device="cuda")
    calls = [lambda any_scales: ex.matmul(A, W, route, out, any_scales=any_scales), lambda any_scales: ex.weight_grad(D, C, route, grads, any_scales=any_scales)]
    for any_scales in (False, True):
        for f in calls:
            f(any_scales)
            torch.cuda.synchronize()
            first = out.clone(), grads.clone()
            assert ex.device_status() == 0
            ex.set_wait_timeout(1_000_000)
            ex.set_debug(tide.TIDE_DEBUG_STALL_PRODUCER)
            f(any_scales)
            torch.cuda.synchronize()
            assert ex.device_status() == 1
            ex.set_debug(0)
            ex.set_wait_timeout(0)
            f(any_scales)
            assert torch.equal(out, first[0]) and torch.equal(grads, first[1]) and ex.device_status() == 0


def test_refusals(tide):
    """Arguments that the C calls refuse before anything is enqueued."""
    L, EI, ER = tide.lib(), tide.TIDE_EINVAL, tide.TIDE_ERANGE
    ex, G = tide.Experts(5, 2), tide.Group(2, [(24, 40), (24, 40), (24, 41), (7, 1)])
    h, B, F = ex.handle, tide.TIDE_BF16, tide.TIDE_F32
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = buf.data_ptr()
    v = ctypes.c_int64()
    far = (1 << 31) - (1 << 18) + 2

    def fp8(codes=p, stride=48, batch=24 * 48, scales=p, scale_stride=4, scale_batch=4):
        return tide._Fp8(codes, stride, batch, scales, scale_stride, scale_batch)

    assert L.tide_experts_sort_workspace(h, -1, ctypes.byref(v)) == EI and L.tide_experts_sort_workspace(h, far, ctypes.byref(v)) == ER and L.tide_experts_sort_workspace(h, 1, None) == EI
    for status, args in ((EI, (None, tide.TIDE_I64, 3, p, p, p, None, 0)), (EI, (p, F, 3, p, p, p, None, 0)), (EI, (p + 4, tide.TIDE_I64, 3, p, p, p, None, 0)),
                         (EI, (p, tide.TIDE_I64, -1, p, p, p, None, 0)), (EI, (p, tide.TIDE_I64, 3, None, p, p, None, 0)), (EI, (p, tide.TIDE_I64, 3, p, None, p, None, 0)),
                         (EI, (p, tide.TIDE_I64, 3, p, p, p + 2, None, 0)), (EI, (p, tide.TIDE_I64, 3, p, p, p, p + 16, 4096)), (ER, (p, tide.TIDE_I64, far, p, p, p, None, 0)),
                         (EI, (p, tide.TIDE_I64, 40000, p, p, p, None, 0)), (EI, (p, tide.TIDE_I64, 40000, p, p, p, p, 256))):
        assert L.tide_experts_sort(h, *args, None) == status, args
    for status, args in ((EI, (None, B, 8, 3, 8, p, p, 8)), (EI, (p + 1, B, 8, 3, 8, p, p, 8)), (EI, (p + 2, F, 8, 3, 8, p, p, 8)), (EI, (p, 2, 8, 3, 8, p, p, 8)),
                         (EI, (p, B, 7, 3, 8, p, p, 8)), (EI, (p, B, 8, -1, 8, p, p, 8)), (EI, (p, B, 8, 3, 0, p, p, 8)), (EI, (p, B, 8, 3, 8, None, p, 8)),
                         (EI, (p, B, 8, 3, 8, p, None, 8)), (EI, (p, B, 8, 3, 8, p, p, 7)), (ER, (p, B, 8, far, 8, p, p, 8)), (ER, (p, B, 1 << 31, 3, (1 << 30) + 1, p, p, 1 << 31)),
                         (ER, (p, B, 1 << 62, 3, 8, p, p, 8))):
        assert L.tide_experts_dispatch(h, *args, None) == status, args
        src, kind, stride, T, n, slots, rows, rows_stride = args
        assert L.tide_experts_combine(h, rows, kind, rows_stride, T, n, slots, None, src, stride, None) == status, args
        assert L.tide_experts_combine_grad(h, src, kind, stride, rows, rows_stride, T, n, slots, p, p, 1 << 40, p, None) == status, args
    assert L.tide_experts_combine(h, p, B, 8, 3, 8, p, p + 2, p, 8, None) == EI
    assert L.tide_experts_combine_grad(h, p, B, 8, p, 8, 3, 8, p, None, p, 8, p, None) == EI and L.tide_experts_combine_grad(h, p, B, 8, p, 8, 3, 8, p, p, p, 8, None, None) == EI
    bad = (fp8(codes=None), fp8(codes=p + 8), fp8(stride=47), fp8(stride=32), fp8(scales=None), fp8(scales=p + 2), fp8(scale_stride=0))
    for m in bad:
        assert L.tide_experts_dispatch_fp8(h, p, B, 40, 3, 40, p, m, None) == EI
        assert L.tide_experts_quantize(h, p, B, 40, 6, 6, 40, p, None, m, None, None) == EI
        assert L.tide_experts_matmul(h, m, 6, p, fp8(), 0, 24, 40, p, B, 24, None) == EI
        assert L.tide_experts_matmul(h, fp8(), 6, p, m, 0, 24, 40, p, B, 24, None) == EI
        assert L.tide_all_gather_fp8(G.handle, 2, (ctypes.c_int32 * 2)(0, 1), (ctypes.c_void_p * 2)(p, p), m, None, None) == EI
    assert L.tide_experts_dispatch_fp8(h, p, B, 40, 3, 40, p, None, None) == EI
    columns = fp8(stride=640, scale_stride=40)
    grads = (ctypes.c_void_p * 5)(*[p] * 5)
    for m in (fp8(stride=624, scale_stride=40), fp8(stride=640, scale_stride=39), fp8(codes=None, stride=640, scale_stride=40)):
        assert L.tide_experts_quantize(h, p, B, 40, 6, 6, 40, p, None, None, m, None) == EI
        assert L.tide_experts_weight_grad(h, m, columns, 6, p, 0, 40, 40, grads, B, None) == EI
        assert L.tide_experts_weight_grad(h, columns, m, 6, p, 0, 40, 40, grads, B, None) == EI
    for status, args in ((EI, (None, B, 40, 6, 6, 40, p, None)), (EI, (p, 3, 40, 6, 6, 40, p, None)), (EI, (p, B, 39, 6, 6, 40, p, None)), (EI, (p, B, 40, 5, 6, 40, p, None)),
                         (EI, (p, B, 40, 6, -1, 40, p, None)), (EI, (p, B, 40, 6, 6, 0, p, None)), (EI, (p, B, 40, 6, 6, 40, None, None)), (EI, (p, B, 40, 6, 6, 40, p + 2, None)),
                         (EI, (p, B, 40, 6, 6, 40, p, p + 1)), (ER, (p, B, 40, far, far, 40, p, None)), (ER, (p, B, 1 << 31, 6, 6, (1 << 30) + 1, p, None))):
        assert L.tide_experts_quantize(h, *args, fp8(), None, None) == status, args
    for status, args in ((EI, (-1, p, fp8(), 0, 24, 40, p, B, 24)), (EI, (6, None, fp8(), 0, 24, 40, p, B, 24)), (EI, (6, p, fp8(), 4, 24, 40, p, B, 24)), (EI, (6, p, fp8(), 0, 0, 40, p, B, 24)),
                         (EI, (6, p, fp8(), 0, 24, 0, p, B, 24)), (EI, (6, p, fp8(), 0, 24, 40, None, B, 24)), (EI, (6, p, fp8(), 0, 24, 40, p + 1, B, 24)), (EI, (6, p, fp8(), 0, 24, 40, p, 2, 24)),
                         (EI, (6, p, fp8(), 0, 24, 40, p, B, 23)), (EI, (6, p, fp8(batch=24), 0, 24, 40, p, B, 24)), (EI, (6, p, fp8(scale_batch=-1), 0, 24, 40, p, B, 24)),
                         (ER, (far, p, fp8(), 0, 24, 40, p, B, 24)), (ER, (6, p, fp8(), 0, (1 << 30) + 1, 40, p, B, 1 << 31))):
        assert L.tide_experts_matmul(h, fp8(), *args, None) == status, args
    assert L.tide_experts_matmul(h, None, 6, p, fp8(), 0, 24, 40, p, B, 24, None) == EI and L.tide_experts_matmul(h, fp8(), 6, p, None, 0, 24, 40, p, B, 24, None) == EI
    for status, args in ((EI, (-1, p, 0, 40, 40, grads, B)), (EI, (6, None, 0, 40, 40, grads, B)), (EI, (6, p, tide.TIDE_FP8_TRANSPOSED, 40, 40, grads, B)), (EI, (6, p, 0, 0, 40, grads, B)),
                         (EI, (6, p, 0, 40, 40, None, B)), (EI, (6, p, 0, 40, 40, grads, tide.TIDE_I32)), (EI, (6, p, 0, 40, 40, (ctypes.c_void_p * 5)(p, p, p, None, p), B)),
                         (EI, (6, p, 0, 40, 40, (ctypes.c_void_p * 5)(p, p, p, p + 2, p), F)), (ER, (far, p, 0, 40, 40, grads, B))):
        assert L.tide_experts_weight_grad(h, columns, columns, *args, None) == status, args
    shards = (ctypes.c_void_p * 2)(p, p)
    for ps, sh, w, wt in (((0, 2), shards, fp8(), None), ((0, 4), shards, fp8(), None), ((-1, 0), shards, fp8(), None), ((0, 1), (ctypes.c_void_p * 2)(p, None), fp8(), None),
                          ((0, 1), (ctypes.c_void_p * 2)(p, p + 1), fp8(), None), ((0, 1), None, fp8(), None), ((0, 1), shards, None, None), ((0, 1), shards, fp8(), fp8(stride=16)),
                          ((0, 1), shards, fp8(), fp8(codes=None)), ((0, 1), shards, fp8(batch=8), None)):
        assert L.tide_all_gather_fp8(G.handle, 2, (ctypes.c_int32 * 2)(*ps), sh, w, wt, None) == EI
    assert L.tide_all_gather_fp8(G.handle, 0, (ctypes.c_int32 * 2)(0, 1), shards, fp8(), None, None) == EI
    assert L.tide_experts_set_debug(h, 2) == EI
    torch.cuda.synchronize()
    assert not bool(buf.any()) and ex.device_status() == 0


# ---- the example --------------------------------------------------------------------------------------


def test_example_with_experts(tide):
    """A step of the example's layer of experts runs, and its gradients are those of the plain formula, of which 8 bits hold each factor to
    2^-4 of its value or, below a block's smallest normal number, 2^-10 of 2^-8 of the block's largest: products of two are off by (2^-4 + 2^-4 +
    2^-8) of their magnitude, and by 2^-17 of the largest of one factor times the other's, and sums by the sum of these."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sharded_step.py")
    spec = importlib.util.spec_from_file_location("sharded_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    dim, E = 64, 5
    model = module.ShardedModel(2, 211, dim, 96, experts=E, choices=2)
    losses = [float(model.step(module.batches(2, 211, 96, i))) for i in range(3)]
    assert all(x == x and 0 < x < 20 for x in losses) and model.layer.device_status() == 0
    model.gather()
    g = gen(4)
    x = torch.randn(96, dim, generator=g).bfloat16().cuda().requires_grad_(True)
    G = model.params[1].detach().requires_grad_(True)
    h, backward = model.expert_layer(x, G)
    dh = torch.randn(96, dim, generator=g).bfloat16().cuda()
    x.grad = torch.zeros_like(x)
    grads = backward(dh)
    # the formula in 64 bits, with the layer's own choices and signs
    offsets, tokens, slots = model.route.offsets.cpu().tolist(), model.route.tokens.cpu().long(), model.route.slots.cpu().long()
    W = [torch.cat([model.shards[d][model.group.param_layout(2 + e)[1]:][:32 * dim].view(32, dim) for d in range(2)]).cpu().double() for e in range(E)]
    xs, score = x.detach().cpu().double(), (x.detach().cpu().float() @ G.detach().cpu().float().t()).double()
    eps, floor = 2.0 ** -3 + 2.0 ** -8, 2.0 ** -17
    choice = torch.full((96, 2), -1)
    for e in range(E):
        for s in range(offsets[e], offsets[e + 1]):
            choice[tokens[s]][slots[tokens[s]] == s] = e
    p = torch.softmax(score.gather(1, choice), 1)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        t = tokens[a:b]
        pe = p[t][choice[t] == e]
        y = xs[t] @ W[e].t()
        off = eps * (xs[t].abs() @ W[e].abs().t()) + floor * dim * (xs[t].abs().amax(1, keepdim=True) * W[e].abs().max() * 2)
        sure = y.abs() > off * 1.1  # where the sign, and so relu's gradient, is beyond doubt
        dy = dh.cpu().double()[t] * pe[:, None] * (y > 0)
        unsure = dh.cpu().double()[t].abs() * pe[:, None] * ~sure
        want, size = dy.t() @ xs[t], dy.abs().t() @ xs[t].abs()
        slack = (eps + 2.0 ** -7) * size + unsure.t() @ xs[t].abs() * (1 + eps) + floor * (b - a) * 2 * dh.abs().max().item() * xs.abs().max() + 1e-6
        assert bool(((grads[e].cpu().double().view(dim, dim) - want).abs() <= slack).all()), e
    assert G.grad is not None and bool(torch.isfinite(G.grad.float()).all()) and bool(torch.isfinite(x.grad.float()).all()) and bool((x.grad != 0).any())
