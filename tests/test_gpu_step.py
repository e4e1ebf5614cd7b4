"""The sharded training step on the GPU, against plain implementations in 64 bits.

Bounds are those of fp32 arithmetic with unit roundoff u = 2^-24: a sum of n terms is off by at most
(n + 1) u times the sum of the terms' magnitudes, a product or quotient by u times its magnitude.
The lookup has one rounding of a product (and one to bf16), so it is compared bit for bit.  Every
buffer has guard bands around it.
"""
import ctypes
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GUARD = 64  # elements before and after every buffer
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import all_gather_tide_gb300 as t

    t.lib()
    return t


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Guarded:
    """A device copy of a CPU tensor with guard bands, `shift` elements off its alignment."""

    def __init__(self, src, shift=0):
        n = src.numel()
        self.buf = torch.full((GUARD + shift + n + GUARD,), 77, dtype=src.dtype, device="cuda")
        self.lo, self.n = GUARD + shift, n
        self.view = self.buf[self.lo:self.lo + n].view(src.shape)
        self.view.copy_(src)

    def cpu(self):
        assert bool((self.buf[:self.lo] == 77).all()) and bool((self.buf[self.lo + self.n:] == 77).all()), "guard band written"
        return self.view.cpu()


class Table:
    """A group with one parameter `before` a table of rows x length, on R ranks, and plain forms of the
    lookup and its gradient on its CPU copy."""

    def __init__(self, tide, R, rows, length, before=0, flags=0):
        self.R, self.rows, self.len = R, rows, length
        params = ([(before, 1)] if before else []) + [(rows, length)]
        self.p = len(params) - 1
        self.G = tide.Group(R, params, flags)
        self.m, self.o = self.G.param_layout(self.p)
        self.S = self.G.S

    def rows_of(self, shards):
        """The table [rows, len] out of R CPU shards."""
        parts = [s[self.o:self.o + self.m * self.len].view(self.m, self.len) for s in shards]
        return torch.cat(parts)[:self.rows]

    def in_shards(self, table):
        """[R][m * len]: the table's pieces with zero padding."""
        full = torch.zeros(self.R * self.m, self.len, dtype=table.dtype)
        full[:self.rows] = table
        return full.view(self.R, self.m * self.len)


def draw_ids(g, n, rows, masked=0.0, kind="i64"):
    u = torch.rand(n, generator=g, dtype=torch.float64)
    ids = (torch.exp(u * math.log(rows + 1)).long() - 1).clamp(0, rows - 1)
    ids[torch.rand(n, generator=g) < masked] = -1
    return ids.to(TYPES[kind])


SHAPES = [  # R, rows, row length, elements of the parameter before
    (1, 7, 8, 0),
    (2, 33, 256, 0),
    (3, 50, 1027, 5),
    (4, 5, 1, 3),
    (8, 100, 520, 64),
    (8, 3, 24, 8),  # ranks without a row
    (5, 1000, 31, 0),
    (4, 64, 258, 4),
    (70, 201, 40, 0),  # more ranks than travel with a launch
    (2, 40, 4096, 0),
    (3, 300, 2052, 12),
]


@pytest.mark.parametrize("n", [0, 1, 2, 77, 1500])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_lookup_is_exact(tide, shape, n):
    t, g = Table(tide, *shape), gen(n + shape[1])
    for kind, out_type, shift, out_shift, pad, scale in (("i64", "bf16", 0, 0, 0, 1.0), ("i32", "f32", 0, 0, 0, 0.3), ("i64", "f32", 1, 3, 1, 1.7),
                                                         ("i32", "bf16", 3, 1, 5, -2.5), ("i64", "bf16", 4, 4, 4, 8.0), ("i32", "f32", 2, 2, 2, 1.1)):
        shards = [torch.randn(t.S, generator=g).bfloat16() for _ in range(t.R)]
        dev = [Guarded(s, shift) for s in shards]
        ids = draw_ids(g, n, t.rows, 0.2, kind)
        out = Guarded(torch.full((n, t.len + pad), 55.0).to(TYPES[out_type]), out_shift)
        t.G.embedding(t.p, [d.view for d in dev], ids.cuda(), out.view[:, :t.len], scale)
        whole = torch.cat([t.rows_of(shards), torch.zeros(1, t.len).bfloat16()])
        want = (whole[ids.long()].double() * float(torch.tensor(scale, dtype=torch.float32))).float().to(TYPES[out_type])
        got = out.cpu()
        assert torch.equal(got[:, :t.len], want), (kind, out_type, shift)
        assert bool((got[:, t.len:] == 55).all())
    assert t.G.device_status() == 0


@pytest.mark.parametrize("length", [127, 128, 129, 256, 511, 512, 513, 1025, 1537])
def test_lookup_of_rows_that_lie_anywhere(tide, length):
    """Row lengths on both sides of the stretches that a warp takes; tables and outputs off their alignment; NaN in every row
    that no position asks for, so that nothing of a row's neighbours may enter."""
    for before, out_type, out_shift, pad in ((1, "bf16", 0, 0), (3, "bf16", 1, 2), (1, "f32", 1, 3), (5, "f32", 0, 0), (2, "bf16", 3, 1)):
        t, g = Table(tide, 2, 60, length, before), gen(length)
        ids = 2 * torch.randint(0, 30, (45,), generator=g)
        ids[::7] = -1
        shards = [torch.randn(t.S, generator=g).bfloat16() for _ in range(2)]
        for s, first in zip(shards, (0, t.m)):
            s[t.o:t.o + t.m * length].view(t.m, length)[(torch.arange(t.m) + first) % 2 == 1] = float("nan")
        dev = [Guarded(s, 1) for s in shards]
        out = Guarded(torch.full((45, length + pad), 55.0).to(TYPES[out_type]), out_shift)
        t.G.embedding(t.p, [d.view for d in dev], ids.cuda(), out.view[:, :length], -1.5)
        whole = torch.cat([t.rows_of(shards), torch.zeros(1, length).bfloat16()])
        want = (whole[ids].double() * -1.5).float().to(TYPES[out_type])
        want[ids < 0] = 0.0
        got = out.cpu()
        assert torch.equal(got[:, :length], want) and not bool(torch.signbit(got[ids < 0]).any())
        assert bool((got[:, length:] == 55).all())


def test_lookup_of_ids_past_the_table_gives_zero_rows_and_a_status(tide):
    t = Table(tide, 2, 10, 16)
    shards = [torch.ones(t.S, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ids = torch.tensor([0, 9, 10, -1, 1 << 40, -(1 << 40)], device="cuda")
    out = torch.full((6, 16), 5.0, device="cuda")
    t.G.embedding(t.p, shards, ids, out)
    assert out.sum(1).tolist() == [16, 16, 0, 0, 0, 0]
    assert t.G.device_status() == 64 and t.G.device_status() == 0


def test_lookup_of_batches_of_ids_and_in_a_graph(tide):
    t, g = Table(tide, 4, 30, 64), gen(3)
    shards = [torch.randn(t.S, generator=g).bfloat16() for _ in range(4)]
    dev = [s.cuda() for s in shards]
    ids = draw_ids(g, 12, 30).view(3, 4).cuda()
    out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        t.G.embedding(t.p, dev, ids, out)
    for seed in range(3):
        ids.copy_(draw_ids(gen(seed), 12, 30).view(3, 4))
        graph.replay()
        assert torch.equal(out.cpu(), t.rows_of(shards)[ids.cpu()])


def test_lookup_of_few_ctas_and_on_a_side_stream(tide):
    """TIDE_FLAG_OVERLAP bounds the CTAs, which then walk the work; ids, shards and out made on the stream used."""
    t, g = Table(tide, 4, 5000, 264, 8, tide.TIDE_FLAG_OVERLAP), gen(4)
    shards = [torch.randn(t.S, generator=g).bfloat16() for _ in range(4)]
    ids = draw_ids(g, 30_000, 5000, 0.1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dev, di = [s.cuda() for s in shards], ids.cuda()
        out = torch.empty(30_000, 264, dtype=torch.bfloat16, device="cuda")
    t.G.embedding(t.p, dev, di, out, stream=side)
    side.synchronize()
    whole = torch.cat([t.rows_of(shards), torch.zeros(1, 264).bfloat16()])
    assert torch.equal(out.cpu(), whole[ids])


def check_grad(t, ids, douts, old, shards, scale, add):
    """R CPU shards against sums in 64 bits; `old`: the shards before the call."""
    i = torch.cat([x.long() for x in ids])
    x = torch.cat([d.double() for d in douts])
    keep = (i >= 0) & (i < t.rows)
    total = torch.zeros(t.rows, t.len, dtype=torch.float64).index_add_(0, i[keep], x[keep])
    size = torch.zeros(t.rows, t.len, dtype=torch.float64).index_add_(0, i[keep], x[keep].abs())
    count = torch.zeros(t.rows, 1, dtype=torch.float64).index_add_(0, i[keep], torch.ones(int(keep.sum()), 1, dtype=torch.float64))
    scale = float(torch.tensor(scale, dtype=torch.float32))
    want, bound = t.in_shards(total * scale), t.in_shards((count + 3) * U * size * abs(scale))
    touched = t.in_shards((count > 0).expand(-1, t.len))
    for d in range(t.R):
        got, was = shards[d], old[d]
        a, b = t.o, t.o + t.m * t.len
        assert torch.equal(got[:a], was[:a]) and torch.equal(got[b:], was[b:]), "another parameter's piece was written"
        g, w = got[a:b].double(), was[a:b].double()
        if add:
            assert torch.equal(got[a:b][~touched[d]], was[a:b][~touched[d]]), "a row without a token was written"
            err, lim = (g - w - want[d]).abs(), bound[d] + 2 * U * (w.abs() + want[d].abs())
        else:
            assert bool((g[~touched[d]] == 0).all()) and not bool(torch.signbit(got[a:b][~touched[d]]).any())
            err, lim = (g - want[d]).abs(), bound[d]
        assert bool((err <= lim).all()), float((err - lim).max())


def run_grad(tide, t, ids, douts, scale, add, shift=0, dout_shift=0, pad=0, seed=0):
    g = gen(seed)
    old = [torch.randn(t.S, generator=g) for _ in range(t.R)]
    dev = [Guarded(s, shift) for s in old]
    dd = []
    for x in douts:
        wide = torch.full((x.shape[0], t.len + pad), 3.0).to(x.dtype)
        wide[:, :t.len] = x
        dd.append(Guarded(wide, dout_shift))
    n = sum(x.numel() for x in ids)
    work = Guarded(torch.zeros(t.G.embedding_grad_workspace(t.p, n).numel(), dtype=torch.uint8), 256 - GUARD)
    di = [x.cuda() for x in ids]
    results = []
    for again in range(2):  # equal calls give equal bits, whatever the workspace holds
        for d, o in zip(dev, old):
            d.view.copy_(o)
        work.view.fill_(255 * again)
        t.G.embedding_grad(t.p, di, [x.view[:, :t.len] for x in dd], [d.view for d in dev], scale, add, workspace=work.view)
        results.append([d.cpu() for d in dev])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    work.cpu()
    check_grad(t, ids, [x.float() for x in douts], old, results[0], scale, add)


@pytest.mark.parametrize("sizes", [(0,), (1,), (3, 0, 5), (40, 1, 100), (700, 900)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient_by_token(tide, shape, sizes):
    t, g = Table(tide, *shape), gen(sum(sizes))
    for kind, dout, shift, dshift, pad, add, scale in (("i64", "bf16", 0, 0, 0, False, 1.0), ("i32", "f32", 0, 0, 0, True, 0.3),
                                                       ("i64", "f32", 1, 3, 1, False, 1.7), ("i32", "bf16", 3, 1, 5, True, -2.5),
                                                       ("i64", "bf16", 4, 8, 8, True, 8.0), ("i32", "f32", 8, 2, 2, False, 1.1)):
        ids = [draw_ids(g, n, t.rows, 0.1, kind) for n in sizes]
        douts = [torch.randn(n, t.len, generator=g).to(TYPES[dout]) for n in sizes]
        run_grad(tide, t, ids, douts, scale, add, shift, dshift, pad)
    assert t.G.device_status() == 0


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("what", ["one token", "two tokens", "none", "descending", "many batches", "past the table"])
def test_gradient_of_unusual_texts(tide, what, add):
    t, g = Table(tide, 4, 3001, 264, 16), gen(5)
    n = 5003
    ids = {"one token": torch.full((n,), 2999), "two tokens": torch.arange(n) % 2 * 3000, "none": torch.full((n,), -1),
           "descending": (n - 1 - torch.arange(n)) % 3001, "many batches": draw_ids(g, n, 3001), "past the table": torch.arange(n)}[what]
    x = torch.randn(n, t.len, generator=g).bfloat16()
    cuts = [0, n] if what != "many batches" else sorted({0, n, *torch.randint(0, n, (150,), generator=g).tolist()})
    run_grad(tide, t, [ids[a:b] for a, b in zip(cuts, cuts[1:])], [x[a:b] for a, b in zip(cuts, cuts[1:])], 1.5, add)
    assert t.G.device_status() == (64 if what == "past the table" else 0)


@pytest.mark.parametrize("rows, n", [(50, 256), (50, 257), (3000, 2048), (3000, 2049), (1, 300), (2, 70000), (1023, 20000), (1024, 20000), (200_000, 50_000), (1_100_000, 9000)])
def test_gradient_over_many_rows_and_positions(tide, rows, n):
    """Row counts on both sides of one, two and three digits of the sort, lists on both sides of the lengths
    at which another sort takes over, and lists beyond one CTA's."""
    t, g = Table(tide, 3, rows, 8), gen(rows)
    ids = [draw_ids(g, n, rows, 0.01, "i32")]
    run_grad(tide, t, ids, [torch.randn(n, 8, generator=g)], 1.0, False)


@pytest.mark.parametrize("n", [200, 900])
@pytest.mark.parametrize("length", [9, 255, 257, 520, 1027])
def test_gradient_of_rows_that_lie_anywhere(tide, length, n):
    """Douts off their alignment by every number of elements in 16 bytes, short lists and sorted ones; rows of positions
    without a token, which lie beside the others, hold NaN."""
    t, g = Table(tide, 2, 300, length, 3), gen(length + n)
    for shift in range(8):
        dout, add = (torch.bfloat16, torch.float32)[shift % 2], shift % 4 < 2
        ids = draw_ids(g, n, 300, 0.3)
        x = torch.randn(n, length, generator=g).to(dout)
        x[ids < 0] = float("nan")
        old = [torch.randn(t.S, generator=g) for _ in range(2)]
        dev, dx = [Guarded(o, shift % 3) for o in old], Guarded(x, shift)
        t.G.embedding_grad(t.p, [ids.cuda()], [dx.view], [d.view for d in dev], 0.7, add)
        check_grad(t, [ids], [torch.nan_to_num(x.float())], old, [d.cpu() for d in dev], 0.7, add)


@pytest.mark.parametrize("rows", [127, 129, 4095, 8193, (1 << 22) - 1, (1 << 22) + 1])
def test_gradient_zeros_the_rows_without_a_token(tide, rows):
    """Tables on both sides of the sizes at which zeros go beside the sort and in larger groups of rows; tokens at the
    ends of groups, one of them repeated."""
    t = Table(tide, 3, rows, 2)
    ids = torch.cat([torch.arange(0, rows, max(1, rows // 300)), torch.tensor([0, 1, rows - 1, rows - 2, rows // 2]).repeat(80), torch.full((300,), 31)])
    for k in range(5, 13):
        ids = torch.cat([ids, torch.tensor([x for x in ((1 << k) - 1, 1 << k, (128 << k) - 1, 128 << k) if x < rows], dtype=torch.long)])
    x = torch.randn(ids.numel(), 2, generator=gen(rows))
    run_grad(tide, t, [ids], [x], 1.0, False)


def whole_numbers(n, length, dtype, seed):
    """Rows of whole numbers from -8 to 8 on the GPU."""
    return torch.randint(-8, 9, (n, length), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def check_exactly(t, ids, x, add, cuts=(), seed=0):
    """The gradient of douts that are whole numbers, whose sums fp32 holds exactly: every element of every shard is what sums
    in 64 bits give, zeros, padding and the other parameters' pieces among them.  cuts: where batches after the first begin."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    old = torch.randint(-8, 9, (t.R, t.S), generator=g, device="cuda").float()
    shards, at = old.clone(), [0, *cuts, ids.numel()]
    t.G.embedding_grad(t.p, [ids[a:b] for a, b in zip(at, at[1:])], [x[a:b] for a, b in zip(at, at[1:])], list(shards), 0.5, add)
    keep = (ids >= 0) & (ids < t.rows)
    total = torch.zeros(t.R * t.m, t.len, dtype=torch.float64, device="cuda").index_add_(0, ids[keep].long(), x[keep].double() * 0.5)
    assert float(total.abs().max()) < 2 ** 22
    want, piece = old.double(), slice(t.o, t.o + t.m * t.len)
    want[:, piece] = total.view(t.R, -1) + (want[:, piece] if add else 0)
    wrong = (shards.double() != want).nonzero()
    assert wrong.numel() == 0, (wrong.shape[0], wrong[0].tolist())


@pytest.mark.parametrize("below", [0, 4000])
def test_gradient_keeps_the_last_row_of_a_group_that_is_zeroed(tide, below):
    """A short list and a sorted one; 33 positions in the group of rows 127,968 to 127,999, of which the last is alone in its row:
    one more than the search for the group's end looks at in one step."""
    t = Table(tide, 8, 128_000, 64)
    ids = torch.cat([torch.arange(below) % 1000, 127_968 + torch.arange(32) // 4, torch.tensor([127_990])]).cuda()
    check_exactly(t, ids, whole_numbers(ids.numel(), 64, torch.float32, below), False)


@pytest.mark.parametrize("seed", range(10))
def test_gradient_of_many_rows_that_are_written_beside_zeros(tide, seed):
    t, n = Table(tide, 8, 128_000, 128), 131_072
    ids = torch.randint(0, t.rows, (n,), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    check_exactly(t, ids, whole_numbers(n, 128, torch.bfloat16, seed), False)


@pytest.mark.parametrize("n", [300, 5000])
def test_gradient_is_written_after_the_kernel_before_has_read_the_shard(tide, n):
    """Zeros are written while the positions are sorted, but not before what was launched earlier has ended."""
    t, g = Table(tide, 1, 100_000, 256), gen(n)
    ids, x = draw_ids(g, n, t.rows).cuda(), torch.randn(n, 256, generator=g).cuda()
    T = tide.TensorList([t.S])
    grad, moment, other = torch.ones(t.S, device="cuda"), torch.zeros(t.S, device="cuda"), torch.zeros(t.S, device="cuda")
    param, work = torch.zeros(t.S, device="cuda"), t.G.embedding_grad_workspace(t.p, n)
    for rep in range(5):
        grad.fill_(1.0)
        moment.zero_()
        torch.cuda.synchronize()
        T.adamw([param], [grad], [moment], [other], lr=0.1, betas=(0.5, 0.5), step=1)
        t.G.embedding_grad(t.p, [ids], [x], [grad], workspace=work)
        assert bool((moment == 0.5).all())
        held = torch.zeros(t.rows, dtype=torch.bool, device="cuda")
        held[ids[ids >= 0]] = True
        assert bool((grad.view(t.rows, 256)[~held] == 0).all())


def test_gradient_does_not_read_rows_of_positions_without_a_token(tide):
    for length in (256, 13):
        t, g = Table(tide, 2, 50, length), gen(7)
        for n in (100, 1000):  # a short list and a sorted one
            ids = draw_ids(g, n, 50, 0.3)
            x = torch.randn(n, length, generator=g)
            x[ids < 0] = float("nan")
            shards = [torch.zeros(t.S, device="cuda") for _ in range(2)]
            t.G.embedding_grad(t.p, [ids.cuda()], [x.cuda()], shards)
            assert all(bool(s.isfinite().all()) for s in shards)
            check_grad(t, [ids], [torch.nan_to_num(x)], [torch.zeros(t.S)] * 2, [s.cpu() for s in shards], 1.0, False)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("n", [200, 20_000])
def test_gradient_of_few_ctas_on_a_side_stream_without_a_workspace(tide, n, add):
    t, g = Table(tide, 4, 3000, 520, 8, tide.TIDE_FLAG_OVERLAP), gen(n)
    ids, x = draw_ids(g, n, 3000, 0.1), torch.randn(n, 520, generator=g).bfloat16()
    old = [torch.randn(t.S, generator=g) for _ in range(4)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dev, di, dx = [o.cuda() for o in old], ids.cuda(), x.cuda()
    t.G.embedding_grad(t.p, [di], [dx], dev, 1.5, add, stream=side)
    side.synchronize()
    check_grad(t, [ids], [x.float()], old, [d.cpu() for d in dev], 1.5, add)


@pytest.mark.parametrize("n", [50, 3000])
def test_gradient_in_a_graph(tide, n):
    t, g = Table(tide, 3, 400, 64), gen(n)
    ids, x = draw_ids(g, n, 400).cuda(), torch.randn(n, 64, generator=g).cuda()
    shards = [torch.empty(t.S, device="cuda") for _ in range(3)]
    work = t.G.embedding_grad_workspace(t.p, n)
    t.G.embedding_grad(t.p, [ids], [x], shards, workspace=work)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        t.G.embedding_grad(t.p, [ids], [x], shards, workspace=work)
    for seed in range(3):
        ids.copy_(draw_ids(gen(seed), n, 400))
        graph.replay()
        check_grad(t, [ids.cpu()], [x.cpu()], [torch.zeros(t.S)] * 3, [s.cpu() for s in shards], 1.0, False)


def test_table_of_more_than_2_to_the_31_elements(tide):
    rows, length = 70_000, 32_768  # 2.3 billion elements on one rank
    G = tide.Group(1, [(rows, length)])
    shard = torch.zeros(G.S, dtype=torch.bfloat16, device="cuda")
    table = shard.view(rows, length)
    ids = torch.tensor([69_999, 65_536, 0, 65_535, 69_999, -1], device="cuda")
    for k, t in enumerate((69_999, 65_536, 0, 65_535)):
        table[t] = k + 1
    out = torch.empty(6, length, device="cuda")
    G.embedding(0, [shard], ids, out, 2.0)
    assert out[:, 0].tolist() == [2, 4, 6, 8, 2, 0] and bool((out == out[:, :1]).all())
    grad = torch.full((G.S,), 7.0, device="cuda")
    for many in (1, 100):  # a short list and a sorted one
        G.embedding_grad(0, [ids.repeat(many)], [out.repeat(many, 1)], [grad])
        rows_sum = grad.view(rows, length)
        assert rows_sum[[69_999, 65_536, 0, 65_535], 5].tolist() == [4 * many, 4 * many, 6 * many, 8 * many]
        assert float(rows_sum.sum(dtype=torch.float64)) == 22.0 * many * length
    del table, rows_sum
    norm = torch.zeros(1, device="cuda")
    T = tide.TensorList([G.S])
    T.clip_grad_norm([grad], 1.0, norm)
    want = 100 * math.sqrt((16 + 16 + 36 + 64) * length)
    assert abs(norm.item() - want) <= 18 * U * want
    assert abs(float(grad.square().sum(dtype=torch.float64)) - 1) < 1e-5


def test_gradient_is_the_lookups_difference(tide):
    """f(W) = <lookup(W), x> is linear in W, so the difference of f over a step of one element is the
    gradient times the step; steps and x are chosen so that f has no rounding."""
    t, g = Table(tide, 3, 20, 24, 4), gen(9)
    ids = draw_ids(g, 50, 20, 0.1)
    x = torch.randint(-8, 9, (50, 24), generator=g).float()
    shards = [torch.randint(-8, 9, (t.S,), generator=g).bfloat16() for _ in range(3)]
    grad = [torch.full((t.S,), 9.0, device="cuda") for _ in range(3)]
    t.G.embedding_grad(t.p, [ids.cuda()], [x.cuda()], grad, scale=0.5)

    def f(parts):
        out = torch.empty(50, 24, device="cuda")
        t.G.embedding(t.p, [s.cuda() for s in parts], ids.cuda(), out, scale=0.5)
        return float((out.cpu().double() * x.double()).sum())

    base = f(shards)
    for row, col in [(0, 0), (1, 23), (6, 5), (7, 0), (13, 7), (19, 23)]:
        d, e = row // t.m, t.o + (row % t.m) * 24 + col
        moved = [s.clone() for s in shards]
        moved[d][e] += 2
        assert (f(moved) - base) / 2 == float(grad[d][e])


def test_gradient_refusals(tide):
    t = Table(tide, 2, 10, 16, 4)
    E = tide.TIDE_EINVAL
    ids, x = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(3, 16, device="cuda")
    shards = [torch.zeros(t.S, device="cuda") for _ in range(2)]
    work = t.G.embedding_grad_workspace(t.p, 3)

    def status(**change):
        a = dict(p=t.p, ids=[ids], douts=[x], shards=shards, workspace=work)
        a.update(change)
        with pytest.raises(tide.TideError) as e:
            t.G.embedding_grad(**a)
        return e.value.status

    assert status(p=2) == E and status(p=-1) == E
    assert status(shards=shards[:1]) == E
    assert status(ids=[]) == E and status(douts=[x, x]) == E
    assert status(ids=[ids.float()]) == E and status(douts=[x.half()]) == E
    assert status(ids=[ids, ids.int()], douts=[x, x]) == E
    assert status(douts=[x[:2]]) == E and status(douts=[x.t()]) == E
    assert status(workspace=work[:-1]) == E
    assert status(workspace=torch.empty(work.numel() + 1, dtype=torch.uint8, device="cuda")[1:]) == E
    assert status(shards=[shards[0].data_ptr() + 2, shards[1]]) == E and status(shards=[s.bfloat16() for s in shards]) == E
    with pytest.raises(tide.TideError) as e:
        tide.tide_embedding_grad_workspace(t.G.handle, t.p, 1 << 31)
    assert e.value.status == tide.TIDE_ERANGE
    L = tide.lib()
    table = tide.pointer_table(shards)
    assert L.tide_embedding(t.G.handle, t.p, table, ids.data_ptr(), tide.TIDE_I64, 3, 1.0, x.data_ptr(), tide.TIDE_F32, 15, None) == E  # rows overlap
    assert L.tide_embedding(t.G.handle, t.p, table, ids.data_ptr(), tide.TIDE_F32, 3, 1.0, x.data_ptr(), tide.TIDE_F32, 16, None) == E
    assert L.tide_embedding(t.G.handle, t.p, table, ids.data_ptr() + 4, tide.TIDE_I64, 2, 1.0, x.data_ptr(), tide.TIDE_F32, 16, None) == E
    assert L.tide_embedding(t.G.handle, t.p, table, None, tide.TIDE_I64, 2, 1.0, x.data_ptr(), tide.TIDE_F32, 16, None) == E
    assert L.tide_embedding(t.G.handle, t.p, table, None, tide.TIDE_I64, -1, 1.0, x.data_ptr(), tide.TIDE_F32, 16, None) == E
    assert L.tide_embedding(t.G.handle, t.p, table, ids.data_ptr(), tide.TIDE_I64, 1 << 61, 1.0, x.data_ptr(), tide.TIDE_F32, 16, None) == tide.TIDE_ERANGE
    torch.cuda.synchronize()


@pytest.mark.parametrize("length", [1, 300, 1024, 4096, 8192])
def test_workspace_sizes_never_fall(tide, length):
    t = Table(tide, 1, 10, length)
    sizes = [tide.tide_embedding_grad_workspace(t.G.handle, t.p, n) for n in (*range(0, 130_000, 5), 10 ** 6, 10 ** 7, 10 ** 9, 2 * 10 ** 9)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("length, most", [(1024, 4241), (4096, 7265)])
def test_a_workspace_serves_fewer_positions(tide, length, most):
    """Lists on both sides of the lengths at which pieces get shorter, of which a shorter list has more partial sums."""
    t = Table(tide, 2, 500, length)
    work = Guarded(torch.zeros(t.G.embedding_grad_workspace(t.p, most).numel(), dtype=torch.uint8), 256 - GUARD)
    for n in (most, most - 1, most - 16, 4233, 3000, 1500, 1057, 1056, 257, 256, 1):
        ids, x = torch.arange(n, device="cuda") * 7 % 400, whole_numbers(n, length, torch.float32, n)
        shards = [torch.full((t.S,), 3.0, device="cuda") for _ in range(2)]
        t.G.embedding_grad(t.p, [ids], [x], shards, workspace=work.view)
        want = torch.zeros(500, length, dtype=torch.float64, device="cuda").index_add_(0, ids, x.double())
        assert torch.equal(torch.stack(shards).double().view(500, length), want)
    work.cpu()


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("sizes", [(0,), (1,), (256,), (0, 100, 3), (4,) * 64], ids=lambda s: f"{len(s)}x{sum(s)}")
def test_short_lists_need_no_workspace(tide, sizes, add, monkeypatch):
    t, g = Table(tide, 3, 90, 520, 8), gen(sum(sizes))
    ids = draw_ids(g, sum(sizes), 90, 0.1).cuda()
    cuts = torch.tensor(sizes).cumsum(0)[:-1].tolist()
    monkeypatch.setattr(t.G, "embedding_grad_workspace", lambda *a: pytest.fail("a workspace was allocated"))
    check_exactly(t, ids, whole_numbers(ids.numel(), 520, torch.bfloat16, 1), add, cuts)


def test_longer_lists_need_a_workspace(tide):
    t = Table(tide, 2, 90, 64)
    shards = [torch.zeros(t.S, device="cuda") for _ in range(2)]
    for sizes in ((257,), (2,) * 65):
        ids, x = [torch.zeros(n, dtype=torch.int64, device="cuda") for n in sizes], [torch.zeros(n, 64, device="cuda") for n in sizes]
        with pytest.raises(tide.TideError) as e:
            tide.tide_embedding_grad(t.G.handle, t.p, ids, x, shards, None)
        assert e.value.status == tide.TIDE_EINVAL
        t.G.embedding_grad(t.p, ids, x, shards)  # allocates one
    torch.cuda.synchronize()


def test_workspaces_that_do_not_fit_are_refused(tide):
    """On the host, with gaps, or too small; one of other elements is as large as its bytes."""
    t, n = Table(tide, 2, 500, 64), 1000
    ids, x = torch.arange(n, device="cuda") % 500, whole_numbers(n, 64, torch.float32, 0)
    need = tide.tide_embedding_grad_workspace(t.G.handle, t.p, n)
    shards = [torch.zeros(t.S, device="cuda") for _ in range(2)]
    for bad in (torch.empty(2 * need, dtype=torch.uint8), torch.empty(need, dtype=torch.uint8).pin_memory(), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2],
                torch.empty(need // 4 - 1, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")):
        with pytest.raises(tide.TideError) as e:
            t.G.embedding_grad(t.p, [ids], [x], shards, workspace=bad)
        assert e.value.status == tide.TIDE_EINVAL
    t.G.embedding_grad(t.p, [ids], [x], shards, workspace=torch.empty(need // 4, device="cuda"))
    want = torch.zeros(500, 64, dtype=torch.float64, device="cuda").index_add_(0, ids, x.double())
    assert torch.equal(torch.stack(shards).double().view(500, 64), want)


def launches_of(call):
    """Grid sizes of the kernels that call(stream) launches, in order: the call is captured into a graph and not run."""
    cu = ctypes.CDLL("libcuda.so.1")

    class Kernel(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
        _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                    ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]

    stream, graph, count, kind, out = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t(), ctypes.c_int(), []
    handle = ctypes.c_void_p(stream.cuda_stream)
    assert cu.cuStreamBeginCapture_v2(handle, 2) == 0  # relaxed
    try:
        call(stream)
    finally:
        ended = cu.cuStreamEndCapture(handle, ctypes.byref(graph))
    assert ended == 0 and cu.cuGraphGetNodes(graph, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(count)) == 0
    for node in nodes:
        p = Kernel()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0 and cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0:
            out.append(p.grid[0])
    assert cu.cuGraphDestroy(graph) == 0
    return out


@pytest.mark.parametrize("n, batches", [(100, 1), (300, 1), (2048, 1), (20_000, 1), (100, 70), (2000, 70), (60_000, 130)])
def test_few_ctas_are_kept_by_every_launch(tide, n, batches):
    """Short lists, counted and sorted ones, and more batches than travel with a launch, under TIDE_FLAG_OVERLAP."""
    t, g = Table(tide, 4, 3000, 64, 0, tide.TIDE_FLAG_OVERLAP), gen(n)
    ids, x = draw_ids(g, n, t.rows, 0.1).cuda(), whole_numbers(n, 64, torch.float32, n)
    shards, work = [torch.zeros(t.S, device="cuda") for _ in range(4)], t.G.embedding_grad_workspace(t.p, n)
    cuts = [n * k // batches for k in range(batches + 1)]
    parts = [ids[a:b] for a, b in zip(cuts, cuts[1:])], [x[a:b] for a, b in zip(cuts, cuts[1:])]
    torch.cuda.synchronize()
    grids = launches_of(lambda s: t.G.embedding_grad(t.p, *parts, shards, workspace=work, stream=s))
    few = torch.cuda.get_device_properties(0).multi_processor_count // 9
    assert len(grids) == (1 if n <= 256 and batches <= 64 else 2 + (-(-batches // 64) if batches > 64 else 0))
    assert max(grids) <= few, grids
    out, table = torch.empty(n, 64, device="cuda"), [torch.zeros(t.S, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    looked_up = launches_of(lambda s: t.G.embedding(t.p, table, ids, out, stream=s))
    assert len(looked_up) == 1 and looked_up[0] <= few
    for add in (False, True):
        check_exactly(t, ids, x, add, cuts[1:-1])


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("n, length, piece", [(600, 8, 8), (20_000, 300, 16), (4000, 8192, 32), (140_000, 8, 32), (710_000, 300, 64), (1_500_000, 8, 64)])
def test_gradient_in_pieces_of_every_length(tide, n, length, piece, add):
    """A frequent row runs over many pieces and, from 140,000 positions on, over many blocks of pieces; from there on a warp of the
    sort also takes its positions in several batches.  Sums of whole numbers, so that a position lost or added twice shows."""
    t, g = Table(tide, 3, 500, length, 5), gen(n)
    ids, x = draw_ids(g, n, t.rows, 0.05).cuda(), whole_numbers(n, length, torch.bfloat16 if n % 3 else torch.float32, n)
    shards, work = [torch.zeros(t.S, device="cuda") for _ in range(3)], t.G.embedding_grad_workspace(t.p, n)
    torch.cuda.synchronize()
    grids = launches_of(lambda s: t.G.embedding_grad(t.p, [ids], [x], shards, accumulate=True, workspace=work, stream=s))
    assert grids[-1] == -(-(-(-n // piece) * -(-length // 256)) // 8)  # eight warps to a CTA
    check_exactly(t, ids, x, add, (n // 3, n // 2))
    check_exactly(t, torch.where(ids < 0, ids, 7), x, add, (n // 3, n // 2))


# ---- lists of tensors ----------------------------------------------------------------------------

LISTS = [(1,), (0, 1, 0), (31, 32, 33), (2047, 2048, 2049, 7), (8, 5, 100_003, 0, 1, 4096), (300_000,), tuple(range(0, 900, 7)), (0,), (0, 0)]


def make_list(tide, elems, kinds, seed, sigma=1.0, shift=0):
    g = gen(seed)
    types = [tide.TIDE_BF16 if kinds == "bf16" or (kinds == "mixed" and k % 2) else tide.TIDE_F32 for k in range(len(elems))]
    host = [(torch.randn(n, generator=g) * sigma).to(torch.bfloat16 if ty == tide.TIDE_BF16 else torch.float32) for n, ty in zip(elems, types)]
    dev = [Guarded(x, shift and (shift + k) % 9) for k, x in enumerate(host)]
    return tide.TensorList(elems, types), host, dev


@pytest.mark.parametrize("kinds, shift", [("f32", 0), ("bf16", 0), ("mixed", 1)])
@pytest.mark.parametrize("elems", LISTS, ids=lambda e: f"{len(e)}x{sum(e)}")
def test_norm(tide, elems, kinds, shift):
    T, host, dev = make_list(tide, elems, kinds, 1, shift=shift)
    norm, sumsq = torch.full((1,), -1.0, device="cuda"), torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
    got = []
    for _ in range(2):
        T.grad_norm([d.view for d in dev], norm, sumsq)
        got.append((norm.item(), sumsq.item()))
    assert got[0] == got[1]
    want = sum(float(x.double().square().sum()) for x in host)
    # 32 squares are summed in fp32 (each square and the 31 additions are off by u at most), the rest in fp64
    assert abs(sumsq.item() - want) <= 33 * U * want
    assert abs(norm.item() - math.sqrt(want)) <= 18 * U * math.sqrt(want)
    for x, d in zip(host, dev):
        assert torch.equal(d.cpu(), x)


@pytest.mark.parametrize("sigma", [1e-38, 1e-30, 1e-20, 1e15, 1e19, 1e30, 3e37])
def test_norm_neither_overflows_nor_vanishes(tide, sigma):
    for n in (5, 5000):
        T, host, dev = make_list(tide, (n,), "f32", 2, sigma)
        norm, sumsq = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.float64, device="cuda")
        T.grad_norm([d.view for d in dev], norm, sumsq)
        want = float(host[0].double().square().sum())
        assert abs(sumsq.item() - want) <= 33 * U * want
        if math.sqrt(want) < 3e38:
            assert abs(norm.item() - math.sqrt(want)) <= 18 * U * math.sqrt(want) + 2.0 ** -149


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_norm_of_values_that_are_not_finite(tide, value):
    T, host, dev = make_list(tide, (10, 5000), "mixed", 3)
    dev[1].view[4321] = value
    norm = torch.zeros(1, device="cuda")
    T.grad_norm([d.view for d in dev], norm)
    assert math.isnan(norm.item()) if math.isnan(value) else norm.item() == float("inf")


def clip_factor(norm, max_norm):
    return min(1.0, float(torch.tensor(max_norm, dtype=torch.float32)) / (norm + float(torch.tensor(1e-6, dtype=torch.float32))))


@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 3.0, 1e9, float("inf")])
@pytest.mark.parametrize("kinds, shift", [("f32", 0), ("bf16", 0), ("mixed", 1)])
@pytest.mark.parametrize("elems", LISTS[1:6], ids=lambda e: f"{len(e)}x{sum(e)}")
def test_clip(tide, elems, kinds, shift, max_norm):
    T, host, dev = make_list(tide, elems, kinds, 4, shift=shift)
    norm = torch.zeros(1, device="cuda")
    T.clip_grad_norm([d.view for d in dev], max_norm, norm)
    want_norm = math.sqrt(sum(float(x.double().square().sum()) for x in host))
    assert abs(norm.item() - want_norm) <= 18 * U * want_norm
    c = clip_factor(norm.item(), max_norm)
    for x, d in zip(host, dev):
        got = d.cpu()
        if c == 1:
            assert torch.equal(got, x)
            continue
        want = x.double() * c
        # the factor's sum and quotient, the product: 3 u; then one rounding to bf16
        lim = 4 * U * want.abs() + (2.0 ** -8 * want.abs() if x.dtype == torch.bfloat16 else 0) + 2.0 ** -140
        assert bool(((got.double() - want).abs() <= lim).all())


def test_a_list_without_elements(tide):
    T = tide.TensorList((0, 0))
    norm = torch.full((1,), 5.0, device="cuda")
    T.clip_grad_norm([0, 0], 1.0, norm)
    assert norm.item() == 0
    T.clip_grads([0, 0], norm, 1.0)
    T.adamw([0, 0], [0, 0], [0, 0], [0, 0], lr=0.1, step=1)
    torch.cuda.synchronize()


def test_clip_by_a_norm_that_is_not_finite(tide):
    T, host, dev = make_list(tide, (100, 3000), "mixed", 5)
    T.clip_grads([d.view for d in dev], torch.full((1,), float("inf"), device="cuda"), 1.0)
    assert all(bool((d.cpu() == 0).all()) for d in dev)
    T, host, dev = make_list(tide, (100, 3000), "mixed", 5)
    T.clip_grads([d.view for d in dev], torch.full((1,), float("nan"), device="cuda"), 1.0)
    assert all(bool(d.cpu().isnan().all()) for d in dev)


def test_clip_by_a_bound_that_is_infinite(tide):
    """Nothing is scaled, unless the norm is infinite too: the factor is then a quotient of infinities."""
    for value, nan in ((3.0, False), (float("inf"), True)):
        T, host, dev = make_list(tide, (100, 3000), "mixed", 5)
        T.clip_grads([d.view for d in dev], torch.full((1,), value, device="cuda"), float("inf"))
        assert all(bool(d.cpu().isnan().all()) if nan else torch.equal(d.cpu(), x) for x, d in zip(host, dev))


def check_adamw(p, g, m, v, c, lr, b1, b2, eps, wd, step, got):
    """got: (param, exp_avg, exp_avg_sq, shard or None) against 64 bits."""
    p, g, m, v = (x.double() for x in (p, g, m, v))
    g = g * c
    m_parts = (b1 * m).abs() + ((1 - b1) * g).abs()
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    den = (v2 / (1 - b2 ** step)).sqrt() + eps
    size = lr / (1 - b1 ** step)
    p2 = p * (1 - lr * wd) - size * m2 / den
    gp, gm, gv, gs = got
    tiny = 2.0 ** -140
    # g carries 3 u (the factor and the product); every product and sum adds one, and each factor its own
    assert bool(((gm.double() - m2).abs() <= 8 * U * m_parts + tiny).all())
    assert bool(((gv.double() - v2).abs() <= 12 * U * v2 + tiny).all())
    # half of v's, the root, its factor, eps, the quotient and the step size on top of m's
    lim = 4 * U * p.abs() + 32 * U * size * m_parts / den + 2 * U * p2.abs() + tiny
    assert bool(((gp.double() - p2).abs() <= lim).all()), float(((gp.double() - p2).abs() - lim).max())
    if gs is not None:
        assert torch.equal(gs, gp.bfloat16())


@pytest.mark.parametrize("kinds, shift", [("f32", 0), ("bf16", 0), ("mixed", 1), ("f32", 4)])
@pytest.mark.parametrize("elems", LISTS[1:6], ids=lambda e: f"{len(e)}x{sum(e)}")
def test_adamw(tide, elems, kinds, shift):
    K = len(elems)
    for case, (step, b1, b2, eps, decay, norm, max_norm, with_shards) in enumerate((
            (1, 0.9, 0.95, 1e-8, 0.1, None, 0.0, True), (7, 0.9, 0.999, 1e-8, None, 40.0, 1.0, False),
            (1000, 0.0, 0.5, 1e-5, "each", 0.5, 1.0, True), (3, 0.99, 0.0, 1e-3, 0.0, 2.0, 0.5, True))):
        T, grads, dg = make_list(tide, elems, kinds, 6 + case, 1e-2, shift=shift)
        g = gen(60 + case)
        host = [[torch.randn(n, generator=g) * s for n in elems] for s in (0.02, 1e-3)] + [[(torch.randn(n, generator=g) * 1e-2).square() for n in elems]]
        # the arrays' alignments agree, except with shift 4, where each has its own
        dev = [[Guarded(x, shift and ((shift + k) % 9 if shift == 1 else (shift * a + k) % 9)) for k, x in enumerate(xs)] for a, xs in enumerate(host)]
        ds = [Guarded(torch.zeros(n).bfloat16(), shift and (shift + k) % 9) for k, n in enumerate(elems)]
        decays = [0.01 * k for k in range(K)] if decay == "each" else decay
        T.adamw(*[[x.view for x in xs] for xs in (dev[0], dg, dev[1], dev[2])], [x.view for x in ds] if with_shards else None, lr=1e-2, betas=(b1, b2),
                eps=eps, weight_decay=decays, step=step, norm=None if norm is None else torch.full((1,), norm, device="cuda"), max_norm=max_norm)
        c = 1.0 if norm is None else clip_factor(norm, max_norm)
        for k in range(K):
            wd = (decays[k] if decay == "each" else decay) or 0.0
            check_adamw(host[0][k], grads[k], host[1][k], host[2][k], c, 1e-2, b1, b2, eps, wd, step,
                        (dev[0][k].cpu(), dev[1][k].cpu(), dev[2][k].cpu(), ds[k].cpu() if with_shards else None))
            assert torch.equal(dg[k].cpu(), grads[k])
            if not with_shards:
                assert bool((ds[k].cpu() == 0).all())


def test_adamw_leaves_all_unchanged_after_a_norm_that_is_not_finite(tide):
    for value in (float("inf"), float("nan")):
        T, grads, dg = make_list(tide, (50, 4000), "f32", 8)
        bufs = [[torch.randn(n, generator=gen(n)).cuda() for n in T.elems] for _ in range(3)]
        before = [[x.clone() for x in xs] for xs in bufs]
        shards = [torch.ones(n, dtype=torch.bfloat16, device="cuda") for n in T.elems]
        a = dict(lr=0.1, step=1, norm=torch.full((1,), value, device="cuda"), max_norm=1.0)
        T.adamw(bufs[0], [d.view for d in dg], bufs[1], bufs[2], shards, flags=tide.TIDE_ADAMW_SKIP_NONFINITE, **a)
        assert all(torch.equal(x, y) for xs, ys in zip(bufs, before) for x, y in zip(xs, ys)) and all(bool((s == 1).all()) for s in shards)
        T.adamw(bufs[0], [d.view for d in dg], bufs[1], bufs[2], shards, **a)
        assert not torch.equal(bufs[1][1], before[1][1])


def test_list_refusals(tide):
    T, host, dev = make_list(tide, (4, 6), "mixed", 9)
    views = [d.view for d in dev]
    f = [torch.zeros(n, device="cuda") for n in T.elems]
    norm = torch.zeros(1, device="cuda")
    E = tide.TIDE_EINVAL

    def status(fn, *a, **k):
        with pytest.raises(tide.TideError) as e:
            fn(*a, **k)
        return e.value.status

    assert status(T.grad_norm, views[:1], norm) == E
    assert status(T.grad_norm, [views[0], views[1][:5]], norm) == E
    assert status(T.grad_norm, [views[0].data_ptr() + 2, views[1]], norm) == E
    assert status(T.grad_norm, [0, views[1]], norm) == E
    assert status(T.grad_norm, [views[0], views[1].float()], norm) == E and status(T.grad_norm, views, norm.double()) == E
    assert status(T.grad_norm, views, norm, norm) == E and status(T.grad_norm, [v.cpu() for v in views], norm) == E
    assert status(T.clip_grads, views, norm, -1.0) == E and status(T.clip_grads, views, norm, float("nan")) == E
    assert status(T.clip_grad_norm, views, -1.0, norm) == E
    good = dict(lr=0.1, step=1)
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(eps=-1.0), dict(eps=float("inf")), dict(step=0), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)),
                dict(norm=norm, max_norm=-1.0), dict(flags=2), dict(weight_decay=-0.1), dict(weight_decay=[0.1, float("nan")]), dict(weight_decay=[0.1])):
        assert status(T.adamw, f, views, f, f, **dict(good, **bad)) == E, bad
    assert status(T.adamw, f, views, f, f, [f[0].bfloat16()], **good) == E
    torch.cuda.synchronize()


def test_lists_are_not_captured(tide):
    """Their pointer tables are shared with later calls, so a graph must not hold them."""
    T = tide.TensorList((100,))
    x, norm = torch.ones(100, device="cuda"), torch.zeros(1, device="cuda")
    T.grad_norm([x], norm)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(tide.TideError) as e:
            T.grad_norm([x], norm)
        norm.add_(1)
    assert e.value.status == tide.TIDE_EINVAL
    T.grad_norm([x], norm)
    assert norm.item() == 10


@pytest.mark.parametrize("elems", [(0,), (100,), (5000, 7)], ids=str)
def test_a_list_is_on_the_device_when_it_is_created(tide, elems):
    """Its first call may be on a stream that does not wait for the default one, which is busy here."""
    x, norm, side = [torch.ones(n, device="cuda") for n in elems], torch.full((1,), -1.0, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    assert not torch.cuda.default_stream().query()
    T = tide.TensorList(elems)
    assert torch.cuda.default_stream().query()
    T.grad_norm(x, norm, stream=side)
    side.synchronize()
    want = math.sqrt(sum(elems))
    assert abs(norm.item() - want) <= 18 * U * want


def test_lists_on_several_streams(tide):
    """One list, other tensors on each of six streams (more than its ring holds), all in flight at once."""
    elems = (100_000, 3, 70_001)
    T = tide.TensorList(elems)
    streams, sets = [torch.cuda.Stream() for _ in range(6)], []
    for k in range(6):
        g = gen(k)
        sets.append(([torch.randn(n, generator=g).cuda() for n in elems], torch.zeros(1, device="cuda")))
    want = [math.sqrt(sum(float(x.double().square().sum()) for x in xs)) for xs, _ in sets]
    torch.cuda.synchronize()
    for rep in range(3):
        for s, (xs, norm) in zip(streams, sets):
            T.grad_norm(xs, norm, stream=s)
    torch.cuda.synchronize()
    for w, (_, norm) in zip(want, sets):
        assert abs(norm.item() - w) <= 18 * U * w


def test_one_handle_for_the_streams_of_several_threads(tide):
    """Handle 2 is each thread's own default stream: calls of two threads with equal arguments share nothing on the device."""
    import threading

    per_thread = 2
    elems = (3_000_000, 70_001)
    T = tide.TensorList(elems)
    xs = [torch.randn(n, generator=gen(n)).cuda() for n in elems]
    want = math.sqrt(sum(float(x.double().square().sum()) for x in xs))
    norms = torch.zeros(2, 200, device="cuda")
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def run(k):
        start.wait()
        for rep in range(norms.shape[1]):
            T.grad_norm(xs, norms[k, rep : rep + 1], stream=per_thread)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert float((norms.double() - want).abs().max()) <= 18 * U * want


# ---- all of it together --------------------------------------------------------------------------


def _example():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sharded_step.py")
    spec = importlib.util.spec_from_file_location("sharded_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_sharded_step_is_the_unsharded_step(tide):
    """One step of the example against the same step on whole fp32 tensors: autograd through an index, dense
    gradients rounded to bf16 per rank as the reduce-scatter reads them, sums, norm and AdamW in 64 bits."""
    ex = _example()
    R, vocab, dim, tokens = 3, 101, 64, 40
    model = ex.ShardedModel(R, vocab, dim, tokens)
    G = model.group
    start = [torch.cat([model.master[d][G.param_layout(p)[1]:][:G.valid_rows(d, p) * dim] for d in range(R)]).view(-1, dim).clone() for p in (0, 1)]
    data = ex.batches(R, vocab, tokens, 0)
    model.step(data, lr=1e-2, max_norm=0.05, weight_decay=0.1)
    sums = [torch.zeros_like(p, dtype=torch.float64) for p in start]
    for t, target in data:
        E, W = (p.bfloat16().requires_grad_(True) for p in start)
        x = (start[0].bfloat16().float()[t] * dim ** 0.5).bfloat16().requires_grad_(True)
        loss = torch.nn.functional.cross_entropy((torch.relu(x @ W) @ E.t()).float(), target) / R
        loss.backward()
        sums[0] += E.grad.double()
        sums[1] += W.grad.double()
        sums[0].index_add_(0, t, x.grad.double() * float(torch.tensor(dim ** 0.5, dtype=torch.float32)))
    norm = math.sqrt(sum(float(s.square().sum()) for s in sums))
    assert abs(model.norm.item() - norm) <= 1e-5 * norm and norm > 0.05
    c = 0.05 / (norm + 1e-6)
    for p in (0, 1):
        g = sums[p] * c
        want = start[p].double() * (1 - 1e-2 * 0.1) - 1e-2 * g / (g.abs() + 1e-8)  # the first step: m / sqrt(v) is the gradient's sign
        got = torch.cat([model.master[d][G.param_layout(p)[1]:][:G.valid_rows(d, p) * dim] for d in range(R)]).view(-1, dim)
        # near g = 0 the quotient turns fast: what the sums' rounding (at most 200 terms) can move it by
        slack = 1e-2 * (1e-8 + 2e-5 * g.abs().max()) / (g.abs() + 1e-8)
        assert bool(((got.double() - want).abs() <= 1e-6 + torch.minimum(slack, torch.tensor(2e-2))).all())
    for d in range(R):
        for p in (0, 1):
            o, n = G.param_layout(p)[1], G.valid_rows(d, p) * dim
            assert torch.equal(model.shards[d, o:o + n], model.master[d, o:o + n].bfloat16())


def test_example_learns(tide):
    ex = _example()
    model = ex.ShardedModel(4, 211, 128, 256)
    losses = [float(model.step(ex.batches(4, 211, 256, k))) for k in range(40)]
    assert losses[0] > 4.5 and losses[-1] < 0.5 * losses[0] and all(math.isfinite(x) for x in losses), losses
