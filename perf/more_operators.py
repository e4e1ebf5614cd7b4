"""A layer of experts' operators, as cases to time and compare.

Tokens go to k of E experts each; the (token, expert) pairs are sorted by expert, the experts' weight
matrices (parameters of a sharded group) multiply the sorted rows in 8-bit floating point (e4m3, one
power-of-two scale for each block of 128), and the results go back to their tokens:

* ``dispatch``: the stable sort of the pairs by expert, and the tokens' rows copied into that order;
* ``combine``: each token's k rows back, summed with the router's weights;
* ``back``: the gradients of both: of the rows, of the weights, and of the tokens;
* ``product``: sort, rows into that order in 8 bits, and their product with the experts' weights;
* ``train``: one weight matrix's whole step: weights from the ranks' bf16 shards to 8 bits, the product,
  and from the product's gradient those of the rows and of the weights.

Where ``own`` is false ``run`` computes them with elementary torch operations in fp32; where it is
true it calls ``all_gather_tide_gb300``.
"""
import math

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "int32": torch.int32, "int64": torch.int64}
BLOCK = 128  # values that share a scale


def listed():
    return [
        # one token of a decoding step over 128 experts: latency alone
        _rows("dispatch_one_token", "dispatch", T=1, k=8, E=128, D=2048, ids="int64", dtype="bf16", masked=0.0),
        # eight sequences of 8192 tokens, as this repository's expert layer has them (128 experts of rows of 2048, 8 a token)
        _rows("dispatch_sequences", "dispatch", T=65536, k=8, E=128, D=2048, ids="int64", dtype="bf16", masked=0.0),
        # odd rows in fp32, few experts, pairs without an expert (padding, or dropped by the router)
        _rows("dispatch_odd", "dispatch", T=4099, k=3, E=50, D=1027, ids="int32", dtype="f32", masked=0.05),
        # the way back of those sequences
        _rows("combine_sequences", "combine", T=65536, k=8, E=128, D=2048, ids="int64", dtype="bf16", masked=0.0),
        # odd rows: every row off its vector boundary
        _rows("combine_odd", "combine", T=4099, k=3, E=50, D=1027, ids="int32", dtype="bf16", masked=0.05),
        # a training batch's gradients
        _rows("back_sequences", "back", T=32768, k=8, E=128, D=2048, ids="int64", dtype="bf16", masked=0.0),
        # odd rows in fp32, pairs without an expert
        _rows("back_odd", "back", T=4099, k=3, E=50, D=1027, ids="int32", dtype="f32", masked=0.05),
        # one token of a decoding step: the weights of 8 experts are read for one row each
        _product("product_one_token", "product", T=1, k=8, E=128, N=1536, K=2048, ids="int64", out="bf16", masked=0.0),
        # prompts of 8 x 8192 tokens through gate and up projections side by side
        _product("product_sequences", "product", T=65536, k=8, E=128, N=1536, K=2048, ids="int64", out="bf16", masked=0.0),
        # sizes off every tile, an output in fp32, pairs without an expert
        _product("product_odd", "product", T=3001, k=2, E=5, N=1003, K=1027, ids="int32", out="f32", masked=0.05),
        # two sequences of 8192 tokens of a training step, the weights on 8 ranks
        _product("train_sequences", "train", T=16384, k=8, E=128, N=768, K=2048, ids="int64", out="bf16", masked=0.0, R=8),
        # a short batch, odd sizes, more rows a rank than the last one has
        _product("train_odd", "train", T=1500, k=2, E=9, N=331, K=525, ids="int32", out="bf16", masked=0.05, R=3),
    ]


def _rows(name, op, T, k, E, D, ids, dtype, masked):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "D": D, "ids": ids, "dtype": dtype, "masked": masked}


def _product(name, op, T, k, E, N, K, ids, out, masked, R=1):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "ids": ids, "out": out, "masked": masked, "R": R}


# ---- drawn cases -------------------------------------------------------------------------------


def _between(rng, lo, hi):
    """A whole number spread over its logarithm, any remainder."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    v = _between(rng, lo, hi)
    return v if rng.random() < 0.4 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(("dispatch", "combine", "back", "product", "product", "train"))
    E = _between(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    ids, masked = rng.choice(("int32", "int64")), rng.choice((0.0, 0.0, 0.05, 0.5))
    if op in ("dispatch", "combine", "back"):
        D = _width(rng, 64, 8192)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        row = D * (2 if dtype == "bf16" else 4)
        most = 32768 * 26 * 4096 // ((3 * k + 2) * row) if op == "back" else 65536 * 9 * 4096 // ((k + 1) * row)
        c = _rows("", op, T=_between(rng, 1, min(65536, most)), k=k, E=E, D=D, ids=ids, dtype=dtype, masked=masked)
    else:
        N, K = _width(rng, 64, 4096), _width(rng, 64, 4096)
        E = min(E, max(2, 128 * 1536 * 2048 // (N * K)))
        k = min(k, E)
        most = (65536 * 8 * 1536 * 2048 if op == "product" else 16384 * 8 * 768 * 2048) // (k * N * K)
        R = rng.choice((1, 2, 3, 8)) if op == "train" else 1
        c = _product("", op, T=_between(rng, 1, min(65536, most)), k=k, E=E, N=N, K=K, ids=ids, out=rng.choice(("bf16", "bf16", "f32")), masked=masked, R=R)
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)


def _normal(g, shape, sigma, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").mul_(sigma).to(dtype)


def _activations(g, rows, width, dtype):
    """Normal values, some columns being ten times as large as the others, as a model's are."""
    large = torch.where(torch.rand(width, generator=g, device="cuda") < 0.01, 10.0, 1.0)
    return torch.randn(rows, width, generator=g, device="cuda").mul_(large).to(dtype)


def _ids(case, g):
    """The k experts with the largest of random scores of each token, some experts being more popular, and a share of the pairs without one."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.rand(T, E, generator=g, device="cuda").log_().neg_().log_().neg_()
    score += _normal(g, (E,), 0.5)
    ids = score.topk(k, dim=1).indices
    if case["masked"]:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["masked"], torch.full_like(ids, -1), ids)
    return ids.to(TORCH[case["ids"]])


def _weights(g, T, k):
    """The router's weights: they add up to one for each token."""
    return torch.softmax(_normal(g, (T, k), 1.0), dim=1)


def _m(case):
    return -(-case["N"] // case["R"])


def _inputs(case, seed):
    g = _generator(seed)
    T, k, E, M = case["T"], case["k"], case["E"], case["T"] * case["k"]
    x = {"ids": _ids(case, g)}
    if case["op"] in ("dispatch", "combine", "back"):
        D, dtype = case["D"], TORCH[case["dtype"]]
        if case["op"] == "dispatch":
            x["x"] = _normal(g, (T, D), 1.0, dtype)
            return x
        x["rows"], x["weights"] = _normal(g, (M, D), 1.0, dtype), _weights(g, T, k)
        if case["op"] == "back":
            x["dout"], x["grads"] = _normal(g, (T, D), 1e-3, dtype), _normal(g, (M, D), 1e-3, dtype)
        return x
    N, K, R = case["N"], case["K"], case["R"]
    m = _m(case)
    x["x"] = _activations(g, T, K, torch.bfloat16)
    # the ranks' packed shards: of every expert's N x K matrix each holds m rows, zeros behind the last
    full = torch.zeros(E, R * m, K, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        full[e, :N] = _normal(g, (N, K), K ** -0.5)
    x["shards"] = full.view(E, R, m * K).transpose(0, 1).reshape(R, E * m * K)
    if case["op"] == "train":
        x["dy"] = _normal(g, (M, N), 1e-4, torch.bfloat16)
    return x


def _matrices(case, shards):
    """[E, N, K] from the ranks' shards."""
    R, m = case["R"], _m(case)
    return shards.view(R, case["E"], m, case["K"]).transpose(0, 1).reshape(case["E"], R * m, case["K"])[:, :case["N"]]


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    M, dev = T * k, {"device": "cuda"}
    if op in ("dispatch", "combine", "back"):
        D, dtype = case["D"], TORCH[case["dtype"]]
        if op != "dispatch":  # a layer has its order from the way there
            state["offsets"], state["slots"], state["tokens"] = _sorted(state["ids"], E)
        if op != "combine":
            state["new_rows"] = torch.zeros(M, D, dtype=dtype, **dev)
        if op != "dispatch":
            state["out"] = torch.empty(T, D, dtype=dtype, **dev)
        if op == "back":
            state["dweights"] = torch.empty(T, k, **dev)
    else:
        N, K = case["N"], case["K"]
        state["y"] = torch.zeros(M, N, dtype=TORCH[case["out"]], **dev)
        if op == "train":
            state["dx"] = torch.zeros(M, K, dtype=TORCH[case["out"]], **dev)
            state["dw"] = torch.empty(E, N, K, dtype=torch.bfloat16, **dev)
        elif not own:  # weights laid out once, as a server keeps them
            state["w8"] = _blocks(_matrices(case, state["shards"]))
    if own:
        import all_gather_tide_gb300 as tide

        state["experts"] = tide.Experts(E, k)
        state["route"] = state["experts"].route(T)
        if op in ("combine", "back"):
            for name in ("offsets", "slots", "tokens"):
                getattr(state["route"], name).copy_(state[name])
        if op in ("product", "train"):
            state["group"] = tide.Group(case["R"], [(N, K)] * E)
            state["table"] = tide.pointer_table(list(state["shards"]))
            state["w8"] = tide.Fp8Weights(E, N, K, transposed=op == "train")
            state["x8"] = tide.Fp8Rows(M, K)
            if op == "train":
                state["xt8"], state["dy8"], state["dyt8"] = tide.Fp8Columns(M, K, E), tide.Fp8Rows(M, N), tide.Fp8Columns(M, N, E)
            else:
                state["group"].all_gather_fp8(range(E), state["table"], state["w8"])
    return state


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_dispatch(st):
    ex, route = st["experts"], st["route"]
    ex.sort(st["ids"], route)
    ex.dispatch(st["x"], route, st["new_rows"])
    return {"offsets": route.offsets, "slots": route.slots, "tokens": route.tokens, "rows": st["new_rows"]}


def _own_combine(st):
    st["experts"].combine(st["rows"], st["route"], st["out"], st["weights"])
    return st["out"]


def _own_back(st):
    ex, route = st["experts"], st["route"]
    ex.combine_grad(st["dout"], st["rows"], route, st["weights"], st["new_rows"], st["dweights"])
    ex.combine(st["grads"], route, st["out"])
    return {"drows": st["new_rows"], "dweights": st["dweights"], "dx": st["out"]}


def _own_product(st):
    ex, route = st["experts"], st["route"]
    ex.sort(st["ids"], route)
    ex.dispatch_fp8(st["x"], route, st["x8"])
    ex.matmul(st["x8"], st["w8"], route, st["y"])
    return st["y"]


def _own_train(st):
    ex, route = st["experts"], st["route"]
    st["group"].all_gather_fp8(range(st["case"]["E"]), st["table"], st["w8"])
    ex.sort(st["ids"], route)
    ex.dispatch_fp8(st["x"], route, st["x8"])
    ex.matmul(st["x8"], st["w8"], route, st["y"])
    ex.quantize(st["dy"], route, rows=st["dy8"], columns=st["dyt8"])
    ex.matmul(st["dy8"], st["w8"], route, st["dx"], transposed=True)
    ex.quantize(st["x"], route, columns=st["xt8"], gather=True)
    ex.weight_grad(st["dyt8"], st["xt8"], route, st["dw"])
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def _sorted(ids, E):
    """offsets, slots and tokens of the stable order by expert; -1 for pairs without an expert and for rows behind the last."""
    flat = ids.flatten().long()
    held = (flat >= 0) & (flat < E)
    key = torch.where(held, flat, E)
    order = key.sort(stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    slots = torch.where(held, place, -1).to(torch.int32).view(ids.shape)
    tokens = torch.where(held[order], order // ids.shape[1], -1).to(torch.int32)
    return offsets, slots, tokens


def _plain_dispatch(st):
    offsets, slots, tokens = _sorted(st["ids"], st["case"]["E"])
    held = tokens >= 0
    rows = st["new_rows"]
    rows.copy_(torch.where(held[:, None], st["x"][tokens.clamp(min=0).long()], rows))
    return {"offsets": offsets, "slots": slots, "tokens": tokens, "rows": rows}


def _plain_combine(st):
    return _weighted(st["rows"], st["slots"], st["weights"], st["out"])


def _weighted(rows, slots, weights, out):
    total = torch.zeros(out.shape, device="cuda")
    for j in range(slots.shape[1]):
        s = slots[:, j].long()
        part = rows[s.clamp(min=0)].float()
        if weights is not None:
            part *= weights[:, j, None]
        total += torch.where(s[:, None] >= 0, part, 0.0)
    return out.copy_(total)


def _plain_back(st):
    rows, dout, new = st["rows"], st["dout"].float(), st["new_rows"]
    for j in range(st["case"]["k"]):
        s = st["slots"][:, j].long()
        at = torch.nonzero(s >= 0).flatten()
        d = dout[at]
        new[s[at]] = (d * st["weights"][at, j, None]).to(new.dtype)
        st["dweights"][:, j] = 0
        st["dweights"][at, j] = (rows[s[at]].float() * d).sum(1)
    return {"drows": new, "dweights": st["dweights"], "dx": _weighted(st["grads"], st["slots"], None, st["out"])}


def _scale(amax):
    """The smallest power of two, from 2^-126 to 2^120, by which the largest value comes within e4m3's 448; 1 for zeros."""
    mantissa, exponent = torch.frexp(amax)
    exponent = exponent - torch.where(mantissa <= 0.875, 9, 8)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), exponent.clamp(-126, 120)), 1.0)


def _rounded(x, scale):
    """The values that 8 bits hold of x, once scaled, times the scale."""
    return (x / scale).to(torch.float8_e4m3fn).float() * scale


def _padded(x, rows, columns):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % columns, 0, -x.shape[-2] % rows))


def _by_row(x):
    """x in 8 bits with a scale for each block of a row's 128 columns."""
    p = _padded(x.float(), 1, BLOCK).unflatten(1, (-1, BLOCK))
    return _rounded(p, _scale(p.abs().amax(2, keepdim=True))).flatten(1)[:, :x.shape[1]]


def _by_column(x):
    """x in 8 bits with a scale for each block of a column's 128 rows."""
    p = _padded(x.float(), BLOCK, 1).unflatten(0, (-1, BLOCK))
    return _rounded(p, _scale(p.abs().amax(1, keepdim=True))).flatten(0, 1)[:x.shape[0]]


def _blocks(w):
    """[E, N, K] in 8 bits with a scale for each block of 128 x 128."""
    out = torch.empty(w.shape, device="cuda")
    for e, x in enumerate(w):
        p = _padded(x.float(), BLOCK, BLOCK).unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))
        out[e] = _rounded(p, _scale(p.abs().amax((1, 3), keepdim=True))).flatten(2, 3).flatten(0, 1)[:x.shape[0], :x.shape[1]]
    return out


def _plain_product(st):
    offsets, _, tokens = _sorted(st["ids"], st["case"]["E"])
    x8, at = _by_row(st["x"]), offsets.tolist()
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if b > a:
            st["y"][a:b] = (x8[tokens[a:b].long()] @ st["w8"][e].t()).to(st["y"].dtype)
    return st["y"]


def _plain_train(st):
    offsets, _, tokens = _sorted(st["ids"], st["case"]["E"])
    w8, x8, dy8, at = _blocks(_matrices(st["case"], st["shards"])), _by_row(st["x"]), _by_row(st["dy"]), offsets.tolist()
    for e, (a, b) in enumerate(zip(at, at[1:])):
        t = tokens[a:b].long()
        if b > a:
            st["y"][a:b] = (x8[t] @ w8[e].t()).to(st["y"].dtype)
            st["dx"][a:b] = (dy8[a:b] @ w8[e]).to(st["dx"].dtype)
            st["dw"][e] = (_by_column(st["dy"][a:b]).t() @ _by_column(st["x"][t])).to(torch.bfloat16)
        else:
            st["dw"][e] = 0
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


_own = {"dispatch": _own_dispatch, "combine": _own_combine, "back": _own_back, "product": _own_product, "train": _own_train}
_plain = {"dispatch": _plain_dispatch, "combine": _plain_combine, "back": _plain_back, "product": _plain_product, "train": _plain_train}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def _order(ids, E):
    """Pairs of every expert, in order, on the host's side of the definition: one list of pair numbers an expert."""
    flat = ids.flatten().long()
    return [torch.nonzero(flat == e).flatten() for e in range(E)]


def _e4m3(x, dims):
    """x in 64 bits, rounded to the values that e4m3 (3 bits of mantissa, exponents from -6, at most 448) and one power of two for each
    block over `dims` hold, halves to even."""
    amax = x.abs().amax(dims, keepdim=True)
    power = torch.ceil(torch.log2(torch.where(amax > 0, amax, 448.0) / 448.0)).clamp(-126, 120)
    x = x * torch.exp2(-power)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step * torch.exp2(power)


def _in_rows(x):
    c = x.shape[1]
    return torch.cat([_e4m3(x[:, i:i + BLOCK], (1,)) for i in range(0, c, BLOCK)], 1)


def _in_columns(x):
    return torch.cat([_e4m3(x[i:i + BLOCK], (0,)) for i in range(0, x.shape[0], BLOCK)])


def _in_blocks(w):
    return torch.cat([torch.cat([_e4m3(w[i:i + BLOCK, j:j + BLOCK], (0, 1)) for j in range(0, w.shape[1], BLOCK)], 1) for i in range(0, w.shape[0], BLOCK)])


def exact(case, seed):
    x, k, E = _inputs(case, seed), case["k"], case["E"]
    T, M, op = case["T"], case["T"] * case["k"], case["op"]
    order = _order(x["ids"], E)
    if op == "dispatch":
        pairs = torch.cat(order)
        n = pairs.numel()
        offsets = torch.tensor([0] + [len(o) for o in order], device="cuda").cumsum(0).to(torch.int32)
        slots = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        slots[pairs] = torch.arange(n, dtype=torch.int32, device="cuda")
        tokens = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        tokens[:n] = pairs // k
        rows = torch.zeros(M, case["D"], dtype=torch.float64, device="cuda")
        rows[:n] = x["x"].double()[pairs // k]
        return {"offsets": offsets, "slots": slots.view(T, k), "tokens": tokens, "rows": rows}
    if op in ("combine", "back"):
        pairs = torch.cat(order)
        n = pairs.numel()
        t, w = pairs // k, x["weights"].double().flatten()[pairs][:, None]

        def back(rows, by):
            out = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
            for a in range(0, n, 1 << 16):
                b = min(n, a + (1 << 16))
                out.index_add_(0, t[a:b], rows[a:b].double() * by[a:b])
            return out

        if op == "combine":
            return back(x["rows"], w)
        drows = torch.zeros(M, case["D"], dtype=torch.float64, device="cuda")
        dweights = torch.zeros(M, dtype=torch.float64, device="cuda")
        for a in range(0, n, 1 << 16):
            b = min(n, a + (1 << 16))
            d = x["dout"][t[a:b]].double()
            drows[a:b] = d * w[a:b]
            dweights[pairs[a:b]] = (d * x["rows"][a:b].double()).sum(1)
        return {"drows": drows, "dweights": dweights.view(T, k), "dx": back(x["grads"], torch.ones_like(w))}
    # products in 64 bits take a second for each 10^12 operations
    N, K = case["N"], case["K"]
    m = _m(case)
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    dx = torch.zeros(M, K, dtype=torch.float64, device="cuda") if op == "train" else None
    dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda") if op == "train" else None
    a = 0
    for e, pairs in enumerate(order):
        b = a + len(pairs)
        if b == a:
            continue
        w = _in_blocks(torch.cat([s[e * m * K:(e + 1) * m * K].view(m, K) for s in x["shards"]])[:N].double())
        rows = x["x"][pairs // k].double()
        y[a:b] = _in_rows(rows) @ w.t()
        if op == "train":
            dy = x["dy"][a:b].double()
            dx[a:b] = _in_rows(dy) @ w
            dw[e] = _in_columns(dy).t() @ _in_columns(rows)
        a = b
    return {"y": y, "dx": dx, "dw": dw} if op == "train" else y


# ---- what a pass cannot do without -------------------------------------------------------------


def _hit(case):
    """Experts that at least one of the tokens asks for, expected as if all were equally popular."""
    share = case["k"] / case["E"] * (1 - case["masked"])
    return case["E"] * -math.expm1(case["T"] * math.log1p(-min(share, 1 - 1e-12)))


def work(case):
    T, k, E = case["T"], case["k"], case["E"]
    M = T * k
    held = M * (1 - case["masked"])
    ids = M * {"int32": 4, "int64": 8}[case["ids"]]
    order = M * 8 + (E + 1) * 4
    if case["op"] in ("dispatch", "combine", "back"):
        row = case["D"] * {"bf16": 2, "f32": 4}[case["dtype"]]
        if case["op"] == "dispatch":
            return {"bytes": ids + order + (T + held) * row, "flops": 0}
        if case["op"] == "combine":
            return {"bytes": M * 8 + (T + held) * row, "flops": 2 * held * case["D"]}
        return {"bytes": M * 12 + (2 * T + 3 * held) * row, "flops": 4 * held * case["D"]}
    N, K, out = case["N"], case["K"], {"bf16": 2, "f32": 4}[case["out"]]
    if case["op"] == "product":
        return {"bytes": ids + T * K * 2 + _hit(case) * N * K + held * N * out, "flops": 2 * held * N * K}
    return {"bytes": ids + T * K * 2 + E * N * K * 4 + held * (N * 2 + (N + K) * out), "flops": 6 * held * N * K}
