"""The sharded training step's operators, as cases to time and compare.

Four operators over the packed dim-0 shards of a parameter group (R ranks, parameter p split into
R pieces of m = ceil(rows / R) rows, the pieces of all parameters back to back in each rank's shard):

* ``lookup``: embedding rows read from the ranks' bf16 shards, scaled;
* ``lookup_grad``: its gradient, summed by token into the ranks' fp32 gradient shards;
* ``clip``: the global norm over many gradient tensors, and clipping in place;
* ``adamw``: the optimizer step over the shards with the clip factor folded in, writing the fp32
  master, both moments and the bf16 shards that the lookup and the all-gather read.

Where ``own`` is false ``run`` computes them with elementary torch operations in fp32; where it is
true it calls ``all_gather_tide_gb300``.
"""
import math

import torch

own = False

LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "int32": torch.int32, "int64": torch.int64}

# Decoder-layer and expert-layer parameter lists of this repository's workloads: count*(rows x row_len + ...)
DENSE_8192 = "2*8192x8192;2*1024x8192;2*28672x8192;1*8192x28672;2*8192x1"
EXPERTS = "1*4096x2048;2*512x2048;1*2048x4096;2*128x1;1*128x2048;128*768x2048+768x2048+2048x768;2*2048x1"
SMALL_LAYER = "2*256x256;2*64x256;2*896x256;1*256x896;2*256x1"


def listed():
    return [
        # one token of a decoding step: latency alone
        _lookup("lookup_one_token", R=8, rows=128000, len=4096, n=1, ids="int64", out="bf16", masked=0.0),
        # eight sequences of 8192 tokens at once, wide rows
        _lookup("lookup_sequences", R=8, rows=128000, len=8192, n=65536, ids="int64", out="bf16", masked=0.0),
        # an odd row length behind a small parameter (every address off its vector boundary), with
        # positions that hold no token, into fp32
        _lookup("lookup_odd", R=3, rows=50021, len=1027, before=5, n=4099, ids="int32", out="f32", masked=0.05),
        # the gradient of a short batch in a small table: latency
        _grad("grad_short", R=2, rows=2048, len=256, n=64, batches=2, ids="int64", dout="bf16", masked=0.0, add=False),
        # a table with its own gradient: every row of the shards is written, most with zeros
        _grad("grad_untied", R=8, rows=128000, len=8192, n=65536, batches=8, ids="int64", dout="bf16", masked=0.0, add=False),
        # a table shared with the output layer, whose gradient is already in the shards: added to
        _grad("grad_tied", R=8, rows=128000, len=4096, n=131072, batches=8, ids="int64", dout="bf16", masked=0.02, add=True),
        # odd rows, three ragged batches, positions without a token, fp32 in
        _grad("grad_odd", R=3, rows=50021, len=1027, before=5, n=12289, batches=3, ids="int32", dout="f32", masked=0.05, add=False),
        # a small layer's shards: latency
        _clip("clip_small", R=8, params=SMALL_LAYER, grads="f32", max_norm=0.1),
        # 3144 pieces of many sizes: the shards of a layer with 128 experts, over the bound
        _clip("clip_experts", R=8, params=EXPERTS, grads="f32", max_norm=1.0),
        # one rank's bf16 gradients of a wide layer, within the bound: nothing to scale
        _clip("norm_within_bound", R=1, params=DENSE_8192, grads="bf16", max_norm=1000.0),
        # a small layer's step: latency
        _adamw("adamw_small", R=8, params=SMALL_LAYER, max_norm=0.1),
        # all eight shards of a wide layer
        _adamw("adamw_wide", R=8, params=DENSE_8192, max_norm=1.0),
    ]


def _lookup(name, R, rows, len, n, ids, out, masked, before=0, scale=1.5):
    return {"name": name, "op": "lookup", "R": R, "rows": rows, "len": len, "before": before, "n": n, "ids": ids, "out": out, "masked": masked, "scale": scale}


def _grad(name, R, rows, len, n, batches, ids, dout, masked, add, before=0, scale=1.5):
    return {"name": name, "op": "lookup_grad", "R": R, "rows": rows, "len": len, "before": before, "n": n, "batches": batches, "ids": ids, "dout": dout,
            "masked": masked, "add": add, "scale": scale}


def _clip(name, R, params, grads, max_norm):
    return {"name": name, "op": "clip", "R": R, "params": params, "grads": grads, "max_norm": max_norm}


def _adamw(name, R, params, max_norm):
    return {"name": name, "op": "adamw", "R": R, "params": params, "max_norm": max_norm}


# ---- drawn cases -------------------------------------------------------------------------------


def _between(rng, lo, hi):
    """A whole number spread over its logarithm, any remainder."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _row_len(rng, hi=8192):
    v = _between(rng, 64, hi)
    return v if rng.random() < 0.4 else v // 8 * 8


def _params(rng, most):
    """A few parameters, some repeated, of at most about `most` elements in all, and some of one-element rows."""
    blocks = rng.randint(1, 5)
    share = _between(rng, 60_000, most) / blocks
    out = []
    for _ in range(blocks):
        length = _row_len(rng)
        count = rng.choice((1, 1, 2, 5, 40))
        rows = max(1, int(share * rng.uniform(0.3, 1.0) / (length * count)))
        out.append("%d*%dx%d" % (count, rows, length))
        if rng.random() < 0.5:
            out.append("%d*%dx1" % (count, length))
    return ";".join(out)


def draw(rng):
    op = rng.choice(("lookup", "lookup_grad", "clip", "adamw"))
    if op in ("lookup", "lookup_grad"):
        common = dict(R=rng.choice((1, 2, 3, 4, 8, 16)), rows=_between(rng, 500, 128000), len=_row_len(rng), before=rng.choice((0, 0, 1, 5, 64)),
                      ids=rng.choice(("int32", "int64")), masked=rng.choice((0.0, 0.0, 0.05, 0.5)), scale=rng.choice((1.0, 1.5, 64.0)))
        if op == "lookup":
            c = _lookup("", n=_between(rng, 1, 65536), out=rng.choice(("bf16", "bf16", "f32")), **common)
        else:
            n = _between(rng, 1, min(131072, 65536 * 8192 // common["len"]))
            c = _grad("", n=n, batches=rng.choice((1, 2, 3, 8)), dout=rng.choice(("bf16", "bf16", "f32")), add=rng.random() < 0.5, **common)
    elif op == "clip":
        grads = rng.choice(("f32", "f32", "bf16"))
        c = _clip("", R=rng.choice((1, 2, 3, 8, 16)), params=_params(rng, 600_000_000), grads=grads, max_norm=rng.choice((0.001, 1.0, 1000.0)))
    else:
        c = _adamw("", R=rng.choice((1, 2, 3, 8, 16)), params=_params(rng, 600_000_000), max_norm=rng.choice((0.001, 1.0, 1000.0)))
    del c["name"]
    return c


# ---- shapes ------------------------------------------------------------------------------------


def _shapes(text):
    out = []
    for block in text.split(";"):
        count, shapes = block.split("*")
        out += [tuple(int(v) for v in s.split("x")) for s in shapes.split("+")] * int(count)
    return out


def _layout(R, shapes):
    """(m, s, o) of every parameter and the shard's elements S."""
    m = [-(-r // R) for r, _ in shapes]
    s = [a * l for a, (_, l) in zip(m, shapes)]
    o = [0]
    for v in s:
        o.append(o[-1] + v)
    return m, s, o[:-1], o[-1]


def _table(case):
    """The table's place in its group: shapes, its index, and m, s, o, S."""
    shapes = ([(case["before"], 1)] if case["before"] else []) + [(case["rows"], case["len"])]
    m, s, o, S = _layout(case["R"], shapes)
    return shapes, len(shapes) - 1, m[-1], s[-1], o[-1], S


def _pieces(R, shapes):
    """(rank, parameter, first element, elements) of every piece's valid rows."""
    m, _, o, _ = _layout(R, shapes)
    return [(d, p, o[p], max(0, min(m[p], rows - d * m[p])) * length) for d in range(R) for p, (rows, length) in enumerate(shapes)]


def _batches(case):
    """First positions of the batches, ragged where there are several, and the total."""
    n, b = case["n"], case["batches"]
    return [int(n * (k / b) ** 1.25) for k in range(b)] + [n]


# ---- inputs ------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _normal(g, shape, sigma, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(sigma)


def _ids(case, g):
    """Tokens as a text has them: the frequency falls as one over the rank, low numbers being frequent,
    and a share of the positions hold no token (-1)."""
    u = torch.rand(case["n"], generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(case["rows"] + 1)).long() - 1).clamp_(0, case["rows"] - 1)
    if case["masked"]:
        ids = torch.where(torch.rand(case["n"], generator=g, device="cuda") < case["masked"], torch.full_like(ids, -1), ids)
    return ids.to(TORCH[case["ids"]])


def _valid(R, shapes, buffer):
    """Zeroes the padding rows of [R, S] shards."""
    m, s, o, _ = _layout(R, shapes)
    for p, (rows, length) in enumerate(shapes):
        for d in range(rows // m[p], R):
            held = max(0, rows - d * m[p])
            buffer[d, o[p] + held * length:o[p] + s[p]] = 0
    return buffer


def _inputs(case, seed):
    g = _generator(seed)
    R = case["R"]
    if case["op"] == "lookup":
        shapes, _, _, _, _, S = _table(case)
        return {"shards": _valid(R, shapes, _normal(g, (R, S), 0.02, torch.bfloat16)), "ids": _ids(case, g)}
    if case["op"] == "lookup_grad":
        shapes, _, _, _, _, S = _table(case)
        state = {"ids": _ids(case, g), "douts": _normal(g, (case["n"], case["len"]), 1e-3, TORCH[case["dout"]])}
        state["shards"] = _valid(R, shapes, _normal(g, (R, S), 1e-3)) if case["add"] else torch.zeros(R, S, device="cuda")
        return state
    shapes = _shapes(case["params"])
    S = _layout(R, shapes)[3]
    if case["op"] == "clip":
        return {"grads": _valid(R, shapes, _normal(g, (R, S), 1e-3, TORCH[case["grads"]]))}
    state = {"master": _valid(R, shapes, _normal(g, (R, S), 0.02)), "grads": _valid(R, shapes, _normal(g, (R, S), 1e-3))}
    state["exp_avg"] = _valid(R, shapes, _normal(g, (R, S), 3e-4))
    state["exp_avg_sq"] = _valid(R, shapes, _normal(g, (R, S), 1e-3).square_())
    state["shards"] = state["master"].bfloat16()
    state["norm"] = torch.full((1,), 1e-3 * math.sqrt(R * S), device="cuda")
    state["step"] = 10
    return state


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    R, op = case["R"], case["op"]
    if op == "lookup":
        state["out"] = torch.empty(case["n"], case["len"], dtype=TORCH[case["out"]], device="cuda")
    if op == "lookup_grad":
        at = _batches(case)
        state["batch_ids"] = [state["ids"][a:b] for a, b in zip(at, at[1:])]
        state["batch_douts"] = [state["douts"][a:b] for a, b in zip(at, at[1:])]
    if op in ("clip", "adamw"):
        state["result"], state["passes"] = torch.zeros(1, device="cuda"), 0
        shapes = _shapes(case["params"])
        # no decay for the one-element rows (norm weights)
        state["decay"] = [DECAY if length > 1 else 0.0 for _, length in shapes]
        sizes = torch.tensor(_layout(R, shapes)[1], device="cuda")
        if op == "adamw":
            state["decay_of"] = torch.repeat_interleave(torch.tensor(state["decay"], device="cuda"), sizes)
    if own:
        import all_gather_tide_gb300 as tide

        if op in ("lookup", "lookup_grad"):
            shapes, p, _, _, _, _ = _table(case)
            state["group"], state["p"] = tide.Group(R, shapes), p
            state["rows"] = tide.pointer_table(list(state["shards"]))
            if op == "lookup_grad":
                state["workspace"] = state["group"].embedding_grad_workspace(p, case["n"])
        else:
            pieces = _pieces(R, shapes)
            kind = {"f32": tide.TIDE_F32, "bf16": tide.TIDE_BF16}[case.get("grads", "f32")]
            state["list"] = tide.TensorList([n for _, _, _, n in pieces], [kind] * len(pieces))
            names = ("grads",) if op == "clip" else ("master", "grads", "exp_avg", "exp_avg_sq", "shards")
            state["tables"] = [tide.pointer_table([state[k][d, o:o + n] for d, _, o, n in pieces]) for k in names]
            state["decays"] = tide.float_table([state["decay"][p] for _, p, _, _ in pieces])
    return state


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_lookup(st):
    st["group"].embedding(st["p"], st["rows"], st["ids"], st["out"], scale=st["case"]["scale"])
    return st["out"]


def _own_grad(st):
    st["group"].embedding_grad(st["p"], st["batch_ids"], st["batch_douts"], st["rows"], scale=st["case"]["scale"], accumulate=st["case"]["add"],
                               workspace=st["workspace"])
    return st["shards"]


def _bound(st):
    """The bound falls a little with every pass, so that gradients which the last pass clipped are over it
    again, as a training step's new ones are."""
    st["passes"] += 1
    return st["case"]["max_norm"] * 0.9999 ** (st["passes"] - 1)


def _own_clip(st):
    st["list"].clip_grad_norm(st["tables"][0], _bound(st), st["result"])
    return {"norm": st["result"], "grads": st["grads"]}


def _own_adamw(st):
    st["step"] += 1
    st["list"].adamw(*st["tables"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=st["decays"], step=st["step"], norm=st["norm"],
                     max_norm=st["case"]["max_norm"])
    return {k: st[k] for k in ("master", "exp_avg", "exp_avg_sq", "shards")}


def _plain_lookup(st):
    c, (_, _, m, s, o, _) = st["case"], _table(st["case"])
    table = st["shards"][:, o:o + s].unflatten(1, (m, c["len"]))
    ids = st["ids"].long()
    held = (ids >= 0) & (ids < c["rows"])
    t = torch.where(held, ids, 0)
    rows = table[t // m, t % m].float() * c["scale"]
    return torch.where(held[:, None], rows, 0.0).to(TORCH[c["out"]])


def _plain_grad(st):
    c, (_, _, m, s, o, _) = st["case"], _table(st["case"])
    R, length = c["R"], c["len"]
    ids = st["ids"].long()
    held = (ids >= 0) & (ids < c["rows"])
    # positions without a token go to a row of their own past the table
    t = torch.where(held, ids, R * m)
    total = torch.zeros(R * m + 1, length, device="cuda").index_add_(0, t, st["douts"].float() * c["scale"])
    part = st["shards"][:, o:o + s]
    total = total[:R * m].view(R, s)
    part.add_(total) if c["add"] else part.copy_(total)
    return st["shards"]


def _plain_clip(st):
    g = st["grads"]
    norm = g.float().square().sum().sqrt().reshape(1)
    factor = torch.clamp(_bound(st) / (norm + 1e-6), max=1.0)
    g.copy_(g.float() * factor)
    st["result"].copy_(norm)
    return {"norm": st["result"], "grads": g}


def _plain_adamw(st):
    st["step"] += 1
    p, m, v = st["master"], st["exp_avg"], st["exp_avg_sq"]
    g = st["grads"] * torch.clamp(st["case"]["max_norm"] / (st["norm"] + 1e-6), max=1.0)
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_(g * g * (1 - BETA2))
    c1, c2 = 1 - BETA1 ** st["step"], 1 - BETA2 ** st["step"]
    denom = v.sqrt() / math.sqrt(c2) + EPS
    p.mul_(1 - LR * st["decay_of"])
    p.sub_(m / denom * (LR / c1))
    st["shards"].copy_(p)
    return {k: st[k] for k in ("master", "exp_avg", "exp_avg_sq", "shards")}


_own = {"lookup": _own_lookup, "lookup_grad": _own_grad, "clip": _own_clip, "adamw": _own_adamw}
_plain = {"lookup": _plain_lookup, "lookup_grad": _plain_grad, "clip": _plain_clip, "adamw": _plain_adamw}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "lookup":
        shapes, p, m, s, o, _ = _table(case)
        # the whole table in row order, with one zero row at its end for positions without a token
        whole = torch.cat([x["shards"][d, o:o + s].view(m, case["len"]) for d in range(case["R"])])[:case["rows"]]
        whole = torch.cat([whole, torch.zeros_like(whole[:1])])
        ids = x["ids"].long()
        return whole[torch.where((ids < 0) | (ids >= case["rows"]), case["rows"], ids)].double() * case["scale"]
    if case["op"] == "lookup_grad":
        shapes, p, m, s, o, _ = _table(case)
        ids = x["ids"].long()
        keep = torch.nonzero((ids >= 0) & (ids < case["rows"])).flatten()
        whole = torch.zeros(case["R"] * m, case["len"], dtype=torch.float64, device="cuda")
        for at in keep.split(16384):
            whole.index_add_(0, ids[at], x["douts"][at].double())
        whole *= case["scale"]
        out = x["shards"].double()
        for d, piece in enumerate(whole.split(m)):
            out[d, o:o + s] = piece.flatten() + (out[d, o:o + s] if case["add"] else 0)
        return out
    if case["op"] == "clip":
        flat = x["grads"].flatten()
        total = sum(float(c.double().square().sum()) for c in flat.split(1 << 28))
        norm = math.sqrt(total)
        factor = min(1.0, case["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64), "grads": x["grads"].double() * factor}
    shapes = _shapes(case["params"])
    t = x["step"] + 1
    factor = min(1.0, case["max_norm"] / (float(x["norm"]) + 1e-6))
    g = x["grads"].double().mul_(factor)
    m = x["exp_avg"].double().mul_(BETA1).add_(g, alpha=1 - BETA1)
    v = x["exp_avg_sq"].double().mul_(BETA2).add_(g.square_(), alpha=1 - BETA2)
    p = x["master"].double()
    _, sizes, offsets, _ = _layout(case["R"], shapes)
    for o, s, (_, length) in zip(offsets, sizes, shapes):
        if length > 1:
            p[:, o:o + s] *= 1 - LR * DECAY
    p -= LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    return {"master": p, "exp_avg": m, "exp_avg_sq": v, "shards": p}


# ---- what a pass cannot do without -------------------------------------------------------------


def _distinct(case):
    """Rows expected among the case's tokens: sum over rows of 1 - (1 - share)^n, in blocks of rows."""
    n, rows, total = case["n"] * (1 - case["masked"]), case["rows"], 0.0
    span = math.log(rows + 1)
    k = 1
    while k <= rows:
        many = max(1, k // 64)  # rows of nearly the same share
        many = min(many, rows + 1 - k)
        share = math.log((k + many) / k) / span / many
        total += many * -math.expm1(n * math.log1p(-min(share, 1 - 1e-12)))
        k += many
    return total


def work(case):
    size = {"bf16": 2, "f32": 4, "int32": 4, "int64": 8}
    if case["op"] == "lookup":
        n, length = case["n"], case["len"]
        return {"bytes": n * size[case["ids"]] + _distinct(case) * length * 2 + n * length * size[case["out"]], "flops": n * length}
    if case["op"] == "lookup_grad":
        n, length = case["n"] * (1 - case["masked"]), case["len"]
        written = 2 * _distinct(case) * length if case["add"] else case["R"] * _table(case)[3]
        return {"bytes": case["n"] * size[case["ids"]] + n * length * size[case["dout"]] + written * 4, "flops": n * length}
    elements = sum(n for _, _, _, n in _pieces(case["R"], _shapes(case["params"])))
    if case["op"] == "clip":
        over = 1e-3 * math.sqrt(elements) > case["max_norm"]
        return {"bytes": elements * size[case["grads"]] * (3 if over else 1) + 4, "flops": elements * (3 if over else 2)}
    return {"bytes": elements * 30 + 4, "flops": elements * 16}
