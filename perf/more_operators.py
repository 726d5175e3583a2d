"""Cases of the operators of a linear attention layer: linear attention with a
decay for each head (prompts, and steps of one or a few tokens), the norm of
queries and keys for each head with the position rotation, which comes before
it and before a KDA layer, and the gated norm of the outputs, which comes after.

Each case is one call on the buffers that a serving program holds: packed
ragged tokens, a pool of per-slot states, a slot table.  `run` returns the
outputs and the updated pool.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one long prompt, q, k and v the thirds of one projection
        dict(name="linear prompt 8192", op="linear", dtype="bf16", rows=1, tokens=8192, heads=32,
             qk_heads=32, d_k=128, d_v=128, fixed=False, views=True, slots=64, draft=0),
        # a prefill pass of many prompts of all lengths
        dict(name="linear prompt ragged 16384", op="linear", dtype="bf16", rows=37, tokens=16384,
             heads=32, qk_heads=32, d_k=128, d_v=128, fixed=False, views=False, slots=64, draft=0),
        # queries and keys shared by all heads, values of half the width
        dict(name="linear prompt shared 4096", op="linear", dtype="bf16", rows=4, tokens=4096,
             heads=64, qk_heads=1, d_k=128, d_v=64, fixed=False, views=True, slots=16, draft=0),
        # a narrow layer in fp32, odd lengths, one decay for every token
        dict(name="linear prompt small f32", op="linear", dtype="f32", rows=3, tokens=333, heads=6,
             qk_heads=6, d_k=64, d_v=32, fixed=True, views=False, slots=16, draft=0),
        # one sequence decoding alone: a call's latency
        dict(name="linear step 1 row", op="linear", dtype="bf16", rows=1, tokens=1, heads=32,
             qk_heads=32, d_k=128, d_v=128, fixed=True, views=True, slots=64, draft=1),
        # a mixed decode batch: most rows one token, every eighth row 8 drafts
        dict(name="linear step 64 rows mixed", op="linear", dtype="bf16", rows=64, tokens=120,
             heads=32, qk_heads=32, d_k=128, d_v=128, fixed=False, views=True, slots=256, draft=8),
        # a large decode batch, one token a row
        dict(name="linear step 256 rows", op="linear", dtype="bf16", rows=256, tokens=256, heads=32,
             qk_heads=32, d_k=128, d_v=128, fixed=False, views=True, slots=256, draft=1),
        # the queries and keys of a long prompt, all channels rotated
        dict(name="qk norm prompt 8192", op="qk", dtype="bf16", tokens=8192, q_heads=32, k_heads=32,
             dim=128, norm="rms", rot=128, pairs="halves", views=True),
        # a speculative step: 16 rows of 8 drafts, fewer key heads, half the channels rotated
        dict(name="qk norm 128 tokens", op="qk", dtype="bf16", tokens=128, q_heads=32, k_heads=4,
             dim=128, norm="rms", rot=64, pairs="neighbours", views=True),
        # the keys' length of a KDA layer, fp32, odd sizes, no rotation
        dict(name="qk norm odd f32", op="qk", dtype="f32", tokens=1001, q_heads=6, k_heads=6,
             dim=80, norm="l2", rot=0, pairs="halves", views=False),
        # the fp32 outputs of a KDA layer's prompt on their way to the output projection
        dict(name="gated norm prompt 8192", op="gate", dtype="f32", gate="bf16", tokens=8192,
             heads=32, dim=128, act="sigmoid", views=True),
        # the outputs of one decoding sequence
        dict(name="gated norm 1 token", op="gate", dtype="bf16", gate="bf16", tokens=1, heads=32,
             dim=128, act="silu", views=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "qk", "gate"])
    if op == "qk":
        dim = rng.choice([16, 32, 48, 64, 80, 96, 128, 128, 192, 256])
        if rng.random() < 0.2:  # sizes that are no multiple of a vector
            dim = 2 * rng.randint(3, 100)
        k_heads = rng.choice([1, 2, 3, 4, 8, 16, 32])
        q_heads = k_heads * rng.choice([1, 1, 2, 4, 8])
        tokens = _log(rng, 1, min(8192, 2 ** 25 // (dim * q_heads)))
        rot = rng.choice([0, dim, dim, dim // 4 * 2])
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), tokens=tokens, q_heads=q_heads,
                    k_heads=k_heads, dim=dim, norm=rng.choice(["rms", "rms", "l2", "none"]), rot=rot,
                    pairs=rng.choice(["halves", "neighbours"]), views=rng.random() < 0.5)
    if op == "gate":
        dim = rng.choice([16, 32, 64, 80, 128, 128, 256])
        if rng.random() < 0.2:
            dim = rng.randint(5, 200)
        heads = rng.choice([1, 2, 3, 6, 8, 16, 32, 64])
        x, gate = rng.choice([("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
        return dict(op=op, dtype=x, gate=gate, tokens=_log(rng, 1, min(8192, 2 ** 25 // (dim * heads))),
                    heads=heads, dim=dim, act=rng.choice(["sigmoid", "silu"]), views=rng.random() < 0.5)
    qk_heads = rng.choice([1, 2, 3, 4, 8, 16, 32])
    heads = qk_heads * rng.choice([1, 1, 1, 2, 4])
    form = rng.choice(["prompt", "step"])
    d_k, d_v = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (64, 128), (32, 32), (16, 64), (16, 16)])
    most = 2 ** 33 // (heads * d_k * d_v)  # no more work than the largest listed prompt
    if form == "prompt":
        rows, draft = _log(rng, 1, 64), 0
        tokens = min(max(rows, _log(rng, 16, 8192)), most) | 1
    else:
        draft = rng.choice([1, 1, 2, 4, 8])
        rows = min(_log(rng, 1, 256), max(1, 2 ** 27 // (heads * d_k * d_v)))
        tokens = _step_tokens(rows, draft)
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, tokens=tokens, heads=heads,
                qk_heads=qk_heads, d_k=d_k, d_v=d_v, fixed=rng.random() < 0.3, views=rng.random() < 0.5,
                slots=max(4, rows + rng.randint(0, 32)), draft=draft)


def _step_tokens(rows, draft):
    """A step's tokens: every eighth row has `draft` drafts, the others one."""
    if draft <= 1 or rows <= 16:
        return rows * max(1, draft)
    spec = -(-rows // 8)
    return spec * draft + rows - spec


def _lengths(case, rng):
    """The rows' lengths: they sum to `tokens` whatever the seed."""
    rows, tokens, draft = case["rows"], case["tokens"], case["draft"]
    if draft:
        if tokens == rows * draft:
            return np.full(rows, draft)
        lens = np.ones(rows, dtype=np.int64)
        lens[rng.permutation(rows)[: -(-rows // 8)]] = draft
        return lens
    # prompts: a few long ones, many short ones, and now and then an empty row
    share = np.exp(rng.standard_normal(rows))
    share[rng.random(rows) < 0.1] = 0.0
    share[0] = max(share[0], 0.5)
    lens = np.floor(share / share.sum() * tokens).astype(np.int64)
    lens[int(np.argmax(lens))] += tokens - lens.sum()
    return lens


def _inputs(case, seed):
    """The tensors and host lengths of a case, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    n = case["tokens"]

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def ints(a):
        return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()

    def heads(views, widths, dtype):
        """Tensors [n][H][d], parts of the rows of one projection or of their own."""
        if not views:
            return [normal(n, h, d, dtype=dtype) for h, d in widths]
        wide = normal(n, sum(h * d for h, d in widths), dtype=dtype)
        parts = wide.split([h * d for h, d in widths], 1)
        return [p.unflatten(1, w) for p, w in zip(parts, widths)]

    s = dict(case=case)
    if case["op"] == "qk":
        d, rot = case["dim"], case["rot"]
        hq, hk = case["q_heads"], case["k_heads"]
        if case["views"]:  # the values stand behind them in the rows
            s["q"], s["k"], _ = heads(True, [(hq, d), (hk, d), (hk, d)], dt)
        else:
            s["q"], s["k"] = heads(False, [(hq, d), (hk, d)], dt)
        plain = case["norm"] != "rms"
        s["wq"] = None if plain else (1.0 + normal(d, std=0.2)).to(dt)
        s["wk"] = None if plain else (1.0 + normal(d, std=0.2)).to(dt)
        s["table"] = s["pos"] = None
        if rot:
            span = 4 * n + 64
            freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
            angle = torch.arange(span, device="cuda", dtype=torch.float64)[:, None] * freq
            s["table"] = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
            s["pos"] = ints(rng.integers(0, span, n))
        return s
    if case["op"] == "gate":
        d, h = case["dim"], case["heads"]
        s["x"] = normal(n, h, d, dtype=dt)
        s["weight"] = (1.0 + normal(d, std=0.2)).to(DTYPES[case["gate"]])
        s["gate"] = heads(case["views"], [(h, d), (h, d)], DTYPES[case["gate"]])[0]
        return s
    h, hk, dk, dv, rows = case["heads"], case["qk_heads"], case["d_k"], case["d_v"], case["rows"]
    lens = _lengths(case, rng)
    s["lens"] = lens
    s["cu"] = ints(np.concatenate([[0], np.cumsum(lens)]))
    s["slots"] = ints(rng.permutation(case["slots"])[:rows])
    # a step keeps all of a plain row's token and 0..T of a drafted row's
    keep = np.where(lens > 1, rng.integers(0, lens + 1), lens) if case["draft"] > 1 else lens
    s["keep"] = keep
    s["commit"] = ints(keep) if case["draft"] > 1 else None
    s["q"], s["k"], s["v"] = heads(case["views"], [(hk, dk), (hk, dk), (h, dv)], dt)
    # decays from a horizon of a few tokens to one of thousands
    rate = torch.exp(torch.rand(h, generator=gen, device="cuda") * math.log(1000.0) + math.log(3e-4))
    if case["fixed"]:
        s["g"] = -rate
    else:
        u = normal(n, h)
        s["g"] = -rate * (torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs())))
    s["scale"] = dk ** -0.5
    s["pool"] = normal(case["slots"], h, dv, dk)
    # the plain form's tiles of 64 tokens (a step: of its drafts)
    s["tile"] = case["draft"] or 64
    count = -(-lens // s["tile"])
    row = np.repeat(np.arange(rows), count)
    nth = np.arange(len(row)) - np.repeat(np.cumsum(count) - count, count)
    first = np.concatenate([[0], np.cumsum(lens)])[row] + nth * s["tile"]
    size = np.minimum(lens[row] - nth * s["tile"], s["tile"])
    last = nth == count[row] - 1
    s["tiles"] = [torch.from_numpy(np.asarray(a, dtype=np.int64)).cuda() for a in
                  (row, first, size, np.where(last, keep[row] - nth * s["tile"], size))]
    s["ends"] = torch.from_numpy(np.nonzero(last)[0]).cuda()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    # the descriptors of its buffers, which a serving program builds once
    from recurrent_kda_state_gb300 import kda as K
    if case["op"] == "qk":
        s["batch"] = K.QKBatch(s["q"], s["k"], q_weight=s["wq"], k_weight=s["wk"],
                               norm=None if case["norm"] == "none" else case["norm"], eps=1e-6,
                               cos_sin=s["table"], positions=s["pos"],
                               interleaved=case["pairs"] == "neighbours", q_scale=case["dim"] ** -0.5)
    elif case["op"] == "gate":
        s["batch"] = K.GateBatch(s["x"], s["gate"], weight=s["weight"], activation=case["act"], eps=1e-6)
    else:
        cu = None if case["draft"] == 1 else s["cu"]
        s["batch"] = K.LinearBatch(s["q"], s["k"], s["v"], s["g"], cu_seqlens=cu, scale=s["scale"])
        s["own_pool"] = K.StatePool(s["pool"])
        s["work"] = None if case["draft"] else K.linear_workspace(s["batch"])
    return s


def run(s):
    case = s["case"]
    if not own:
        return {"linear": _plain_linear, "qk": _plain_qk, "gate": _plain_gate}[case["op"]](s)
    from recurrent_kda_state_gb300 import kda as K
    if case["op"] == "qk":
        K.kda_qk_norm(s["batch"])
        return s["batch"].q_out, s["batch"].k_out
    if case["op"] == "gate":
        K.kda_gated_norm(s["batch"])
        return s["batch"].y
    if case["draft"]:
        K.kda_linear_step(s["batch"], s["own_pool"], s["slots"], commit_len=s["commit"])
    else:
        K.kda_linear_prefill(s["batch"], s["own_pool"], s["slots"], workspace=s["work"])
    return s["batch"].o, s["pool"]


def _plain_linear(s):
    """Tiles of a row's tokens: products within a tile, and the states between
    tiles from a product with the decays between them."""
    case = s["case"]
    n, h, hk = case["tokens"], case["heads"], case["qk_heads"]
    row, first, size, kept = s["tiles"]
    at = torch.arange(s["tile"], device="cuda")
    live = at < size[:, None]
    token = torch.where(live, first[:, None] + at, 0)

    def tiles(x):  # [tile][head][token][d], zeros behind a row's end
        x = torch.where(live[..., None, None], x[token].float(), 0.0)
        return x.transpose(1, 2).repeat_interleave(h // x.shape[2], 1)

    q, k, v = tiles(s["q"]), tiles(s["k"]), tiles(s["v"])
    g = s["g"].double().expand(n, h)[token]
    g = torch.where(live[..., None], g, 0.0).cumsum(1).transpose(1, 2)  # [tile][head][token]
    seen = at[:, None] >= at
    decay = torch.exp(torch.where(seen, g[..., :, None] - g[..., None, :], -math.inf)).float()
    # what a tile adds to the state after its first `kept` tokens, and what is left of the state before
    end = g.gather(2, (kept - 1).clamp(min=0)[:, None, None].expand(-1, h, 1))
    end = torch.where((kept > 0)[:, None, None], end, 0.0)
    left = torch.where(at < kept[:, None, None], end - g, -math.inf)
    added = v.transpose(2, 3) @ (k * torch.exp(left).float()[..., None])  # [tile][head][d_v][d_k]
    # the state before each tile: the slot's and the earlier tiles' of the row
    total = torch.cat([torch.zeros_like(end[:1]), end.cumsum(0)])[..., 0].T  # [head][tile + 1]
    start = torch.searchsorted(row, row)
    old = s["pool"][s["slots"].long()]
    tile = torch.arange(len(row), device="cuda")
    earlier = (row[:, None] == row) & (tile[:, None] > tile)
    between = torch.exp(torch.where(earlier, total[:, :-1, None] - total[:, None, 1:], -math.inf)).float()
    before = (between @ added.transpose(0, 1).flatten(2)).unflatten(2, added.shape[2:]).transpose(0, 1)
    whole = torch.exp(total[:, :-1] - total[:, start]).float().T
    before = before + whole[..., None, None] * old[row]
    o = ((q @ k.transpose(2, 3)) * decay) @ v + torch.exp(g).float()[..., None] * (q @ before.transpose(2, 3))
    o = (o * s["scale"]).transpose(1, 2).flatten(0, 1)
    out = torch.empty(n, h, case["d_v"], dtype=s["v"].dtype, device="cuda")
    out[token[live]] = o[live.flatten()].to(out.dtype)
    e = s["ends"]
    s["pool"][s["slots"].long()[row[e]]] = added[e] + torch.exp(end[e]).float()[..., None] * before[e]
    return out, s["pool"]


def _plain_qk(s):
    case = s["case"]
    rot, d = case["rot"], case["dim"]

    def one(x, weight, scale):
        y = x.float()
        if case["norm"] != "none":
            total = (y * y).sum(2, keepdim=True)
            y = y / torch.sqrt((total / d if case["norm"] == "rms" else total) + 1e-6)
        if weight is not None:
            y = y * weight.float()
        if rot:
            turn = s["table"][s["pos"].long()][:, None]
            cos, sin = turn[..., : rot // 2], turn[..., rot // 2:]
            if case["pairs"] == "halves":
                a, b = y[..., : rot // 2], y[..., rot // 2: rot]
                y = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], 2)
            else:
                a, b = y[..., 0:rot:2], y[..., 1:rot:2]
                turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
                y = torch.cat([turned, y[..., rot:]], 2)
        return (y * scale).to(x.dtype)

    return one(s["q"], s["wq"], d ** -0.5), one(s["k"], s["wk"], 1.0)


def _plain_gate(s):
    x, gate = s["x"].float(), s["gate"].float()
    y = x / torch.sqrt((x * x).sum(2, keepdim=True) / s["case"]["dim"] + 1e-6) * s["weight"].float()
    act = 1 / (1 + torch.exp(-gate))
    if s["case"]["act"] == "silu":
        act = act * gate
    return (y * act).to(s["gate"].dtype)


def work(case):
    n = case["tokens"]
    size = {"bf16": 2, "f32": 4}
    es = size[case["dtype"]]
    if case["op"] == "qk":
        values = n * (case["q_heads"] + case["k_heads"]) * case["dim"]
        table = n * 4 * (case["rot"] + 1) if case["rot"] else 0
        weights = 2 * case["dim"] * es if case["norm"] == "rms" else 0
        return {"bytes": 2 * values * es + table + weights, "flops": 8 * values}
    if case["op"] == "gate":
        values, gs = n * case["heads"] * case["dim"], size[case["gate"]]
        return {"bytes": values * (es + 2 * gs) + case["dim"] * gs, "flops": 10 * values}
    h, hk, dk, dv, rows = case["heads"], case["qk_heads"], case["d_k"], case["d_v"], case["rows"]
    return {"bytes": n * es * (2 * hk * dk + 2 * h * dv) + 4 * h * (1 if case["fixed"] else n)
            + 8 * rows * h * dk * dv,
            "flops": 4 * n * h * dk * dv}


def exact(case, seed):
    """The definitions in 64 bits, the recurrence token by token."""
    s = _inputs(case, seed)
    d64 = torch.float64
    if case["op"] == "qk":
        d, rot = case["dim"], case["rot"]
        outs = []
        for x, w, scale in ((s["q"], s["wq"], d ** -0.5), (s["k"], s["wk"], 1.0)):
            y = x.to(d64)
            if case["norm"] == "rms":
                y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6)
            elif case["norm"] == "l2":
                y = y * torch.rsqrt(y.pow(2).sum(-1, keepdim=True) + 1e-6)
            if w is not None:
                y = y * w.to(d64)
            if rot:
                row = s["table"].to(d64)[s["pos"].long()]
                turn = torch.complex(row[:, : rot // 2], row[:, rot // 2:])[:, None]
                part = y[..., :rot]
                if case["pairs"] == "halves":
                    part = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
                else:
                    part = part.unflatten(-1, (rot // 2, 2))
                part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
                if case["pairs"] == "halves":
                    part = part.transpose(-1, -2)
                y = torch.cat([part.flatten(-2), y[..., rot:]], -1)
            outs.append(y * scale)
        return tuple(outs)
    if case["op"] == "gate":
        x, gate = s["x"].to(d64), s["gate"].to(d64)
        y = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * s["weight"].to(d64)
        return y * (torch.sigmoid(gate) if case["act"] == "sigmoid" else torch.nn.functional.silu(gate))
    # rows by falling length, so that those with a k-th token come first
    order = np.argsort(-s["lens"], kind="stable")
    lens, keep = s["lens"][order], s["keep"][order]
    begin = np.concatenate([[0], np.cumsum(s["lens"])])[:-1][order]
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int64)).cuda()  # noqa: E731
    slots = s["slots"].long()[dev(order)]
    pool = s["pool"].to(d64)
    state = pool[slots]
    kept = state.clone()
    begin_d, keep_d = dev(begin), dev(keep)
    h, rep = case["heads"], case["heads"] // case["qk_heads"]
    o = torch.zeros(case["tokens"], h, case["d_v"], dtype=d64, device="cuda")
    g = s["g"].to(d64)
    for t in range(int(lens[0])):
        m = int((lens > t).sum())
        at = begin_d[:m] + t
        a = torch.exp(g if case["fixed"] else g[at]).expand(m, h)[..., None, None]
        kt = s["k"][at].to(d64).repeat_interleave(rep, 1)
        qt = s["q"][at].to(d64).repeat_interleave(rep, 1)
        state[:m].mul_(a).add_(s["v"][at].to(d64)[..., None] * kt[..., None, :])
        o[at] = s["scale"] * (state[:m] @ qt[..., None])[..., 0]
        if case["draft"] > 1:
            kept[:m] = torch.where((keep_d[:m] > t).view(-1, 1, 1, 1), state[:m], kept[:m])
    pool[slots] = kept if case["draft"] > 1 else state
    return o, pool
