"""Cases of the recurrent-layer operators: the short causal convolution and the
selective state space scan (prompts, and steps of one or a few tokens), and the
moves of state slots that prefix caching does between them.

Each case is one call on the buffers that a serving program holds: packed
ragged tokens, a pool of per-slot states, a slot table.  `run` returns the
outputs and the updated pools.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the convolution before the q, k, v of 32 heads of 128 (three times
        # 4096 channels), one long prompt
        dict(name="conv prompt 8192x12288", op="conv", dtype="bf16", rows=1, tokens=8192,
             channels=12288, width=4, slots=64, bias=False, views=False, draft=0),
        # a ragged batch of prompts, x a view of a wider projection
        dict(name="conv prompt ragged f32", op="conv", dtype="f32", rows=23, tokens=5003,
             channels=1000, width=3, slots=64, bias=True, views=True, draft=0),
        # a speculative step: 16 sequences, 8 drafted tokens each
        dict(name="conv step 16 rows x 8", op="conv", dtype="bf16", rows=16, tokens=128,
             channels=12288, width=4, slots=64, bias=False, views=False, draft=8),
        # one sequence decoding alone: a call's latency
        dict(name="conv step 1 row", op="conv", dtype="bf16", rows=1, tokens=1,
             channels=4096, width=4, slots=64, bias=True, views=False, draft=1),
        # one long prompt, z the other half of the input projection
        dict(name="scan prompt 8192x4096", op="scan", dtype="bf16", rows=1, tokens=8192,
             channels=4096, state=16, groups=1, slots=64, views=True, gate=True, draft=0),
        # a prefill pass of many prompts of all lengths
        dict(name="scan prompt ragged 16384", op="scan", dtype="bf16", rows=37, tokens=16384,
             channels=4096, state=16, groups=1, slots=64, views=True, gate=True, draft=0),
        # a narrow layer in fp32, odd sizes, a wider state shared by groups
        dict(name="scan prompt small f32", op="scan", dtype="f32", rows=3, tokens=333,
             channels=500, state=64, groups=2, slots=16, views=False, gate=False, draft=0),
        # a mixed decode batch: most rows one token, every eighth row 8 drafts
        dict(name="scan step 64 rows mixed", op="scan", dtype="bf16", rows=64, tokens=120,
             channels=4096, state=16, groups=1, slots=256, views=True, gate=True, draft=8),
        # one sequence decoding alone
        dict(name="scan step 1 row", op="scan", dtype="bf16", rows=1, tokens=1,
             channels=4096, state=16, groups=1, slots=64, views=True, gate=True, draft=1),
        # a large decode batch, one token a row, a wider state
        dict(name="scan step 256 rows", op="scan", dtype="bf16", rows=256, tokens=256,
             channels=4096, state=64, groups=8, slots=256, views=True, gate=True, draft=1),
        # a prefix hit: one checkpoint forked into a live slot in every layer
        dict(name="move fork 1 slot", op="move", layers=8, slots=64, channels=4096, state=16,
             width=4, moves=1, frees=0, chained=False),
        # compaction of a pool: live slots moved down, some of them into slots
        # that others leave in the same call, the rest freed
        dict(name="move compact 64 slots", op="move", layers=8, slots=256, channels=4096,
             state=16, width=4, moves=64, frees=16, chained=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv", "scan", "scan", "scan", "move"])
    if op == "move":
        slots = _log(rng, 8, 256)
        moves = rng.randint(1, max(1, slots // 4))
        return dict(op="move", layers=rng.randint(1, 8), slots=slots,
                    channels=rng.choice([1, 2, 4, 8, 16, 32]) * 128, state=rng.choice([16, 32]),
                    width=rng.choice([2, 3, 4]), moves=moves,
                    frees=rng.randint(0, max(0, slots // 8)), chained=rng.random() < 0.5)
    form = rng.choice(["prompt", "step"])
    rows = _log(rng, 1, 64) if form == "prompt" else _log(rng, 1, 256)
    if form == "prompt":
        draft = 0
        tokens = max(rows, _log(rng, 16, 8192)) | 1
    else:
        draft = rng.choice([1, 1, 2, 4, 8])
        tokens = _step_tokens(rows, draft)
    channels = rng.choice([1, 2, 3, 4, 6, 8, 16, 20, 28, 32]) * 128
    if rng.random() < 0.3:  # sizes that are no multiple of a vector
        channels = _log(rng, 33, 2000) | 1
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, tokens=tokens,
                channels=channels, slots=max(4, rows + rng.randint(0, 64)),
                views=rng.random() < 0.5, draft=draft)
    if op == "conv":
        case.update(width=rng.choice([2, 3, 4]), bias=rng.random() < 0.5)
    else:
        groups = rng.choice([1, 1, 2])
        case["channels"] += channels % groups
        state = rng.choice([16, 16, 32, 64, 128])
        if form == "prompt":  # no more work than the largest listed prompt
            state = min(state, 16 if tokens * channels > 2 ** 23 else 64 if tokens * channels > 2 ** 21 else 128)
        elif rows * channels > 2 ** 19:
            state = min(state, 32)
        case.update(state=state, groups=groups, gate=rng.random() < 0.7)
    return case


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
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def ints(a):
        return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()

    s = dict(case=case)
    if case["op"] == "move":
        nl, slots, d = case["layers"], case["slots"], case["channels"]
        s["states"] = normal(nl, slots, d, case["state"])
        s["taps"] = normal(nl, slots, case["width"] - 1, d, dtype=torch.bfloat16)
        order = rng.permutation(slots)
        m, f = case["moves"], case["frees"]
        if case["chained"]:  # every other move goes where the one after it leaves
            j = np.arange(m)
            src, dst = order[j // 2 * 3 + j % 2], order[j // 2 * 3 + j % 2 + 1]
        else:  # forks: a source may serve several
            dst = order[:m]
            src = rng.choice(order[m: max(m + 1, slots - f)], size=m)
        free = order[slots - f:] if f else order[:0]
        table = np.stack([np.concatenate([src, np.full(f, -1)]), np.concatenate([dst, free])])
        table = table[:, rng.permutation(m + f)]
        s["src"], s["dst"] = ints(table[0]), ints(table[1])
        return s
    dt = DTYPES[case["dtype"]]
    n, d, rows = case["tokens"], case["channels"], case["rows"]
    lens = _lengths(case, rng)
    s["lens"] = lens
    s["cu"] = ints(np.concatenate([[0], np.cumsum(lens)]))
    s["live"] = ints(np.nonzero(lens)[0])
    s["slots"] = ints(rng.permutation(case["slots"])[:rows])
    # a step keeps all of a plain row's token and 0..T of a drafted row's
    s["commit"] = ints(np.where(lens > 1, rng.integers(0, lens + 1), lens)) if case["draft"] > 1 else None
    if case["op"] == "conv":
        w = case["width"]
        wide = normal(n, 2 * d if case["views"] else d, dtype=dt)
        s["x"] = wide[:, :d]
        s["weight"] = normal(d, w, dtype=dt, std=1.0 / math.sqrt(w))
        s["bias"] = normal(d, dtype=dt, std=0.1) if case["bias"] else None
        s["pool"] = normal(case["slots"], w - 1, d, dtype=dt)
        return s
    st, gr = case["state"], case["groups"]
    s["x"] = normal(n, d, dtype=dt)
    rank = -(-d // 16)
    if case["views"]:  # B and C as the tail of one projection's row, z as the half of another's
        proj = normal(n, rank + 2 * gr * st, dtype=dt)
        s["B"] = proj[:, rank: rank + gr * st].unflatten(1, (gr, st))
        s["C"] = proj[:, rank + gr * st:].unflatten(1, (gr, st))
        z = normal(n, 2 * d, dtype=dt)[:, d:]
    else:
        s["B"], s["C"] = normal(n, gr, st, dtype=dt), normal(n, gr, st, dtype=dt)
        z = normal(n, d, dtype=dt)
    s["z"] = z if case["gate"] else None
    s["dt"] = normal(n, d, dtype=dt, std=0.5)
    step = torch.exp(uniform(d) * math.log(100.0) + math.log(1e-3))  # time steps of 0.001 .. 0.1
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, st + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(d, st, std=0.1))
    s["D"] = 1.0 + normal(d, std=0.1)
    s["pool"] = normal(case["slots"], d, st, std=0.1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    # the descriptors of its buffers, which a serving program builds once
    from recurrent_kda_state_gb300 import kda as K
    if case["op"] == "move":
        s["arrays"] = K.SlotArrays([t for pool in (s["states"], s["taps"]) for t in pool])
        s["work"] = K.move_workspace(s["arrays"], s["src"].numel()) if case["chained"] else None
        return s
    cu = None if case["draft"] == 1 else s["cu"]
    if case["op"] == "conv":
        s["batch"] = K.ConvBatch(s["x"], s["weight"], bias=s["bias"], cu_seqlens=cu, activation="silu")
        s["own_pool"] = K.ConvPool(s["pool"])
    else:
        s["batch"] = K.ScanBatch(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                 dt_bias=s["dt_bias"], cu_seqlens=cu, dt_softplus=True)
        s["own_pool"] = K.ScanPool(s["pool"])
        s["work"] = K.scan_workspace(s["batch"]) if not case["draft"] else None
    return s


def run(s):
    case = s["case"]
    if not own:
        return {"conv": _plain_conv, "scan": _plain_scan, "move": _plain_move}[case["op"]](s)
    from recurrent_kda_state_gb300 import kda as K
    if case["op"] == "move":
        K.kda_move_slots(s["arrays"], s["src"], s["dst"], workspace=s["work"])
        return s["states"], s["taps"]
    if case["op"] == "conv":
        if case["draft"]:
            K.kda_conv_step(s["batch"], s["own_pool"], s["slots"], commit_len=s["commit"])
        else:
            K.kda_conv_prefill(s["batch"], s["own_pool"], s["slots"])
    elif case["draft"]:
        K.kda_scan_step(s["batch"], s["own_pool"], s["slots"], commit_len=s["commit"])
    else:
        K.kda_scan_prefill(s["batch"], s["own_pool"], s["slots"], workspace=s["work"])
    return s["batch"].y, s["pool"]


def _rows(s):
    """Of each token: its row and its position in it; of each row: its first
    token and how many of its tokens the stored state takes in."""
    cu = s["cu"].long()
    t = torch.arange(s["case"]["tokens"], device="cuda")
    row = (t[:, None] >= cu[None, 1:]).sum(1)
    keep = s["commit"].long() if s["commit"] is not None else cu[1:] - cu[:-1]
    return cu, row, t - cu[row], keep


def _plain_conv(s):
    case = s["case"]
    w, n, dt = case["width"], case["tokens"], s["x"].dtype
    cu, row, pos, keep = _rows(s)
    slots = s["slots"].long()
    # every row's inputs after the w - 1 that its slot holds
    u = torch.cat([s["pool"][slots].flatten(0, 1), s["x"]]).float()
    tap = torch.arange(w, device="cuda")
    head = case["rows"] * (w - 1)
    at = pos[:, None] + tap  # row u[j] of [state; inputs]
    at = torch.where(at < w - 1, row[:, None] * (w - 1) + at, head + cu[row][:, None] + at - (w - 1))
    y = (u[at] * s["weight"].float().T).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = (y / (1 + torch.exp(-y))).to(dt)
    last = keep[:, None] + tap[None, : w - 1]
    r = torch.arange(case["rows"], device="cuda")[:, None]
    last = torch.where(last < w - 1, r * (w - 1) + last, head + cu[:-1, None] + last - (w - 1))
    s["pool"][slots] = u[last].to(dt)
    return y, s["pool"]


def _plain_scan(s):
    case = s["case"]
    n, d, gr, st = case["tokens"], case["channels"], case["groups"], case["state"]
    cu, row, pos, keep = _rows(s)
    slots = s["slots"].long()
    v = s["dt"].float() + s["dt_bias"]
    delta = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    x = s["x"].float()
    a = torch.exp(delta[:, :, None] * s["A"])
    b = (delta * x).view(n, gr, d // gr, 1) * s["B"].float()[:, :, None, :]
    b = b.view(n, d, st)
    # the stored state enters with a row's first token, and nothing passes it
    live = s["live"].long()
    first = cu[live]
    h0 = s["pool"][slots]
    b[first] += a[first] * h0[live]
    a[first] = 0
    # h_t = a_t h_{t-1} + b_t by doubling: after the pass of width k, b holds
    # the sum over the last 2k tokens and a the product of their decays
    k = 1
    while k < int(s["lens"].max()):
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    y = (b.view(n, gr, d // gr, st) * s["C"].float()[:, :, None, :]).sum(3).view(n, d)
    y = y + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1 + torch.exp(-z)))
    end = torch.where((keep > 0)[:, None, None], b[(cu[:-1] + keep - 1).clamp(min=0)], h0)
    s["pool"][slots] = end
    return y.to(s["x"].dtype), s["pool"]


def _plain_move(s):
    src, dst = s["src"].long(), s["dst"].long()
    taken = (src >= 0)[None, :, None, None]
    src = src.clamp(min=0)
    s["states"][:, dst] = torch.where(taken, s["states"][:, src], 0.0)
    s["taps"][:, dst] = torch.where(taken, s["taps"][:, src], 0.0)
    return s["states"], s["taps"]


def work(case):
    if case["op"] == "move":
        slot = case["layers"] * case["channels"] * (case["state"] * 4 + (case["width"] - 1) * 2)
        return {"bytes": slot * (2 * case["moves"] + case["frees"]), "flops": 0}
    n, d, rows = case["tokens"], case["channels"], case["rows"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "conv":
        w = case["width"]
        return {"bytes": es * (2 * n * d + 2 * rows * (w - 1) * d + d * (w + case["bias"])),
                "flops": n * d * (2 * w + 4)}
    st, gr = case["state"], case["groups"]
    return {"bytes": es * n * (d * (4 if case["gate"] else 3) + 2 * gr * st)
            + 4 * (2 * rows * d * st + d * st + 2 * d),
            "flops": n * d * (7 * st + 12)}


def exact(case, seed):
    """The definitions, token by token, in 64 bits."""
    s = _inputs(case, seed)
    if case["op"] == "move":
        out = []
        for t in (s["states"], s["taps"]):
            old, new = t.double(), t.double()
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                new[:, b] = old[:, a] if a >= 0 else 0.0
            out.append(new)
        return tuple(out)
    # rows by falling length, so that those with a k-th token come first
    order = np.argsort(-s["lens"], kind="stable")
    lens = s["lens"][order]
    first = s["cu"].cpu().numpy()[:-1][order]
    keep = s["commit"].cpu().numpy()[order] if s["commit"] is not None else lens
    slots = s["slots"].cpu().numpy()[order]
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int64)).cuda()  # noqa: E731
    pool = s["pool"].double()
    h = pool[dev(slots)]
    kept = h.clone()
    first_d, keep_d = dev(first), dev(keep)
    y = torch.zeros(case["tokens"], case["channels"], dtype=torch.float64, device="cuda")
    x = s["x"]
    for k in range(int(lens[0])):
        m = int((lens > k).sum())
        at = first_d[:m] + k
        if case["op"] == "conv":
            taps = torch.cat([h[:m], x[at][:, None].double()], 1)
            h[:m] = taps[:, 1:]
            out = torch.einsum("mwd,dw->md", taps, s["weight"].double())
            if s["bias"] is not None:
                out = out + s["bias"].double()
            y[at] = out * torch.sigmoid(out)
        else:
            delta = torch.nn.functional.softplus(s["dt"][at].double() + s["dt_bias"].double(), threshold=700.0)
            rep = case["channels"] // case["groups"]
            bt = s["B"][at].double().repeat_interleave(rep, 1)
            ct = s["C"][at].double().repeat_interleave(rep, 1)
            xt = x[at].double()
            h[:m] = torch.exp(delta[..., None] * s["A"].double()) * h[:m] + (delta * xt)[..., None] * bt
            out = (ct * h[:m]).sum(-1) + s["D"].double() * xt
            if s["z"] is not None:
                zt = s["z"][at].double()
                out = out * zt * torch.sigmoid(zt)
            y[at] = out
        kept = torch.where((keep_d > k).view(-1, 1, 1), h, kept)
    pool[dev(slots)] = kept
    return y, pool
