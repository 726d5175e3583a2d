"""Linear attention and the head norms against their fp64 definitions."""
import numpy as np
import pytest
import torch

import linear_ref
from recurrent_kda_state_gb300 import kda as K
from recurrent_kda_state_gb300._build import build_library

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_library()
    K.kda_get_device_error()
    yield
    assert K.kda_get_device_error() == 0


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(rng, n, shape, dt, view=0, std=1.0):
    """[n][*shape] on the device; view: the tail of wider rows, off by so many elements."""
    size = int(np.prod(shape))
    wide = torch.from_numpy(rng.standard_normal((n, size + view)) * std).to("cuda", DT[dt])
    return wide[:, view:].unflatten(1, shape)


def within(got, want, tol, what):
    bad = ~(np.abs(f64(got) - want) <= tol)
    assert not bad.any(), "%s: %d of %d values out of bounds, first %s, worst %.2f times its bound" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[:4].tolist(),
        np.nanmax(np.abs(f64(got) - want) / np.maximum(tol, 1e-300)))


def cumulate(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def decays(rng, n, H, kind):
    """Log decays [n][H]: from a horizon of a token to one of thousands by head; or
    strong ones; or with tokens that forget everything."""
    rate = np.exp(np.linspace(np.log(1e-4), np.log(2.0), H)) if H > 1 else np.array([0.05])
    g = -rate * rng.exponential(1.0, (n, H))
    if kind == "strong":
        g = g * 40
    if kind == "forget":
        g[rng.random((n, H)) < 0.05] = -np.inf
    if kind == "none":
        g[:] = 0.0
    return g


def linear_case(seed, dt, lens, H, dk, dv, Hk=None, kind="mild", fixed=False, view=0, step=False,
                commit=None, every=0, max_ckpt=0, start=None, workspace=True, extra=3, scale=0.7):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    n, B, Hk = int(lens.sum()), len(lens), Hk or H
    P = B * (1 + max_ckpt) + extra
    q = rows(rng, n + 3, (Hk, dk), dt, view)[:n]
    k = rows(rng, n + 3, (Hk, dk), dt, view, dk ** -0.5)[:n]
    v = rows(rng, n + 3, (H, dv), dt, view)[:n]
    g = decays(rng, 1 if fixed else n, H, kind)
    if fixed:
        g = torch.from_numpy(g[0]).float().cuda()
    else:  # rows with a stride where the others have one
        g = torch.from_numpy(np.concatenate([g, g], 1)).float().cuda()[:, H:] if view else (
            torch.from_numpy(g).float().cuda())
    data = torch.from_numpy(rng.standard_normal((P, H, dv, dk))).float().cuda()
    ids = rng.permutation(P)
    slots = ids[:B]
    ckpt = None
    if max_ckpt:
        ckpt = ids[B:B + B * max_ckpt].reshape(B, max_ckpt).copy()
        ckpt[0, 0] = -1
    cu = cumulate(lens)
    tensor = dt == "bf16" and min(dk, dv) >= 64 and not step
    want, tol, pool, pool_tol = linear_ref.linear(
        f64(q), f64(k), f64(v), np.broadcast_to(f64(g), (n, H)), cu, f64(data), slots, scale, dt, tensor,
        commit, ckpt, every, start)
    single = step and (lens == 1).all()
    wide = torch.full((n + 2, H * dv + view), 7.0, dtype=DT[dt], device="cuda")
    batch = K.LinearBatch(q, k, v, g, None if single else i32(cu), scale,
                          wide[:n, view:].unflatten(1, (H, dv)))
    states = K.StatePool(data)
    if step:
        K.kda_linear_step(batch, states, i32(slots), None if commit is None else i32(commit))
    else:
        K.kda_linear_prefill(batch, states, i32(slots), every, None if ckpt is None else i32(ckpt),
                             None if start is None else i32(start),
                             K.linear_workspace(batch) if workspace else None)
    within(batch.o, want, tol, "o")
    within(states.data, pool, pool_tol, "states")
    assert (wide[n:] == 7).all() and (wide[:, :view] == 7).all()
    return batch, states


LENS = [[1], [2, 0, 1, 3], [63, 64, 65, 0, 0, 17], [130, 1, 517]]
DIMS = [(128, 128), (64, 64), (128, 64), (64, 128), (16, 16), (32, 32), (16, 64), (32, 128), (128, 16)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_prefill(dt, dk, dv):
    for j, lens in enumerate(LENS):
        linear_case(j, dt, lens, 2, dk, dv)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("workspace", [True, False])
def test_prefill_long(dt, workspace):
    linear_case(10, dt, [3000], 3, 64, 64, workspace=workspace)
    linear_case(11, dt, [7, 1900, 0, 450, 64], 2, 128, 128, workspace=workspace)


@pytest.mark.parametrize("dt,lens,H,d", [("bf16", [2048], 32, 64), ("bf16", [1500, 1100], 16, 128),
                                         ("bf16", [700, 9, 400, 300, 64, 500], 24, 64), ("f32", [1500], 16, 32)])
def test_prefill_fills_the_machine(dt, lens, H, d):
    """Parts of all heads on every SM at once, the results the same each time."""
    a, sa = linear_case(19, dt, lens, H, d, d)
    for _ in range(3):
        b, sb = linear_case(19, dt, lens, H, d, d)
        assert torch.equal(a.o, b.o) and torch.equal(sa.data, sb.data)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["strong", "forget", "none"])
def test_prefill_decays(dt, kind):
    linear_case(12, dt, [700, 65], 4, 64, 128, kind=kind)
    linear_case(13, dt, [300], 1, 128, 64, kind=kind, fixed=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("view", [1, 3, 8])
def test_prefill_views_and_shared_heads(dt, view):
    linear_case(14, dt, [100, 33], 6, 64, 64, Hk=2, view=view)
    linear_case(15, dt, [100, 33], 5, 16, 32, Hk=1, view=view, fixed=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("start", [None, [0, 5, 64, 1000]])
@pytest.mark.parametrize("every,lens", [(64, [200, 3, 64, 129]), (128, [2000, 300, 0, 100])])
def test_prefill_checkpoints(dt, start, every, lens):
    linear_case(16, dt, lens, 2, 64, 64, every=every, max_ckpt=3, start=start)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("view", [0, 3, 8])
@pytest.mark.parametrize("lens,H,Hk,kind", [([1, 70, 0, 64, 300], 4, 1, "mild"), ([2, 1900], 6, 3, "forget"),
                                            ([517], 2, 1, "strong"), ([1500, 300, 63, 129], 32, 2, "mild")])
def test_prefill_shared_keys_and_narrow_values(dk, view, lens, H, Hk, kind):
    linear_case(41, "bf16", lens, H, dk, 64, Hk=Hk, view=view, kind=kind, every=64, max_ckpt=3, start=[5] * len(lens))
    linear_case(42, "bf16", lens, H, dk, 64, Hk=Hk, view=view, kind=kind, workspace=False, fixed=True)


def test_prefill_many_segments():
    lens = np.random.default_rng(17).integers(0, 9, 1500)
    linear_case(17, "bf16", lens, 1, 64, 64)
    linear_case(18, "f32", lens, 1, 16, 16)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_step(dt, dk, dv):
    linear_case(20, dt, [1] * 5, 3, dk, dv, step=True)
    linear_case(21, dt, [8, 1, 0, 3, 8, 40], 2, dk, dv, step=True, commit=[0, 1, 0, 2, 8, 17])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_variants(dt):
    linear_case(22, dt, [1] * 200, 2, 64, 64, step=True, fixed=True)
    linear_case(23, dt, [4, 1, 2], 6, 128, 128, Hk=2, step=True, view=3, kind="forget")
    linear_case(24, dt, [1] * 3, 32, 128, 128, step=True, kind="strong", commit=[1, 0, 1])
    linear_case(25, dt, [5] * 64, 8, 128, 128, step=True, commit=[3] * 64)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_steps_follow_a_prompt(dt):
    """A prompt and then steps, with rejected drafts between, are one longer prompt."""
    rng = np.random.default_rng(30)
    H, d, n = 2, 64, 150
    q, k, v = (rows(rng, n, (H, d), dt, std=s) for s in (1, 0.125, 1))
    g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
    data = np.zeros((2, H, d, d))
    want, tol, pool, pool_tol = linear_ref.linear(f64(q), f64(k), f64(v), f64(g), [0, n], data, [1],
                                                  out=dt, rounded_state=dt == "bf16")
    states = K.StatePool.zeros(2, H, d)
    a = K.LinearBatch(q[:100], k[:100], v[:100], g[:100], i32([0, 100]))
    K.kda_linear_prefill(a, states, i32([1]))
    b = K.LinearBatch(q[100:108], k[100:108], v[100:108], g[100:108], i32([0, 8]))
    K.kda_linear_step(b, states, i32([1]), i32([3]))   # three of eight drafts accepted
    c = K.LinearBatch(q[103:], k[103:], v[103:], g[103:], i32([0, n - 103]))
    K.kda_linear_step(c, states, i32([1]))
    within(torch.cat([a.o, b.o[:3], c.o]), want, tol, "o")
    within(states.data, pool, pool_tol, "states")


MARK = 1e30  # no output's value


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bad_tables_skip_their_rows(dt):
    """A slot, a segment or a count that is out of range: that row is left, its bit set."""
    rng = np.random.default_rng(31)
    H, d, n = 2, 64, 70
    q, k, v = (rows(rng, n, (H, d), dt) for _ in range(3))
    g = torch.zeros(H, device="cuda")

    def call(cu, slots, commit=None, step=False):
        o = torch.full((n, H, d), MARK, dtype=DT[dt], device="cuda")
        states = K.StatePool(torch.full((3, H, d, d), 0.5, device="cuda"))
        b = K.LinearBatch(q, k, v, g, i32(cu), o=o)
        if step:
            K.kda_linear_step(b, states, i32(slots), None if commit is None else i32(commit))
        else:
            K.kda_linear_prefill(b, states, i32(slots), workspace=K.linear_workspace(b))
        return o, states.data, K.kda_get_device_error()
    for step in (False, True):
        good, kept, bits = call([0, 65, 70], [0, 2], step=step)
        assert bits == 0 and (kept[1] == 0.5).all() and not (good == good.new_tensor(MARK)).any()
        for bad in (3, -1, 2 ** 31 - 1):
            o, s, bits = call([0, 65, 70], [0, bad], step=step)
            assert bits == K.KDA_DERR_SLOT
            assert torch.equal(o[:65], good[:65]) and (o[65:] == o.new_tensor(MARK)).all()
            assert torch.equal(s[0], kept[0]) and (s[1:] == 0.5).all()
        for cu in ([0, 65, 71], [0, 65, 64], [-5, 65, 60]):
            _, s, bits = call(cu, [0, 2], step=step)
            assert bits == K.KDA_DERR_SEGMENT and (s[1:] == 0.5).all()
    for commit in ([66, 1], [-1, 1]):
        o, s, bits = call([0, 65, 70], [0, 2], commit, step=True)
        assert bits == K.KDA_DERR_ACCEPT and (s[:2] == 0.5).all() and (o[:65] == o.new_tensor(MARK)).all()


def test_states_past_32_bits():
    """The last slot of a pool of more than 2^31 floats."""
    H, d = 32, 128
    P = 2 ** 31 // (H * d * d) + 4
    data = torch.empty(P, H, d, d, device="cuda")
    data[-1] = 0
    rng = np.random.default_rng(32)
    q, k, v = (rows(rng, 70, (H, d), "bf16") for _ in range(3))
    g = torch.full((H,), -0.1, device="cuda")
    small = K.StatePool.zeros(1, H, d)
    a, b = (K.LinearBatch(q, k, v, g, i32([0, 70])) for _ in range(2))
    K.kda_linear_prefill(a, K.StatePool(data), i32([P - 1]))
    K.kda_linear_prefill(b, small, i32([0]))
    assert torch.equal(a.o, b.o) and torch.equal(data[-1], small.data[0])
    K.kda_linear_step(a, K.StatePool(data), i32([P - 1]))
    K.kda_linear_step(b, small, i32([0]))
    assert torch.equal(a.o, b.o) and torch.equal(data[-1], small.data[0])


@pytest.mark.parametrize("dt,n", [("bf16", 2000), ("f32", 700)])
def test_same_bits_on_any_stream_and_in_a_graph(dt, n):
    rng = np.random.default_rng(33)
    H, d = 4, 64
    q, k, v = (rows(rng, n, (H, d), dt) for _ in range(3))
    g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
    batch = K.LinearBatch(q, k, v, g, i32([0, n - 90, n]))
    first = torch.from_numpy(rng.standard_normal((3, H, d, d))).float().cuda()
    slots, commit, work = i32([2, 0]), i32([5, 90]), K.linear_workspace(batch)
    states = K.StatePool(first.clone())

    def once(stream=None):
        K.kda_linear_prefill(batch, states, slots, workspace=work, stream=stream)
        K.kda_linear_step(batch, states, slots, commit, stream=stream)
    once()
    o, s = batch.o.clone(), states.data.clone()
    side = torch.cuda.Stream()
    states.data.copy_(first)
    side.wait_stream(torch.cuda.current_stream())
    once(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, batch.o) and torch.equal(s, states.data)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for _ in range(2):
        states.data.copy_(first)
        batch.o.zero_()
        graph.replay()
        assert torch.equal(o, batch.o) and torch.equal(s, states.data)


def test_two_streams_at_once():
    """Batches with pools and workspaces of their own, on two streams together."""
    rng = np.random.default_rng(34)
    H, d, n = 8, 128, 1500
    work = []
    for _ in range(2):
        q, k, v = (rows(rng, n, (H, d), "bf16") for _ in range(3))
        g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
        b = K.LinearBatch(q, k, v, g, i32([0, 1000, n]))
        work.append((b, K.StatePool.zeros(2, H, d), K.linear_workspace(b)))
    slots, streams = i32([1, 0]), [torch.cuda.Stream() for _ in range(2)]
    want = []
    for b, pool, ws in work:
        K.kda_linear_prefill(b, pool, slots, workspace=ws)
        want.append((b.o.clone(), pool.data.clone()))
    for _ in range(5):
        for b, pool, ws in work:
            b.o.zero_()
            pool.data.zero_()
        torch.cuda.synchronize()
        for (b, pool, ws), st in zip(work, streams):
            K.kda_linear_prefill(b, pool, slots, workspace=ws, stream=st)
        torch.cuda.synchronize()
        for (b, pool, ws), (o, states) in zip(work, want):
            assert torch.equal(b.o, o) and torch.equal(pool.data, states)


@pytest.mark.parametrize("workspace", [True, False])
def test_bounded_waits(workspace):
    """A wait that gives up is reported, slots stay as they are, and the next call is
    right."""
    rng = np.random.default_rng(35)
    H, d, n = 2, 64, 900
    q, k, v = (rows(rng, n, (H, d), "bf16") for _ in range(3))
    batch = K.LinearBatch(q, k, v, torch.full((H,), -0.01, device="cuda"), i32([0, n]))
    states = K.StatePool(torch.full((2, H, d, d), 0.5, device="cuda"))
    ws = K.linear_workspace(batch) if workspace else None
    K.kda_set_wait_limit(0)
    try:
        K.kda_linear_prefill(batch, states, i32([1]), workspace=ws)
        assert K.kda_get_device_error() == K.KDA_DERR_TIMEOUT
    finally:
        K.kda_set_wait_limit(-1)
    assert (states.data == 0.5).all()
    K.kda_linear_prefill(batch, states, i32([1]), workspace=ws)
    o, states_1 = batch.o.clone(), states.data.clone()
    states.data.fill_(0.5)
    K.kda_linear_prefill(batch, states, i32([1]), workspace=ws)
    assert torch.equal(o, batch.o) and torch.equal(states.data, states_1)


def test_other_sequences_values_stay_out():
    """A chunk's rows behind a segment's end are its neighbour's: NaN there, and in
    tokens of no segment, reach nothing."""
    rng = np.random.default_rng(36)
    H, d, n = 2, 64, 300
    for dt in ("bf16", "f32"):
        q, k, v = (rows(rng, n, (H, d), dt) for _ in range(3))
        g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
        cu = [0, 70, 200]
        clean = K.LinearBatch(q.clone(), k.clone(), v.clone(), g.clone(), i32(cu))
        for t in (q, k, v, g):
            t[70:] = float("nan")
        dirty = K.LinearBatch(q, k, v, g, i32(cu))
        got = []
        for b in (clean, dirty):
            pool = K.StatePool.zeros(2, H, d)
            K.kda_linear_prefill(b, pool, i32([1, 0]))
            got.append((b.o[:70].clone(), pool.data[1].clone()))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert got[0][0].isfinite().all()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dt,dk,dv", [("bf16", 128, 64), ("bf16", 64, 128), ("bf16", 128, 32), ("f32", 64, 64)])
def test_tokens_behind_the_last_sequence(dt, dk, dv, workspace):
    """A padded batch: what lies behind the last segment is not read into anything, and
    its outputs stay as they were; with room for more segments, empty ones at the end."""
    rng = np.random.default_rng(38)
    H, n, last = 4, 1100, 1000
    q, v = rows(rng, n, (H, dk), dt), rows(rng, n, (H, dv), dt)
    k = rows(rng, n, (H, dk), dt, std=dk ** -0.5)
    g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
    first = torch.from_numpy(rng.standard_normal((5, H, dv, dk))).float().cuda()

    def call(cu, slots, step):
        b = K.LinearBatch(q, k, v, g, i32(cu), o=torch.full((n, H, dv), MARK, dtype=DT[dt], device="cuda"))
        pool = K.StatePool(first.clone())
        if step:
            K.kda_linear_step(b, pool, i32(slots))
        else:
            K.kda_linear_prefill(b, pool, i32(slots), workspace=K.linear_workspace(b) if workspace else None)
        return b.o, pool.data
    for step in (False, True):
        tensor = dt == "bf16" and dv >= 64 and not step
        ref = linear_ref.linear(f64(q[:last]), f64(k[:last]), f64(v[:last]), f64(g[:last]), [0, 930, last],
                                f64(first), [3, 1], 1.0, dt, tensor)
        want, states = call([0, 930, last], [3, 1], step)
        for t in (q, k, v, g):
            t[last:] = float("nan")
        got, states_2 = call([0, 930, last], [3, 1], step)
        assert torch.equal(got, want) and torch.equal(states, states_2) and got[:last].isfinite().all()
        assert (got[last:] == got.new_tensor(MARK)).all() and torch.equal(states[[0, 2, 4]], first[[0, 2, 4]])
        got, states_2 = call([0, 930, last, last, last], [3, 1, 0, 4], step)
        assert (got[last:] == got.new_tensor(MARK)).all() and torch.equal(states_2[[0, 2, 4]], first[[0, 2, 4]])
        within(got[:last], ref[0][:last], ref[1][:last], "o")
        within(states_2, ref[2], ref[3], "states")
        for t in (q, k, v, g):
            t[last:] = 0.0


def test_two_graphs_share_a_workspace():
    """Captured calls of different batches, one workspace, replayed in turn and beside
    an eager call of a third."""
    rng = np.random.default_rng(39)
    H, d = 8, 64
    batches = []
    for lens in ([1500], [700, 60, 900], [2500, 3]):
        n = sum(lens)
        q, k, v = (rows(rng, n, (H, d), "bf16") for _ in range(3))
        g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
        b = K.LinearBatch(q, k, v, g, i32(cumulate(lens)))
        batches.append((b, K.StatePool.zeros(len(lens), H, d), i32(np.arange(len(lens)))))
    size = max(K.linear_workspace(b).numel() for b, _, _ in batches)
    work, want = torch.empty(size, dtype=torch.uint8, device="cuda"), []

    def call(i):
        b, pool, slots = batches[i]
        pool.data.zero_()
        K.kda_linear_prefill(b, pool, slots, workspace=work)
    for i, (b, pool, _) in enumerate(batches):
        call(i)
        want.append((b.o.clone(), pool.data.clone()))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            call(i)
    for order in ((0, 2, 1), (1, 0, 2), (1, 2, 0)):
        for b, pool, _ in batches:
            b.o.zero_()
            pool.data.fill_(7.0)
        for i in order:
            graphs[i].replay() if i < 2 else call(2)
        for (b, pool, _), (o, states) in zip(batches, want):
            assert torch.equal(b.o, o) and torch.equal(pool.data, states)


def test_a_nan_reaches_what_follows_it():
    """A decay that is NaN: the tokens from it on, and the state."""
    rng = np.random.default_rng(37)
    H, d, n = 2, 64, 200
    for dt in ("bf16", "f32"):
        q, k, v = (rows(rng, n, (H, d), dt) for _ in range(3))
        g = torch.full((n, H), -0.1, device="cuda")
        g[100, 1] = float("nan")
        for ws in (True, False):
            b = K.LinearBatch(q, k, v, g, i32([0, n]))
            pool = K.StatePool.zeros(1, H, d)
            K.kda_linear_prefill(b, pool, i32([0]), workspace=K.linear_workspace(b) if ws else None)
            assert b.o[:, 0].isfinite().all() and b.o[:100].isfinite().all() and b.o[100:, 1].isnan().all()
            assert pool.data[0, 0].isfinite().all() and pool.data[0, 1].isnan().all()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dt,dk,dv", [("bf16", 64, 64), ("bf16", 128, 64), ("bf16", 64, 128), ("f32", 64, 64)])
def test_where_a_nan_of_q_k_or_v_goes(dt, dk, dv, workspace):
    """q: its token; k: its head's later tokens; v: its channel's later tokens, and on
    the tensor cores those of its chunk of 64."""
    rng = np.random.default_rng(40)
    H, n, at = 3, 500, 300
    tc = dt == "bf16"
    base = [rows(rng, n, (H, dk), dt), rows(rng, n, (H, dk), dt, std=dk ** -0.5), rows(rng, n, (H, dv), dt)]
    g = torch.full((n, H), -0.1, device="cuda")

    def call(which, bad):
        x = [t.clone() for t in base]
        if which is not None:
            x[which][at, 1, 5] = bad
        b = K.LinearBatch(*x, g, i32([0, n]))
        pool = K.StatePool.zeros(1, H, dk, d_v=dv)
        K.kda_linear_prefill(b, pool, i32([0]), workspace=K.linear_workspace(b) if workspace else None)
        return b.o, pool.data[0]
    clean, state = call(None, 0.0)
    for bad in (float("nan"), float("inf")):
        for which in range(3):
            o, s = call(which, bad)
            touched = torch.zeros(n, H, dv, dtype=torch.bool, device="cuda")
            states = torch.zeros(H, dv, dk, dtype=torch.bool, device="cuda")
            if which == 0:
                touched[at, 1] = True
            elif which == 1:
                touched[at:, 1] = True
                states[1, :, 5] = True
            else:
                touched[at // 64 * 64 if tc else at:, 1, 5] = True
                states[1, 5] = True
            assert torch.equal(o[~touched], clean[~touched]) and torch.equal(s[~states], state[~states])
            assert not s[states].isfinite().any()
            if which == 2 or bad != bad:
                hit = touched.clone()
                hit[:at] = False
                assert not o[hit].isfinite().any()


# ------------------------------------------------------------- head norms
def qk_case(seed, dt, n, hq, hk, d, norm="rms", rot=0, interleaved=False, view=0, weights=True,
            scale=0.3, in_place=False, span=50):
    rng = np.random.default_rng(seed)
    q = rows(rng, n, (hq, d), dt, view, 3.0) if hq else None
    k = rows(rng, n, (hk, d), dt, view, 0.2) if hk else None
    wq, wk = ((torch.from_numpy(rng.standard_normal(d)).to("cuda", DT[dt]) if weights else None)
              for _ in range(2))
    table = pos = None
    if rot:
        angle = rng.uniform(0, 7, (span, rot // 2))
        table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float().cuda()
        pos = i32(rng.integers(0, span, n))
    want = [None if x is None else
            linear_ref.qk_norm(f64(x), None if w is None else f64(w), norm, 1e-5,
                               None if table is None else f64(table),
                               None if pos is None else pos.cpu().numpy(), interleaved, s, dt)
            for x, w, s in ((q, wq, scale), (k, wk, 1.0))]
    batch = K.QKBatch(q, k, wq, wk, norm, 1e-5, table, pos, interleaved, scale,
                      *((q, k) if in_place else ()))
    K.kda_qk_norm(batch)
    for got, w, what in zip((batch.q_out, batch.k_out), want, "qk"):
        if w is not None:
            within(got, w[0], w[1], what)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
def test_qk_norm(dt, norm):
    qk_case(40, dt, 37, 8, 2, 128, norm, rot=128)
    qk_case(41, dt, 1, 32, 32, 128, norm, rot=64, interleaved=True)
    qk_case(42, dt, 5, 3, 3, 80, norm)
    qk_case(43, dt, 100, 1, 1, 256, norm, rot=256, interleaved=True, weights=False)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(2, 2), (6, 4), (16, 16), (64, 16), (64, 24), (96, 96), (128, 2),
                                   (192, 64), (250, 100), (256, 128)])
def test_qk_norm_dims(dt, interleaved, d, rot):
    qk_case(44, dt, 19, 6, 2, d, rot=rot, interleaved=interleaved)
    qk_case(45, dt, 19, 5, 2, d, rot=rot, interleaved=interleaved, view=3, in_place=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_qk_norm_heads_and_places(dt):
    qk_case(46, dt, 300, 0, 3, 64, rot=32)
    qk_case(47, dt, 300, 36, 0, 64, rot=32)
    qk_case(48, dt, 70, 71, 13, 128, rot=128, view=8, in_place=True)
    qk_case(49, dt, 3000, 4, 1, 16, "l2", weights=False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt,n,hq,hk,d,rot", [
    ("bf16", 1301, 31, 5, 128, 128),   # heads that leave sets of four unfull
    ("bf16", 1800, 13, 0, 256, 64),    # queries alone, wide heads
    ("bf16", 700, 0, 70, 80, 32),      # keys alone, lanes without channels
    ("bf16", 200, 201, 9, 128, 32),    # more heads than a block takes
    ("f32", 1700, 10, 3, 128, 128), ("f32", 3001, 8, 8, 64, 0)])
def test_qk_norm_walking_down_the_tokens(interleaved, dt, n, hq, hk, d, rot):
    """Sizes from which a block goes on to further tokens."""
    qk_case(52, dt, n, hq, hk, d, rot=rot, interleaved=interleaved, view=8, in_place=interleaved)


@pytest.mark.parametrize("d", [64, 128])
def test_qk_norm_skips_tokens_past_the_table_walking(d):
    rng = np.random.default_rng(53)
    n, h = 2500, 32
    q = rows(rng, n, (h, d), "bf16")
    out = torch.full_like(q, MARK)
    pos = rng.integers(-3, 8, n)
    table = torch.cat([torch.ones(5, d // 2), torch.zeros(5, d // 2)], 1).cuda()
    K.kda_qk_norm(K.QKBatch(q, None, cos_sin=table, positions=i32(pos), q_out=out))
    assert K.kda_get_device_error() == K.KDA_DERR_POSITION
    want, tol = linear_ref.qk_norm(f64(q), None, "rms", 1e-6, None, None, False, 1.0, "bf16")
    live = (pos >= 0) & (pos < 5)
    within(out[torch.from_numpy(live).cuda()], want[live], tol[live], "q")
    assert (out[torch.from_numpy(~live).cuda()] == out.new_tensor(MARK)).all()


def test_qk_norm_of_one_projection_in_place():
    """q and k are parts of the rows that hold v too, and v stays as it is."""
    rng = np.random.default_rng(50)
    wide = rows(rng, 40, (10 * 64,), "bf16")
    before = wide.clone()
    q, k = wide[:, :384].unflatten(1, (6, 64)), wide[:, 384:512].unflatten(1, (2, 64))
    batch = K.QKBatch(q, k, norm="l2", q_out=q, k_out=k)
    K.kda_qk_norm(batch)
    assert torch.equal(wide[:, 512:], before[:, 512:])
    want, tol = linear_ref.qk_norm(f64(before[:, :512].unflatten(1, (8, 64))), None, "l2", 1e-6, None,
                                   None, False, 1.0, "bf16")
    within(wide[:, :512].unflatten(1, (8, 64)), want, tol, "qk")


@pytest.mark.parametrize("d", [64, 66])
def test_qk_norm_skips_tokens_past_the_table(d):
    rng = np.random.default_rng(51)
    q = rows(rng, 4, (2, d), "bf16")
    out = torch.full_like(q, 9.0)
    table = torch.cat([torch.ones(5, d // 2), torch.zeros(5, d // 2)], 1).cuda()
    K.kda_qk_norm(K.QKBatch(q, None, cos_sin=table, positions=i32([4, 5, -1, 0]), q_out=out))
    assert K.kda_get_device_error() == K.KDA_DERR_POSITION
    want, tol = linear_ref.qk_norm(f64(q), None, "rms", 1e-6, None, None, False, 1.0, "bf16")
    within(out[[0, 3]], want[[0, 3]], tol[[0, 3]], "q")
    assert (out[1:3] == 9).all()


def gate_case(seed, xdt, dt, n, H, d, silu=False, gate=True, weights=True, view=0, place=None):
    rng = np.random.default_rng(seed)
    x = rows(rng, n, (H, d), xdt, view, 2.0)
    u = rows(rng, n, (H, d), dt, view, 4.0) if gate else None
    w = torch.from_numpy(rng.standard_normal(d)).to("cuda", DT[dt]) if weights else None
    want, tol = linear_ref.gated_norm(f64(x), None if u is None else f64(u), None if w is None else f64(w),
                                      silu, 1e-5, dt)
    batch = K.GateBatch(x, u, w, "silu" if silu else "sigmoid", 1e-5, {"x": x, "gate": u, None: None}[place])
    assert batch.y.dtype == DT[dt]
    K.kda_gated_norm(batch)
    within(batch.y, want, tol, "y")


@pytest.mark.parametrize("xdt,dt", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("d", [1, 5, 16, 64, 80, 128, 200, 256])
def test_gated_norm(xdt, dt, d):
    gate_case(60, xdt, dt, 21, 5, d)
    gate_case(61, xdt, dt, 1, 32, d, silu=True, view=8)
    gate_case(62, xdt, dt, 33, 3, d, weights=False, view=1)
    gate_case(63, xdt, dt, 9, 2, d, gate=False)


def test_gated_norm_walking_down_the_rows():
    """Sizes from which a block goes on to further rows."""
    gate_case(67, "f32", "bf16", 3001, 7, 128, view=8)
    gate_case(68, "bf16", "bf16", 2000, 31, 64, silu=True, place="gate")
    gate_case(69, "f32", "f32", 5000, 3, 37)


def test_gated_norm_in_place():
    gate_case(64, "f32", "bf16", 50, 3, 128, place="gate")
    gate_case(65, "bf16", "bf16", 50, 3, 128, place="x", silu=True, view=8)
    gate_case(66, "f32", "f32", 50, 3, 37, place="x", view=1)


def test_a_layer_from_projection_to_projection():
    """The calls together, as a layer makes them: a prompt, then a step with drafts."""
    rng = np.random.default_rng(70)
    H, d, lens = 4, 64, [90, 33]
    cu, dt = cumulate(lens), "bf16"
    angle = np.outer(np.arange(256), 10000.0 ** (-np.arange(d // 2) * 2 / d))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float().cuda()
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(d)).to("cuda", DT[dt])
    states = K.StatePool(torch.from_numpy(rng.standard_normal((4, H, d, d))).float().cuda())
    slots = [3, 1]
    pool = f64(states.data)

    def layer(n, cu, pos, commit):
        proj = rows(rng, n, (4 * H * d,), dt)
        q, k, v, gate = (p.unflatten(1, (H, d)) for p in proj.split(H * d, 1))
        g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
        qk = K.QKBatch(q, k, w, w, cos_sin=table, positions=i32(pos), q_scale=d ** -0.5)
        K.kda_qk_norm(qk)
        batch = K.LinearBatch(qk.q_out, qk.k_out, v, g, i32(cu))
        if commit is None:
            K.kda_linear_prefill(batch, states, i32(slots), workspace=K.linear_workspace(batch))
        else:
            K.kda_linear_step(batch, states, i32(slots), i32(commit))
        out = K.GateBatch(batch.o, gate, w)
        K.kda_gated_norm(out)
        # each call against the definition on what the one before it gave
        for x, got, s in ((q, qk.q_out, d ** -0.5), (k, qk.k_out, 1.0)):
            want, tol = linear_ref.qk_norm(f64(x), f64(w), "rms", 1e-6, f64(table), pos, False, s, dt)
            within(got, want, tol, "qk")
        o, tol, new, new_tol = linear_ref.linear(f64(qk.q_out), f64(qk.k_out), f64(v), f64(g), cu, pool,
                                                 slots, 1.0, dt, True, commit)
        within(batch.o, o, tol, "o")
        within(states.data, new, new_tol, "states")
        want, tol = linear_ref.gated_norm(f64(batch.o), f64(gate), f64(w), False, 1e-6, dt)
        within(out.y, want, tol, "y")
        return f64(states.data)
    pos = np.concatenate([np.arange(n) for n in lens])
    pool = layer(sum(lens), cu, pos, None)
    layer(9, [0, 8, 9], np.array([*range(90, 98), 33]), [5, 1])
