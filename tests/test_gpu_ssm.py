"""The state space layers' operators against their fp64 definitions: the short
causal convolution, the selective scan (prompts and steps) and slot moves."""
import numpy as np
import pytest
import torch

import ssm_dispatch
import ssm_ref
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


def rows(rng, n, shape, dt, view):
    """[n][*shape] on the device; view: the tail of wider rows, off 16 bytes."""
    size = int(np.prod(shape))
    wide = torch.from_numpy(rng.standard_normal((n, size + (3 if view else 0))))
    wide = wide.to("cuda", DT[dt])
    return (wide[:, 3:] if view else wide).unflatten(1, shape) if len(shape) > 1 else (
        wide[:, 3:] if view else wide)


def within(got, want, tol, what):
    bad = ~(np.abs(f64(got) - want) <= tol)
    assert not bad.any(), "%s: %d of %d values out of bounds, first %s" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[:4].tolist())


def cumulate(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


# ------------------------------------------------------------- convolution
def conv_case(seed, dt, lens, D, W, bias=True, act=True, view=False, step=False, commit=None,
              every=0, max_ckpt=0, start=None, extra=3):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    n, B = int(lens.sum()), len(lens)
    P = B * (1 + max_ckpt) + extra
    x = rows(rng, n, (D,), dt, view)
    w = torch.from_numpy(rng.standard_normal((D, W))).to("cuda", DT[dt])
    b = torch.from_numpy(rng.standard_normal(D)).to("cuda", DT[dt]) if bias else None
    data = torch.from_numpy(rng.standard_normal((P, W - 1, D))).to("cuda", DT[dt])
    ids = rng.permutation(P)
    slots = ids[:B]
    ckpt = None
    if max_ckpt:
        ckpt = ids[B:B + B * max_ckpt].reshape(B, max_ckpt).copy()
        ckpt[0, 0] = -1
    cu = cumulate(lens)
    want, tol, pool = ssm_ref.conv(
        f64(x), f64(w), None if b is None else f64(b), cu, f64(data), slots, act, dt,
        commit, ckpt, every, start)
    single = step and (lens == 1).all()
    batch = K.ConvBatch(x, w, b, None if single else i32(cu), "silu" if act else None)
    cp = K.ConvPool(data)
    if step:
        K.kda_conv_step(batch, cp, i32(slots), None if commit is None else i32(commit))
    else:
        K.kda_conv_prefill(batch, cp, i32(slots), every, None if ckpt is None else i32(ckpt),
                           None if start is None else i32(start))
    within(batch.y, want, tol, "y")
    np.testing.assert_array_equal(f64(cp.data), pool)


LENS = [[1], [2, 0, 1, 3], [7, 8, 9, 0, 0, 64], [130, 1, 517]]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", LENS)
def test_conv_prefill(dt, W, lens):
    conv_case(1, dt, lens, 136, W)


@pytest.mark.parametrize("D,view", [(1, False), (37, True), (256, True), (1032, False)])
def test_conv_prefill_channels_and_views(D, view):
    conv_case(2, "bf16", [33, 5], D, 4, bias=False, act=False, view=view)
    conv_case(3, "f32", [33, 5], D, 3, view=view)


def test_conv_prefill_many_segments():
    lens = np.random.default_rng(4).integers(0, 4, 700)
    conv_case(4, "bf16", lens, 40, 4)


def test_conv_prefill_long_tiles():
    """Tiles of the largest size, with a segment border inside."""
    conv_case(5, "bf16", [4099, 61, 4000], 2048, 4)


@pytest.mark.parametrize("start", [None, [0, 5, 30]])
def test_conv_checkpoints(start):
    conv_case(6, "bf16", [70, 3, 40], 64, 4, every=16, max_ckpt=3, start=start)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_step(dt, W):
    conv_case(7, dt, [1] * 9, 264, W, step=True)
    conv_case(8, dt, [8, 1, 0, 3, 8, 11], 264, W, step=True, commit=[0, 1, 0, 2, 8, 9])
    conv_case(9, dt, [8, 1, 0, 3], 51, W, step=True, view=True)


def test_conv_steps_follow_a_prompt():
    """A prompt and then steps give what one longer prompt gives."""
    rng = np.random.default_rng(10)
    D, W, n = 96, 4, 29
    x = rows(rng, n, (D,), "bf16", False)
    w = torch.from_numpy(rng.standard_normal((D, W))).to("cuda", torch.bfloat16)
    whole, parts = (K.ConvPool.zeros(2, W, D, torch.bfloat16) for _ in range(2))
    one = K.ConvBatch(x, w, cu_seqlens=i32([0, n]))
    K.kda_conv_prefill(one, whole, i32([1]))
    a = K.ConvBatch(x[:20], w, cu_seqlens=i32([0, 20]))
    K.kda_conv_prefill(a, parts, i32([1]))
    b = K.ConvBatch(x[20:25], w, cu_seqlens=i32([0, 5]))  # two of five drafts accepted
    K.kda_conv_step(b, parts, i32([1]), i32([2]))
    c = K.ConvBatch(x[22:], w, cu_seqlens=i32([0, 7]))
    K.kda_conv_step(c, parts, i32([1]))
    got = torch.cat([a.y, b.y[:2], c.y])
    assert torch.equal(got, one.y) and torch.equal(whole.data, parts.data)


# ------------------------------------------------------------------- scan
def scan_case(seed, dt, lens, D, S, G=1, gate=True, skip=True, bias=True, softplus=True,
              view=False, step=False, commit=None, every=0, max_ckpt=0, start=None, split=True,
              extra=3, dt_scale=1.0, fill=None):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    n, B = int(lens.sum()), len(lens)
    P = B * (1 + max_ckpt) + extra
    x, d = rows(rng, n, (D,), dt, view), rows(rng, n, (D,), dt, view) * dt_scale
    if not softplus:
        d = d.abs() * 0.1
    z = rows(rng, n, (D,), dt, view) if gate else None
    b, c = rows(rng, n, (G, S), dt, view), rows(rng, n, (G, S), dt, view)

    def par(a):
        return torch.from_numpy(a).to("cuda", torch.float32)
    A = par(-np.exp(rng.uniform(-3.0, 3.0, (D, S))))
    skips = par(rng.standard_normal(D)) if skip else None
    # without softplus a time step is dt + bias itself, which is not negative
    dtb = par(rng.uniform(-7.0, 0.0, D) if softplus else rng.uniform(0.0, 0.1, D)) if bias else None
    data = par(rng.standard_normal((P, D, S)))
    ids = rng.permutation(P)
    slots = ids[:B]
    ckpt = None
    if max_ckpt:
        ckpt = ids[B:B + B * max_ckpt].reshape(B, max_ckpt).copy()
        ckpt[0, 0] = -1
    cu = cumulate(lens)

    def opt(t):
        return None if t is None else f64(t)
    want, tol, pool, pool_tol = ssm_ref.scan(
        f64(x), f64(d), f64(A), f64(b), f64(c), opt(skips), opt(z),
        opt(dtb), cu, f64(data), slots, softplus, dt, commit, ckpt,
        every, start)
    single = step and (lens == 1).all()
    batch = K.ScanBatch(x, d, A, b, c, D=skips, z=z, dt_bias=dtb,
                        cu_seqlens=None if single else i32(cu), dt_softplus=softplus)
    sp = K.ScanPool(data)
    if step:
        K.kda_scan_step(batch, sp, i32(slots), None if commit is None else i32(commit))
    else:
        ws = K.scan_workspace(batch) if split else None
        if ws is not None:
            ws.fill_(0xff)  # NaN: nothing may be read before it is written
        K.kda_scan_prefill(batch, sp, i32(slots), every, None if ckpt is None else i32(ckpt),
                           None if start is None else i32(start), ws)
    within(batch.y, want, tol, "y")
    within(sp.data, pool, pool_tol, "states")


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("S", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_scan_prefill(split, dt, S, lens):
    scan_case(11, dt, lens, 72, S, split=split)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,G,view", [(1, 1, False), (37, 1, True), (130, 2, False),
                                      (384, 3, True), (513, 1, False)])
def test_scan_prefill_channels_groups_views(dt, D, G, view):
    scan_case(12, dt, [40, 3, 90], D, 16, G=G, view=view)
    scan_case(13, dt, [40, 3, 90], D, 64, G=G, view=view, gate=False, skip=False)


@pytest.mark.parametrize("kw", [dict(gate=False), dict(skip=False), dict(bias=False),
                                dict(softplus=False), dict(dt_scale=20.0),
                                dict(gate=False, skip=False, bias=False, softplus=False)])
def test_scan_prefill_options(kw):
    scan_case(14, "f32", [100, 31], 64, 16, **kw)
    scan_case(15, "bf16", [100, 31], 64, 16, **kw)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("start", [None, [0, 5, 30]])
@pytest.mark.parametrize("S", [16, 64])
def test_scan_checkpoints(split, start, S):
    scan_case(16, "f32", [300, 3, 100], 40, S, every=32, max_ckpt=4, start=start, split=split)


@pytest.mark.parametrize("split", [False, True])
def test_scan_prefill_long(split):
    """Long segments beside short ones: parts that start and end in tiles."""
    scan_case(17, "bf16", [3001, 17, 0, 700, 1], 160, 16, split=split)


@pytest.mark.parametrize("lens,D,S", [([3001], 40, 16), ([2500, 2500], 24, 32),
                                      ([1100], 520, 128), ([0, 1300, 0], 33, 64)])
def test_scan_prefill_many_parts(lens, D, S):
    """Segments of so many parts that a launch of its own joins them."""
    scan_case(35, "bf16", lens, D, S, start=[7] * len(lens), every=64, max_ckpt=2)
    scan_case(36, "f32", lens, D, S)


def test_scan_prefill_many_segments():
    lens = np.random.default_rng(18).integers(0, 6, 500)
    scan_case(18, "f32", lens, 24, 16)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("S", [16, 32, 64, 128])
def test_scan_step(dt, S):
    scan_case(19, dt, [1] * 11, 200, S, step=True)
    scan_case(20, dt, [8, 1, 0, 3, 8, 11], 200, S, step=True, commit=[0, 1, 0, 2, 8, 9])
    scan_case(21, dt, [8, 1, 0, 3], 51, S, step=True, view=True, gate=False)


def test_scan_step_groups():
    scan_case(22, "bf16", [1] * 5, 384, 16, G=3, step=True, view=True)


def test_scan_steps_follow_a_prompt():
    """Prompt and steps against one prompt, with a draft rejected between."""
    rng = np.random.default_rng(23)
    D, S, n = 64, 16, 53
    t = {k: rows(rng, n, (D,), "f32", False) for k in ("x", "dt", "z")}
    b, c = (rows(rng, n, (1, S), "f32", False) for _ in range(2))
    A = torch.from_numpy(-np.exp(rng.uniform(-2, 2, (D, S)))).to("cuda", torch.float32)

    def part(lo, hi):
        return K.ScanBatch(t["x"][lo:hi], t["dt"][lo:hi], A, b[lo:hi], c[lo:hi],
                           z=t["z"][lo:hi], cu_seqlens=i32([0, hi - lo]))
    whole, parts = K.ScanPool.zeros(2, D, S), K.ScanPool.zeros(2, D, S)
    one = part(0, n)
    K.kda_scan_prefill(one, whole, i32([1]))
    a, d, e = part(0, 40), part(40, 46), part(43, n)
    K.kda_scan_prefill(a, parts, i32([1]))
    K.kda_scan_step(d, parts, i32([1]), i32([3]))
    K.kda_scan_step(e, parts, i32([1]))
    got = torch.cat([a.y, d.y[:3], e.y])
    scale = float(one.y.abs().max())
    assert float((got - one.y).abs().max()) <= (8 * n + 64) * ssm_ref.U32 * 16 * scale
    assert float((whole.data - parts.data).abs().max()) <= \
        (8 * n + 64) * ssm_ref.U32 * 16 * float(whole.data.abs().max())


def test_nan_and_inf_stay_in_their_segment():
    """A NaN token spoils its own segment from there on, and nothing else."""
    rng = np.random.default_rng(24)
    D, S, lens = 64, 16, [40, 300, 50]
    n, cu = sum(lens), cumulate([40, 300, 50])
    args = [rows(rng, n, (D,), "f32", False) for _ in range(2)]
    b, c = (rows(rng, n, (1, S), "f32", False) for _ in range(2))
    A = torch.from_numpy(-np.exp(rng.uniform(-2, 2, (D, S)))).to("cuda", torch.float32)
    args[0][60, 7] = float("nan")
    args[0][70, 9] = float("inf")
    batch = K.ScanBatch(args[0], args[1], A, b, c, cu_seqlens=i32(cu))
    pool = K.ScanPool.zeros(3, D, S)
    K.kda_scan_prefill(batch, pool, i32([0, 1, 2]), workspace=K.scan_workspace(batch))
    bad = ~torch.isfinite(batch.y).cpu().numpy()
    assert bad[60:340, 7].all() and bad[70, 9]
    bad[60:340, 7] = bad[70:340, 9] = False
    assert not bad.any()
    w = torch.ones(D, 4, device="cuda")
    cb = K.ConvBatch(args[0], w, cu_seqlens=i32(cu), activation=None)
    K.kda_conv_prefill(cb, K.ConvPool.zeros(3, 4, D, torch.float32), i32([0, 1, 2]))
    bad = ~torch.isfinite(cb.y).cpu().numpy()
    assert bad[60:64, 7].all() and bad[70:74, 9].all() and bad.sum() == 8


def test_time_steps_far_out():
    """softplus at both ends: steps that vanish and steps that forget all."""
    D, S = 16, 16
    v = torch.linspace(-100.0, 100.0, 41, device="cuda")[:, None].expand(41, D).contiguous()
    x = torch.ones(41, D, device="cuda")
    b = torch.ones(41, 1, S, device="cuda")
    A = -torch.ones(D, S, device="cuda")
    pool = K.ScanPool(torch.ones(1, D, S, device="cuda"))
    batch = K.ScanBatch(x, v, A, b, b, cu_seqlens=i32([0, 41]))
    want, tol, end, end_tol = ssm_ref.scan(
        f64(x), f64(v), f64(A), f64(b), f64(b), None, None, None, np.array([0, 41]),
        np.ones((1, D, S)), [0])
    K.kda_scan_prefill(batch, pool, i32([0]))
    within(batch.y, want, tol, "y")
    within(pool.data, end, end_tol, "states")


# ------------------------------------------------------------------ streams
def test_calls_take_their_stream_and_can_be_captured():
    rng = np.random.default_rng(25)
    D, S, n = 128, 16, 600
    x, d = (rows(rng, n, (D,), "bf16", False) for _ in range(2))
    b, c = (rows(rng, n, (1, S), "bf16", False) for _ in range(2))
    w = torch.from_numpy(rng.standard_normal((D, 4))).to("cuda", torch.bfloat16)
    A = torch.from_numpy(-np.exp(rng.uniform(-2, 2, (D, S)))).to("cuda", torch.float32)
    cu, slots = i32([0, n]), i32([0])
    conv, u = K.ConvPool.zeros(2, 4, D, torch.bfloat16), torch.empty_like(x)
    scan = K.ScanPool.zeros(2, D, S)
    cb = K.ConvBatch(x, w, cu_seqlens=cu, y=u)
    sb = K.ScanBatch(u, d, A, b, c, cu_seqlens=cu)
    ws, src, dst = K.scan_workspace(sb), i32([0]), i32([1])
    arrays = K.SlotArrays([conv.data, scan.data])
    mws = K.move_workspace(arrays, 1)

    def layer(stream=None):
        K.kda_conv_prefill(cb, conv, slots, stream=stream)
        K.kda_scan_prefill(sb, scan, slots, workspace=ws, stream=stream)
        K.kda_move_slots(arrays, src, dst, mws, stream=stream)
    layer()
    torch.cuda.synchronize()
    first = [t.clone() for t in (sb.y, conv.data, scan.data)]
    for t in (conv.data, scan.data, sb.y, u):
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer(side)
    side.synchronize()
    for t, f in zip((sb.y, conv.data, scan.data), first):
        assert torch.equal(t, f)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for t in (conv.data, scan.data, sb.y, u):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for t, f in zip((sb.y, conv.data, scan.data), first):
        assert torch.equal(t, f)


# --------------------------------------------------------------- device data
def test_bad_device_data_is_skipped_and_reported():
    """Slot ids, segment tables and commit counts that are out of range leave
    the row's outputs and state as they were and set their bit."""
    rng = np.random.default_rng(26)
    D, S = 64, 16
    x, d = (rows(rng, 12, (D,), "f32", False) for _ in range(2))
    b, c = (rows(rng, 12, (1, S), "f32", False) for _ in range(2))
    w, A = torch.ones(D, 4, device="cuda"), -torch.ones(D, S, device="cuda")
    cases = [(i32([0, 4, 8, 12]), i32([0, 9, 2]), None, K.KDA_DERR_SLOT, [1]),
             (i32([0, 4, 8, 12]), i32([0, -1, 2]), None, K.KDA_DERR_SLOT, [1]),
             (i32([0, 4, 2, 12]), i32([0, 1, 2]), None, K.KDA_DERR_SEGMENT, [1]),
             (i32([0, 4, 8, 99]), i32([0, 1, 2]), None, K.KDA_DERR_SEGMENT, [2]),
             (i32([0, 4, 8, 12]), i32([0, 1, 2]), i32([4, 5, 0]), K.KDA_DERR_ACCEPT, [1]),
             (i32([0, 4, 8, 12]), i32([0, 1, 2]), i32([4, -1, 0]), K.KDA_DERR_ACCEPT, [1])]
    for cu, slots, commit, bit, skipped in cases:
        for step in (True, False):
            if commit is not None and not step:
                continue
            conv, scan = K.ConvPool.zeros(4, 4, D, torch.float32), K.ScanPool.zeros(4, D, S)
            conv.data.fill_(7.0), scan.data.fill_(7.0)
            cb = K.ConvBatch(x, w, cu_seqlens=cu)
            sb = K.ScanBatch(x, d, A, b, c, cu_seqlens=cu)
            cb.y.fill_(5.0), sb.y.fill_(5.0)
            for call, batch, pool in (("conv", cb, conv), ("scan", sb, scan)):
                if step:
                    getattr(K, "kda_%s_step" % call)(batch, pool, slots, commit)
                else:
                    getattr(K, "kda_%s_prefill" % call)(batch, pool, slots)
                assert K.kda_get_device_error() & bit
                for i in skipped:
                    if bit != K.KDA_DERR_SEGMENT:
                        assert (batch.y[4 * i:4 * i + 4] == 5.0).all()
                    assert (pool.data[1 if i == 1 else i] == 7.0).all()
                assert not (batch.y[:4] == 5.0).any()
    K.kda_get_device_error()


@pytest.mark.parametrize("lens", [[2000], [700, 0, 90, 33, 5] * 30])
def test_the_same_call_gives_the_same_bits(lens):
    """In whatever order the parts of a batch are worked on."""
    rng = np.random.default_rng(54)
    D, S, n, B = 512, 64, sum(lens), len(lens)
    x, d = (rows(rng, n, (D,), "bf16", False) for _ in range(2))
    b, c = (rows(rng, n, (1, S), "bf16", False) for _ in range(2))
    A = torch.from_numpy(-np.exp(rng.uniform(-2, 2, (D, S)))).to("cuda", torch.float32)
    seen = []
    for _ in range(4):
        pool = K.ScanPool.zeros(B, D, S)
        batch = K.ScanBatch(x, d, A, b, c, cu_seqlens=i32(cumulate(lens)))
        K.kda_scan_prefill(batch, pool, i32(np.arange(B)), workspace=K.scan_workspace(batch))
        seen.append((batch.y, pool.data))
    for y, states in seen[1:]:
        assert torch.equal(y, seen[0][0]) and torch.equal(states, seen[0][1])


def test_overlapping_segments_are_reported():
    """A segment table that runs over the batch again and again has more parts
    than a large ragged batch has room for: nothing is done, the bit is set."""
    D, S, n, B = 384, 128, 8000, 41
    x = torch.zeros(n, D, device="cuda")
    b = torch.zeros(n, 1, S, device="cuda")
    A = -torch.ones(D, S, device="cuda")
    cu = i32([0 if i % 2 == 0 else n for i in range(B + 1)])
    pool = K.ScanPool(torch.full((B, D, S), 3.0, device="cuda"))
    batch = K.ScanBatch(x, x.clone(), A, b, b, cu_seqlens=cu)
    batch.y.fill_(5.0)
    K.kda_scan_prefill(batch, pool, i32(np.arange(B)), workspace=K.scan_workspace(batch))
    assert K.kda_get_device_error() == K.KDA_DERR_SEGMENT
    assert bool((batch.y == 5.0).all()) and bool((pool.data == 3.0).all())


# -------------------------------------------------------------------- moves
def move_case(seed, P, src, dst, ws=True, shapes=((4, 33), (128, 16), (5000, 2))):
    rng = np.random.default_rng(seed)
    dts = [torch.bfloat16, torch.float32, torch.int32]
    ts = [torch.from_numpy(rng.integers(-1000, 1000, (P,) + s)).to("cuda", d)
          for s, d in zip(shapes, dts)]
    want = ssm_ref.moves([f64(t) for t in ts], src, dst)
    arrays = K.SlotArrays(ts)
    K.kda_move_slots(arrays, i32(src), i32(dst), K.move_workspace(arrays, len(src)) if ws else None)
    for t, w in zip(ts, want):
        np.testing.assert_array_equal(f64(t), w)


def test_moves():
    move_case(27, 9, [0], [5], ws=False)                       # fork
    move_case(28, 9, [0, 0, 0, -1], [5, 6, 8, 1], ws=False)    # one source, many copies; free
    move_case(29, 9, [0, 1, 2, 3], [1, 2, 3, 0])               # a cycle
    move_case(30, 9, [3, 5, 5, -1, 7, 2], [0, 3, 1, 5, -1, 2])  # chain, fork, free, none, self
    move_case(31, 9, [8, 7, -1, -1], [1, 2, 8, 7])             # compaction
    move_case(32, 1, [-1], [0])


def test_moves_permutation_of_many():
    rng = np.random.default_rng(33)
    move_case(33, 700, rng.permutation(700), rng.permutation(700), shapes=((1, 2), (3, 5), (7, 1)))


def test_moves_out_of_range_are_skipped():
    t = torch.arange(12, device="cuda", dtype=torch.int32).view(4, 3)
    arrays = K.SlotArrays([t])
    K.kda_move_slots(arrays, i32([0, 4, 1]), i32([4, 2, 3]))
    assert K.kda_get_device_error() == K.KDA_DERR_SLOT
    assert t.tolist() == [[0, 1, 2], [3, 4, 5], [6, 7, 8], [3, 4, 5]]


# ------------------------------------------------------------ long offsets
def test_offsets_past_31_bits():
    """Rows and slots whose element offsets pass 2^31."""
    D, S, n = 64, 16, 6
    stride = 2 ** 29 + 8
    wide = torch.zeros(5 * stride + D, dtype=torch.bfloat16, device="cuda")
    x = wide.as_strided((n, D), (stride, 1))
    rng = np.random.default_rng(34)
    x.copy_(rows(rng, n, (D,), "bf16", False))
    d = rows(rng, n, (D,), "bf16", False)
    b, c = (rows(rng, n, (1, S), "bf16", False) for _ in range(2))
    A = torch.from_numpy(-np.exp(rng.uniform(-2, 2, (D, S)))).to("cuda", torch.float32)
    w = torch.from_numpy(rng.standard_normal((D, 4))).to("cuda", torch.bfloat16)
    P = 2 ** 31 // (D * S) + 2
    data = torch.zeros(P, D, S, device="cuda")
    pool, slots, cu = K.ScanPool(data), i32([P - 1]), i32([0, n])
    ref = K.ScanPool.zeros(1, D, S)
    for call in ("prefill", "step"):
        far = K.ScanBatch(x, d, A, b, c, cu_seqlens=cu)
        near = K.ScanBatch(x.contiguous(), d, A, b, c, cu_seqlens=cu)
        getattr(K, "kda_scan_" + call)(far, pool, slots)
        getattr(K, "kda_scan_" + call)(near, ref, i32([0]))
        assert torch.equal(far.y, near.y) and torch.equal(data[-1], ref.data[0])
        cfar, cnear = K.ConvBatch(x, w, cu_seqlens=cu), K.ConvBatch(x.contiguous(), w, cu_seqlens=cu)
        for bt in (cfar, cnear):
            getattr(K, "kda_conv_" + call)(bt, K.ConvPool.zeros(1, 4, D, torch.bfloat16), i32([0]))
        assert torch.equal(cfar.y, cnear.y)
    arrays = K.SlotArrays([data])
    K.kda_move_slots(arrays, i32([P - 1]), i32([P - 2]))
    assert torch.equal(data[-2], data[-1]) and not data[-3].any()


def test_example_serves_what_whole_prefills_give():
    """Prefill, fork, speculative steps and compaction in a stack of layers.
    bf16 layers round a few values differently in another batch: the layers'
    outputs differ by that rounding, 2^-8 of a value, and not by a state's
    history."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "examples", "selective_ssm.py")
    spec = importlib.util.spec_from_file_location("selective_ssm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, bits = mod.main()
    assert bits == 0 and worst < 2.0 ** -7


@pytest.mark.parametrize("seed", range(4))
def test_moves_in_columns(seed):
    """Slots so large that every thread does all moves at its place: chains,
    forks out of chains, cycles with tails, frees, and entries to skip."""
    rng = np.random.default_rng(seed)
    P = 40
    slots = rng.permutation(P).tolist()
    src, dst = [], []
    for n in (2, 3, 5):                             # cycles
        c, slots = slots[:n], slots[n:]
        src += c
        dst += c[1:] + c[:1]
        src += [c[0], c[n - 1]]                     # copies of what a cycle moves
        dst += slots[:2]
        src.append(dst[-1])                         # and what was there goes on
        dst.append(slots[2])
        slots = slots[3:]
    c, slots = slots[:6], slots[6:]                 # a chain with a fork, its start freed
    src += c[:-1] + [c[2], -1]
    dst += c[1:] + [slots[0], c[0]]
    src += [5, 7, -1]
    dst += [-1, 7 if 7 not in dst else -1, -1]      # nothing, itself, nothing
    k = rng.permutation(len(src))
    src, dst = np.array(src)[k], np.array(dst)[k]
    live = dst[dst >= 0]
    assert len(set(live.tolist())) == len(live)
    move_case(40 + seed, P, src, dst, shapes=((512, 516), (1024, 513), (4, 4)))


def test_scan_prefill_ragged_batches_take_their_parts_in_order():
    """Batches so large that their parts are listed first: split and whole
    segments, empty ones, checkpoints and starts that are no multiple of 16."""
    rng = np.random.default_rng(50)
    lens = np.concatenate([rng.integers(0, 60, 90), [2100, 0, 1300, 1, 16, 900]])
    rng.shuffle(lens)
    scan_case(51, "bf16", lens, 16 * 24, 128)
    scan_case(52, "f32", lens, 16 * 24, 128, every=64, max_ckpt=2,
              start=rng.integers(0, 100, len(lens)))
    scan_case(53, "bf16", rng.integers(0, 30, 3000), 48, 128)


@pytest.mark.parametrize("S", [16, 128])
def test_states_that_forget_all(S):
    """A = -inf: a token of a time step above 0 forgets what was there, one of a
    time step of 0 leaves it, in prompts (whole and cut) and in steps alike."""
    rng = np.random.default_rng(82)
    D, n = 24, 300
    x, d = rows(rng, n, (D,), "f32", False), rows(rng, n, (D,), "f32", False).abs()
    d[torch.from_numpy(rng.random(n) < 0.5).cuda()] = 0.0
    d[:2], d[-1] = 0.0, 0.0
    b, c = (rows(rng, n, (1, S), "f32", False) for _ in range(2))
    A = torch.from_numpy(-np.exp(rng.uniform(-2, 2, (D, S)))).to("cuda", torch.float32)
    A[::3], A[:, ::5] = -float("inf"), -float("inf")
    data = torch.from_numpy(rng.standard_normal((n, D, S))).to("cuda", torch.float32)
    # a decay of exp(-1e30 delta) is 0 or, for a time step of 0, 1
    finite = np.where(np.isinf(f64(A)), -1e30, f64(A))

    def run(lens, how):
        cu, slots = cumulate(lens), np.arange(len(lens))
        want, tol, pool, pool_tol = ssm_ref.scan(
            f64(x), f64(d), finite, f64(b), f64(c), None, None, None, cu, f64(data[:len(lens)]),
            slots, softplus_on=False)
        single = how == "one"
        batch = K.ScanBatch(x, d, A, b, c, cu_seqlens=None if single else i32(cu), dt_softplus=False)
        states = K.ScanPool(data[:len(lens)].clone())
        if how in ("whole", "cut"):
            ws = K.scan_workspace(batch) if how == "cut" else None
            K.kda_scan_prefill(batch, states, i32(slots), workspace=ws)
        else:
            K.kda_scan_step(batch, states, i32(slots))
        within(batch.y, want, tol, "y, " + how)
        within(states.data, pool, pool_tol, "states, " + how)
    run([n], "whole")
    run([n], "cut")
    run([n], "rows")
    run([1] * n, "one")


def test_one_workspace_serves_smaller_batches():
    """A workspace of the size for the largest batch of a server, used for batches
    of fewer tokens and prompts, which may be cut into more parts; the bytes after
    it stay as they are."""
    D, S, G, max_tokens, max_seqs = 50, 64, 25, 5000, 19
    n = K.kda_scan_workspace_size(max_tokens, max_seqs, D, S, G)
    buf = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(81)
    A = torch.from_numpy(-np.exp(rng.uniform(-3.0, 3.0, (D, S)))).to("cuda", torch.float32)
    for N, B in ((5000, 19), (5000, 18), (4000, 18), (4900, 1), (33, 2), (3000, 3)):
        lens = rng.multinomial(N, np.full(B, 1.0 / B))
        x, d = (rows(rng, N, (D,), "f32", False) for _ in range(2))
        b, c = (rows(rng, N, (G, S), "f32", False) for _ in range(2))
        data = torch.from_numpy(rng.standard_normal((B, D, S))).to("cuda", torch.float32)
        cu, slots = cumulate(lens), rng.permutation(B)
        want, tol, pool, pool_tol = ssm_ref.scan(f64(x), f64(d), f64(A), f64(b), f64(c), None, None,
                                                 None, cu, f64(data), slots)
        batch = K.ScanBatch(x, d, A, b, c, cu_seqlens=i32(cu))
        K.kda_scan_prefill(batch, K.ScanPool(data), i32(slots), workspace=buf[:n])
        within(batch.y, want, tol, "y")
        within(data, pool, pool_tol, "states")
    assert bool((buf[n:] == 0x5a).all())


@pytest.mark.parametrize("shape,ws", [((4, 4), False), ((4, 4), True), ((5,), True)])
def test_moves_out_of_range_alike_on_every_path(shape, ws):
    """An id that is not below the number of slots sets the bit, also where
    source and target are the same, whichever way the moves are done."""
    src, dst = [1, 0, 9, 3, -1], [2, 12, 4, -1, 10]
    for s, d, bit in ((8, 8, 1), (11, 11, 1), (5, 5, 0), (9, -1, 0)):
        t = torch.arange(8 * int(np.prod(shape)), device="cuda", dtype=torch.int32).view(8, *shape)
        was = t.clone()
        arrays = K.SlotArrays([t])
        area = K.move_workspace(arrays, 8) if ws else None
        K.kda_move_slots(arrays, i32([s]), i32([d]), area)
        assert K.kda_get_device_error() == (K.KDA_DERR_SLOT if bit else 0)
        assert torch.equal(t, was)
        K.kda_move_slots(arrays, i32(src + [s]), i32(dst + [d]), area)
        assert K.kda_get_device_error() == K.KDA_DERR_SLOT
        was[2] = was[1]
        assert torch.equal(t, was)


# ------------------------------------------- blocks of many rows, long chains
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("S,D,B", [(16, 2048, 310), (64, 500, 700), (128, 256, 333),
                                   (128, 4800, 300)])
def test_scan_step_many_rows_of_one_token(dt, S, D, B):
    """Decode batches in which a block takes many rows, one token each: the ring
    of states goes round and each row's token is asked for one row ahead."""
    assert ssm_dispatch.step_rows(dt, S, B, D, table=False) >= 6
    g = torch.Generator(device="cuda").manual_seed(60)

    def normal(*shape, to=DT[dt]):
        return torch.randn(*shape, generator=g, device="cuda").to(to)
    x, d, z = (normal(B, D) for _ in range(3))
    b, c = normal(B, 1, S), normal(B, 1, S)
    A = -torch.exp(torch.rand(D, S, generator=g, device="cuda") * 6.0 - 3.0)
    skip, bias = normal(D, to=torch.float32), normal(D, to=torch.float32) - 3.0
    data = normal(B + 5, D, S, to=torch.float32)
    slots = torch.randperm(B + 5, generator=g, device="cuda")[:B]
    keep = torch.rand(B, generator=g, device="cuda") < 0.7

    # fp64 on the device, with ssm_ref's bounds of a first token
    f = lambda t: t.double()  # noqa: E731
    delta = torch.nn.functional.softplus(f(d) + f(bias), threshold=700.0)
    decay = torch.exp(delta[..., None] * f(A))
    add = (delta * f(x))[..., None] * f(b)
    h0 = f(data)[slots]
    h = decay * h0 + add
    mag = decay * h0.abs() + add.abs()
    del decay, add, h0
    units = (8 + 64) * ssm_ref.U32
    o = (f(c) * h).sum(-1) + f(skip) * f(x)
    err = units * ((f(c).abs() * mag).sum(-1) + (f(skip) * f(x)).abs())
    gate = f(z) * torch.sigmoid(f(z))
    err = err * gate.abs() + (f(z).abs() + 8) * ssm_ref.U32 * (o * gate).abs()
    o = o * gate
    end, end_tol = f(data), torch.zeros_like(data, dtype=torch.float64)
    end[slots[keep]], end_tol[slots[keep]] = h[keep], units * mag[keep]

    batch = K.ScanBatch(x, d, A, b, c, D=skip, z=z, dt_bias=bias)
    K.kda_scan_step(batch, K.ScanPool(data), slots.int(), keep.int())
    assert bool(((f(batch.y) - o).abs() <= err + ssm_ref.U_OUT[dt] * o.abs()).all())
    assert bool(((f(data) - end).abs() <= end_tol).all())


def drafted(seed, B):
    """Lengths of a large step, empty rows and long ones among them, and how
    many tokens of each row the state takes in."""
    rng = np.random.default_rng(seed)
    lens = rng.choice([0, 1, 1, 1, 2, 8, 8, 40], B)
    lens[:2], lens[-1] = 0, 0
    return lens, rng.integers(0, lens + 1)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("S,D,G,B,view", [(16, 2048, 1, 310, False), (16, 700, 700, 300, False),
                                          (32, 1000, 1, 300, True), (128, 264, 1, 340, False)])
def test_scan_step_many_rows_of_several_tokens(dt, S, D, G, B, view):
    """Blocks of many rows of 0 to 40 tokens: items follow one another across
    rows, empty rows are passed over, the stages in shared memory go round."""
    assert ssm_dispatch.step_rows(dt, S, B, D, G) >= 6
    lens, commit = drafted(61, B)
    scan_case(62, dt, lens, D, S, G=G, step=True, commit=commit, view=view)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_conv_step_many_rows(dt):
    lens, commit = drafted(63, 700)
    conv_case(64, dt, lens, 260, 4, step=True, commit=commit)
    conv_case(65, dt, [1] * 700, 260, 3, step=True, commit=commit > 0)


@pytest.mark.parametrize("dt,lens,D", [("bf16", [4099, 61, 4000], 2800), ("f32", [2099, 61, 2000], 3840)])
def test_conv_prefill_largest_tiles(dt, lens, D):
    assert ssm_dispatch.conv_tile(dt, sum(lens), D) == 48
    conv_case(66, dt, lens, D, 4)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lens,D,S,G", [([0, 5000], 33, 64, 1), ([4100], 40, 16, 1),
                                        ([2200, 2100], 24, 32, 3), ([2500, 2500], 20, 128, 1)])
def test_scan_prefill_joined(dt, lens, D, S, G):
    """Batches whose parts are joined by a launch of their own."""
    assert ssm_dispatch.scan_joined(sum(lens), len(lens), D, S, G)
    assert not ssm_dispatch.scan_listed(sum(lens), len(lens), D, S, G)
    scan_case(67, dt, lens, D, S, G=G, every=512, max_ckpt=2, start=[9] * len(lens))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lens,D,S,G", [([1900, 3100], 200, 64, 25), ([5001, 2], 25, 64, 25),
                                        ([2900, 0, 5100], 250, 32, 25)])
def test_scan_prefill_listed_and_joined(dt, lens, D, S, G):
    """A few long prompts: the parts are listed first and joined between."""
    n, B = sum(lens), len(lens)
    assert ssm_dispatch.scan_listed(n, B, D, S, G) and ssm_dispatch.scan_joined(n, B, D, S, G)
    scan_case(68, dt, lens, D, S, G=G)
    scan_case(69, dt, lens, D, S, G=G, every=512, max_ckpt=2, start=[7, 100, 31][:B])


@pytest.mark.parametrize("S,D", [(16, 100), (32, 100), (64, 25)])
def test_scan_prefill_listed_f32(S, D):
    rng = np.random.default_rng(70)
    lens = np.concatenate([rng.integers(0, 60, 40), [1500, 0, 1300, 1, 16, 300]])
    rng.shuffle(lens)
    assert ssm_dispatch.scan_listed(int(lens.sum()), len(lens), D, S, 25)
    scan_case(71, "f32", lens, D, S, G=25, every=64, max_ckpt=2,
              start=rng.integers(0, 100, len(lens)))


# ------------------------------------------------- before a layer of KDA heads
def test_convolution_before_a_kda_layer():
    """q, k, v of KDA heads from one projection, three convolutions of its parts:
    the outputs are the layer's packed tensors as they are.  A speculative step
    runs the drafts with a commit count of 0 before the verify, and again with
    the accepted counts when they are known."""
    import oracle
    rng = np.random.default_rng(80)
    H, d, W, T, P = 3, 32, 4, 4, 5
    D, lens, slots = H * d, [70, 33], i32([4, 1])
    bf16 = torch.bfloat16
    taps = [torch.from_numpy(rng.standard_normal((D, W)) * 0.5).to("cuda", bf16) for _ in range(3)]
    convs = [K.ConvPool.zeros(P, W, D, bf16) for _ in range(3)]
    pool, ring = K.StatePool.zeros(P, H, d), K.ReplayRing(P, H, d, T, bf16)
    sess = oracle.OracleSession(P, H, d, d)

    def project(n):  # the projection's rows, decay and beta
        rest = [rng.uniform(0.6, 1.0, (n, H, d)), rng.uniform(0.0, 1.0, (n, H))]
        return (rows(rng, n, (3 * D,), "bf16", False),
                *(torch.from_numpy(a).to("cuda", bf16) for a in rest))

    def layer(batches, alpha, beta, cu):
        q, k, v = (b.y.unflatten(1, (H, d)) for b in batches)
        k = torch.nn.functional.normalize(k.float(), dim=-1).to(bf16)
        tok = K.TokenBatch(q, k, v, alpha, beta, i32(cu))
        return tok, dict(q=f64(q), k=f64(k), v=f64(v), alpha=f64(alpha), beta=f64(beta),
                         cu_seqlens=cu)

    def batches(x, cu):
        return [K.ConvBatch(x[:, i * D:(i + 1) * D], taps[i], cu_seqlens=i32(cu)) for i in range(3)]

    def check(bs, x, cu, before, commit):
        for i, b in enumerate(bs):
            y, tol, after = ssm_ref.conv(f64(x)[:, i * D:(i + 1) * D], f64(taps[i]), None, cu,
                                         before[i], [4, 1], True, "bf16", commit)
            within(b.y, y, tol, "conv")
            np.testing.assert_array_equal(f64(convs[i].data), after)

    before = [f64(c.data) for c in convs]
    x, alpha, beta = project(sum(lens))
    cu = cumulate(lens)
    bs = batches(x, cu)
    for b, c in zip(bs, convs):
        K.kda_conv_prefill(b, c, slots)
    check(bs, x, cu, before, None)
    tok, host = layer(bs, alpha, beta, cu)
    K.kda_prefill_chunked(tok, pool, slots, 16)
    want, _ = sess.prefill(host, [4, 1])
    assert np.abs(f64(tok.o) - want).max() <= 2e-3
    cu = cumulate([T, T])
    for _ in range(4):
        before = [f64(c.data) for c in convs]
        x, alpha, beta = project(2 * T)
        bs = batches(x, cu)
        for b, c in zip(bs, convs):
            K.kda_conv_step(b, c, slots, i32([0, 0]))
        check(bs, x, cu, before, [0, 0])
        tok, host = layer(bs, alpha, beta, cu)
        K.kda_verify(tok, T, pool, slots, ring)
        assert np.abs(f64(tok.o) - sess.verify(host, [4, 1])).max() <= 2e-3
        accepted = rng.integers(0, T + 1, 2).astype(np.int32)
        K.kda_commit(i32(accepted), slots, pool, ring)
        sess.commit(accepted, [4, 1])
        for b, c in zip(bs, convs):
            K.kda_conv_step(b, c, slots, i32(accepted))
        check(bs, x, cu, before, accepted)
    K.kda_materialize(slots, pool, ring)
    for s in (4, 1):
        got = np.swapaxes(f64(pool.data[s]), -1, -2)
        assert np.linalg.norm(got - sess.pool[s]) <= 1e-3 * np.linalg.norm(sess.pool[s])
