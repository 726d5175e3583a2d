"""Where a NaN or an infinity goes in linear attention prompts: to nothing before it."""
import numpy as np
import pytest
import torch

from recurrent_kda_state_gb300 import kda as K
from test_gpu_linear import _ready, cumulate, decays, i32, rows  # noqa: F401

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf")]


def call(x, g, lens, first, workspace, every=0, ckpt=None, start=None):
    b, pool = K.LinearBatch(*x, g, i32(cumulate(lens))), K.StatePool(first.clone())
    K.kda_linear_prefill(b, pool, i32(np.arange(len(lens))), every, ckpt, start,
                         workspace=K.linear_workspace(b) if workspace else None)
    return b.o, pool.data


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("view", [0, 3])
@pytest.mark.parametrize("dt,dk,dv", [("bf16", 128, 128), ("bf16", 64, 64), ("bf16", 128, 64), ("bf16", 64, 128),
                                      ("bf16", 32, 64), ("f32", 64, 64)])
@pytest.mark.parametrize("start", [0, 5])
def test_a_bad_value_of_v_reaches_its_channel_from_its_token_on(dt, dk, dv, view, workspace, start):
    """One channel of each of several heads: the first, the last and inner tokens of a
    chunk, two in one chunk, and all kinds.  All else keeps its bits."""
    rng = np.random.default_rng(dk + 2 * dv + view)
    H, Hk, lens = 8, 4, [450, 70]
    n = sum(lens)
    x = [rows(rng, n, (Hk, dk), dt, view), rows(rng, n, (Hk, dk), dt, view, dk ** -0.5),
         rows(rng, n, (H, dv), dt, view)]
    g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
    first = torch.from_numpy(rng.standard_normal((2, H, dv, dk))).float().cuda()
    pos = i32([start, 0])
    clean, states = call(x, g, lens, first, workspace, start=pos)
    touched, touched_s = torch.zeros_like(clean, dtype=torch.bool), torch.zeros_like(states, dtype=torch.bool)
    x[2] = x[2].clone()
    # head, token of the batch, channel
    for i, (h, t, c) in enumerate([(0, 0, 0), (1, 63, dv - 1), (2, 64, 9), (3, 150, 17), (3, 130, 17), (3, 140, 3),
                                   (4, 319, 31), (5, 449, 6), (6, 450, 40), (6, 519, 41), (7, 191 - start, 15)]):
        x[2][t, h, c] = BAD[i % 3]
        seg = int(t >= lens[0])
        touched[t:n if seg else lens[0], h, c] = True
        touched_s[seg, h, c] = True
    o, s = call(x, g, lens, first, workspace, start=pos)
    assert torch.equal(o[~touched], clean[~touched]) and torch.equal(s[~touched_s], states[~touched_s])
    assert not o[touched].isfinite().any() and not s[touched_s].isfinite().any()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_checkpoints_before_a_bad_value_stay_clean(dk, dv, workspace):
    rng = np.random.default_rng(7)
    H, n = 2, 500
    x = [rows(rng, n, (H, dk), "bf16"), rows(rng, n, (H, dk), "bf16", std=dk ** -0.5), rows(rng, n, (H, dv), "bf16")]
    g = torch.full((n, H), -0.01, device="cuda")
    first = torch.zeros(8, H, dv, dk, device="cuda")
    ckpt = i32(np.arange(1, 8)[None])
    _, want = call(x, g, [n], first, workspace, 64, ckpt)
    x[2][200, 1, 7] = float("inf")
    _, got = call(x, g, [n], first, workspace, 64, ckpt)
    # slots 1, 2, 3 are the states after 64, 128 and 192 tokens
    assert torch.equal(got[1:4], want[1:4])
    later = [0, 4, 5, 6, 7]
    assert not got[later][:, 1, 7].isfinite().any()
    got[:, 1, 7] = want[:, 1, 7]
    assert torch.equal(got, want)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_a_bad_state_reaches_its_channel(dk, dv, workspace):
    """A NaN or an infinity in a slot: that channel of the outputs and the state, alone."""
    rng = np.random.default_rng(8)
    H, n = 3, 300
    x = [rows(rng, n, (H, dk), "bf16"), rows(rng, n, (H, dk), "bf16", std=dk ** -0.5), rows(rng, n, (H, dv), "bf16")]
    g = torch.full((n, H), -0.01, device="cuda")
    first = torch.from_numpy(rng.standard_normal((1, H, dv, dk))).float().cuda()
    want, states = call(x, g, [n], first, workspace)
    first[0, 0, 5, 3], first[0, 2, dv - 1, dk - 1] = float("nan"), float("inf")
    o, s = call(x, g, [n], first, workspace)
    for h, c in ((0, 5), (2, dv - 1)):
        assert not o[:, h, c].isfinite().any() and not s[0, h, c].isfinite().all()
        o[:, h, c], s[0, h, c] = want[:, h, c], states[0, h, c]
    assert torch.equal(o, want) and torch.equal(s, states)
