"""The norms of the states' errors against the limits of linear_states."""
import numpy as np
import pytest
import torch

from linear_states import TENSOR, WEAK, off, state64, walked
from recurrent_kda_state_gb300 import kda as K
from test_gpu_linear import _ready, f64, i32, rows  # noqa: F401

pytestmark = pytest.mark.gpu
DIMS = [(128, 128), (64, 64), (128, 64), (64, 128)]


def case(seed, dt, lens, H, dk, dv, decay, workspace, step=0, one_way=False):
    """The largest error of a segment's head; decay: a constant log decay, or None."""
    rng = np.random.default_rng(seed)
    n, B = sum(lens), len(lens)
    k, v = rows(rng, n, (H, dk), dt, std=dk ** -0.5), rows(rng, n, (H, dv), dt)
    if one_way:
        k, v = k.abs(), v.abs()
    g = -rng.exponential(0.02, (n, H)) if decay is None else np.full((n, H), decay)
    g = torch.from_numpy(g).float().cuda()
    first = torch.from_numpy(rng.standard_normal((B, H, dv, dk))).float().cuda()
    pool, slots = K.StatePool(first.clone()), i32(np.arange(B))
    if step:
        assert B == 1
        for t in range(0, n, step):
            e = min(t + step, n)
            K.kda_linear_step(K.LinearBatch(k[t:e], k[t:e], v[t:e], g[t:e], i32([0, e - t])), pool, slots)
    else:
        cu = np.concatenate([[0], np.cumsum(lens)])
        b = K.LinearBatch(k, k, v, g, i32(cu))
        K.kda_linear_prefill(b, pool, slots, workspace=K.linear_workspace(b) if workspace else None)
    worst, at = 0.0, 0
    for i, length in enumerate(lens):
        for h in range(H):
            args = [f64(t[at:at + length, h]) for t in (k, v, g)]
            worst = max(worst, off(f64(pool.data[i, h]), state64(*args, f64(first[i, h]))))
        at += length
    return worst


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("lens", [[65], [517, 130], [3000, 64, 1]])
def test_states_of_prompts_on_the_tensor_cores(dk, dv, lens, workspace):
    for decay in (None, WEAK[0]):
        assert case(5, "bf16", lens, 3, dk, dv, decay, workspace) < TENSOR


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_states_of_sums_in_one_direction(dk, dv, workspace):
    assert case(6, "bf16", [2000, 700], 2, dk, dv, WEAK[1], workspace, one_way=True) < TENSOR


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dt,dk,dv", [("f32", 64, 64), ("f32", 128, 128), ("bf16", 32, 32), ("f32", 16, 128)])
@pytest.mark.parametrize("decay", WEAK)
def test_states_of_prompts_token_by_token(dt, dk, dv, workspace, decay):
    assert case(7, dt, [4000], 2, dk, dv, decay, workspace) < walked(4000)


@pytest.mark.parametrize("dt,step", [("bf16", 1), ("f32", 1), ("bf16", 40)])
@pytest.mark.parametrize("decay", WEAK)
def test_states_of_many_steps(dt, step, decay):
    assert case(8, dt, [4000], 2, 64, 64, decay, False, step) < walked(4000)
