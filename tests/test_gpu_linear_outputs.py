"""Outputs of linear attention prompts in bf16, whose state is kept in fp32: how
near they are to the definition."""
import numpy as np
import pytest
import torch

import linear_ref
from recurrent_kda_state_gb300 import kda as K
from test_gpu_linear import _ready, cumulate, decays, f64, i32, rows, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("view", [0, 3])
@pytest.mark.parametrize("dk,dv,H,Hk", [(128, 128, 2, 2), (64, 64, 3, 1), (128, 64, 4, 2), (64, 128, 2, 2)])
def test_outputs_read_the_state_in_more_than_bf16(dk, dv, H, Hk, view, workspace):
    """States that outweigh a chunk's own tokens.  Beside the rounding of the outputs
    and the roundings in fp32 (linear_ref), two factors are split into two bf16, the
    state and the decayed products of q and k: the first keeps 8 bits of 24 by
    cutting them off, the second rounds the next 16 to 8, so that the last of them is
    off by half a unit of bit 15 at most, 2^-16 of its product.  The state as one
    bf16 would be off by 2^-8 of them."""
    rng = np.random.default_rng(dk + dv + view)
    lens = [700, 65, 1, 130]
    n, cu = sum(lens), cumulate(lens)
    q, v = rows(rng, n, (Hk, dk), "bf16", view), rows(rng, n, (H, dv), "bf16", view)
    k = rows(rng, n, (Hk, dk), "bf16", view, dk ** -0.5)
    g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
    data = torch.from_numpy(rng.standard_normal((4, H, dv, dk))).float().cuda()
    args = (f64(q), f64(k), f64(v), f64(g), cu, f64(data), [2, 0, 3, 1], 0.7, "bf16")
    want, tol, pool, pool_tol = linear_ref.linear(*args)
    magnitude = (linear_ref.linear(*args, rounded_state=True)[1] - tol) * 2.0 ** 8
    batch, states = K.LinearBatch(q, k, v, g, i32(cu), 0.7), K.StatePool(data)
    K.kda_linear_prefill(batch, states, i32([2, 0, 3, 1]),
                         workspace=K.linear_workspace(batch) if workspace else None)
    within(batch.o, want, tol + 2.0 ** -16 * magnitude, "o")
    within(states.data, pool, pool_tol, "states")


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_prompts_and_steps_agree(dk, dv, workspace):
    """The same tokens by a prompt and by steps: two roundings to bf16, half a unit in
    the last place (2^-8) each, and what the test above allows."""
    rng = np.random.default_rng(5)
    H, n = 3, 200
    q, v = rows(rng, n, (H, dk), "bf16"), rows(rng, n, (H, dv), "bf16")
    k = rows(rng, n, (H, dk), "bf16", std=dk ** -0.5)
    g = torch.from_numpy(decays(rng, n, H, "mild")).float().cuda()
    data = torch.from_numpy(rng.standard_normal((1, H, dv, dk))).float().cuda()
    args = (f64(q), f64(k), f64(v), f64(g), [0, n], f64(data), [0], 1.0, "bf16")
    want, tol, _, _ = linear_ref.linear(*args)
    magnitude = (linear_ref.linear(*args, rounded_state=True)[1] - tol) * 2.0 ** 8
    prompt, steps = (K.LinearBatch(q, k, v, g, i32([0, n])) for _ in range(2))
    K.kda_linear_prefill(prompt, K.StatePool(data.clone()), i32([0]),
                         workspace=K.linear_workspace(prompt) if workspace else None)
    K.kda_linear_step(steps, K.StatePool(data.clone()), i32([0]))
    within(prompt.o, f64(steps.o), 2 * tol + 2.0 ** -16 * magnitude, "o")


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_the_largest_states_stay_finite(dk, dv, workspace):
    """A state next to the largest fp32 rounds to an infinity in bf16; the outputs that
    read it with q of 2^-100 are its product."""
    H, n = 1, 70
    top = torch.finfo(torch.float32).max
    q = torch.full((n, H, dk), 2.0 ** -100, device="cuda").bfloat16()
    zero = torch.zeros(n, H, dk, device="cuda").bfloat16()
    first = torch.zeros(1, H, dv, dk, device="cuda")
    first[0, 0, :, 1] = top
    batch = K.LinearBatch(q, zero, torch.zeros(n, H, dv, device="cuda").bfloat16(), torch.zeros(H, device="cuda"),
                          i32([0, n]))
    states = K.StatePool(first.clone())
    K.kda_linear_prefill(batch, states, i32([0]), workspace=K.linear_workspace(batch) if workspace else None)
    assert torch.equal(states.data, first)
    want = torch.tensor(top * 2.0 ** -100, dtype=torch.float64)
    # the outputs' rounding (2^-8) and the cut of the state (2^-16)
    assert ((batch.o.double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -16) * want).all()
