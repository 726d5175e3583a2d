"""Segments of no tokens: their table entries count alike whether a batch is cut into
parts or not."""
import numpy as np
import pytest
import torch

import linear_dispatch
from recurrent_kda_state_gb300 import kda as K
from test_gpu_linear import _ready, cumulate, i32, rows  # noqa: F401

pytestmark = pytest.mark.gpu
LENS = {"bf16": [1200, 0, 65, 0], "f32": [700, 0, 33, 0]}


@pytest.mark.parametrize("cut", [True, False])
@pytest.mark.parametrize("dt,d", [("bf16", 64), ("f32", 32)])
def test_slots_of_empty_segments_are_checked(dt, d, cut):
    """A slot out of range is reported for them too; the other rows are served."""
    rng = np.random.default_rng(1)
    H, lens = 2, LENS[dt]
    n = sum(lens)
    assert bool(linear_dispatch.part_chunks(n, len(lens), dt, H, d, d))  # with a workspace
    q, k, v = (rows(rng, n, (H, d), dt) for _ in range(3))
    g = torch.full((H,), -0.05, device="cuda")

    def call(slots, start=None):
        b = K.LinearBatch(q, k, v, g, i32(cumulate(lens)))
        pool = K.StatePool(torch.full((5, H, d, d), 0.5, device="cuda"))
        K.kda_linear_prefill(b, pool, i32(slots), start_pos=None if start is None else i32(start),
                             workspace=K.linear_workspace(b) if cut else None)
        return b.o, pool.data, K.kda_get_device_error()
    o, states, bits = call([0, 1, 2, 3])
    assert bits == 0 and (states[[1, 3, 4]] == 0.5).all()
    for slots in ([0, -1, 2, 3], [0, 1, 2, -1], [0, 5, 2, 2 ** 31 - 1], [0, -1, 2, -1]):
        o_2, states_2, bits = call(slots)
        assert bits == K.KDA_DERR_SLOT
        assert torch.equal(o, o_2) and torch.equal(states, states_2)
    # where an empty segment starts has no part in anything
    o_2, states_2, bits = call([0, 1, 2, 3], [0, -7, 0, -1])
    assert bits == 0 and torch.equal(o, o_2) and torch.equal(states, states_2)
    # a row with a bad slot and a bad start is reported by its slot
    _, states_2, bits = call([0, 1, -1, 3], [0, 0, -3, 0])
    assert bits == K.KDA_DERR_SLOT and torch.equal(states_2[0], states[0]) and (states_2[1:] == 0.5).all()
    _, states_2, bits = call([0, 1, 2, 3], [0, 0, -3, 0])
    assert bits == K.KDA_DERR_SEGMENT and torch.equal(states_2[0], states[0]) and (states_2[1:] == 0.5).all()
