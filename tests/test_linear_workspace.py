"""What kda_linear_prefill itself asks of a workspace, against what the size query gives.

The call refuses a workspace that is too small before it looks for a GPU, and without a
GPU goes no further than that, so its answers on a host without one tell exactly how
many bytes it wants."""
import ctypes
import random

import pytest
import torch

import linear_dispatch
from recurrent_kda_state_gb300 import kda as K
from recurrent_kda_state_gb300._build import build_library

CODE = {"f32": K.KDA_F32, "bf16": K.KDA_BF16}
SHAPES = [("bf16", 32, 128, 128), ("bf16", 1, 64, 64), ("bf16", 64, 128, 64), ("bf16", 500, 64, 64),
          ("f32", 6, 64, 32), ("f32", 32, 128, 128), ("bf16", 3, 16, 16), ("f32", 4000, 16, 128)]
TOKENS = [1, 16, 17, 64, 128, 129, 200, 333, 1000, 4096, 8192, 16384, 40000, 100003, 2 ** 20, 2 ** 24]
SEQS = [1, 2, 3, 4, 7, 16, 37, 64, 200, 500, 1024, 1025, 40000]


@pytest.fixture(scope="module", autouse=True)
def _host():
    build_library()
    if torch.cuda.is_available():
        pytest.skip("with a GPU the call would run")


def status(n, b, dt, H, dk, dv, size):
    """Of the call on such a batch with a workspace of `size` bytes."""
    tok = K.kda_linear_tokens(dtype=CODE[dt], q=0x10000, k=0x20000, v=0x30000, o=0x40000, q_stride=H * dk,
                              k_stride=H * dk, v_stride=H * dv, o_stride=H * dv, g=0x50000, g_stride=H, scale=1.0,
                              cu_seqlens=0x60000, num_seqs=b, num_tokens=n, num_heads=H, num_qk_heads=H, d_k=dk,
                              d_v=dv)
    pool = K.kda_state_pool(base=0x70000, num_slots=4, num_heads=H, d_k=dk, d_v=dv)
    at = ctypes.c_void_p(0x80000)
    return K.lib().kda_linear_prefill(ctypes.byref(tok), ctypes.byref(pool), at, None, 0, 0, None, at, size, None)


def wanted(n, b, *shape):
    """The least size that the call takes, by bisection."""
    low, high = -1, 1 << 60
    assert status(n, b, *shape, high) != K.KDA_ENOSPC
    while high - low > 1:
        mid = (low + high) // 2
        if status(n, b, *shape, mid) == K.KDA_ENOSPC:
            low = mid
        else:
            high = mid
    return high


@pytest.mark.parametrize("dt,H,dk,dv", SHAPES)
def test_the_size_query_covers_what_the_call_wants(dt, H, dk, dv):
    """Of the batch itself and of every smaller one."""
    need = {(n, b): wanted(n, b, dt, H, dk, dv) for n in TOKENS for b in SEQS}
    most = 0
    for j, n in enumerate(TOKENS):
        for i, b in enumerate(SEQS):
            size = K.kda_linear_workspace_size(n, b, H, dk, dv, CODE[dt])
            assert size >= max(need[m, c] for m in TOKENS[:j + 1] for c in SEQS[:i + 1]), (n, b)
            most = max(most, need[n, b])
    assert most > 0 or H >= 500  # some are cut, where the heads do not fill the machine


@pytest.mark.parametrize("dt,H,dk,dv", SHAPES)
def test_the_size_query_covers_batches_at_random(dt, H, dk, dv):
    """Small batches where a segment more or less, or a token, changes the cut."""
    rng = random.Random(dt + str(H))
    for _ in range(60):
        n, b = rng.randint(1, 3000), rng.randint(1, 40)
        size = K.kda_linear_workspace_size(n, b, H, dk, dv, CODE[dt])
        for _ in range(8):
            m, c = rng.randint(1, n), rng.randint(1, b)
            assert status(m, c, dt, H, dk, dv, size) != K.KDA_ENOSPC, (n, b, m, c)


@pytest.mark.parametrize("dt,H,dk,dv", SHAPES)
def test_the_restated_rule_is_the_calls(dt, H, dk, dv):
    for n in TOKENS:
        for b in SEQS:
            assert wanted(n, b, dt, H, dk, dv) == linear_dispatch.workspace(n, b, dt, H, dk, dv), (n, b)
