"""The norm of queries and keys before a KDA layer and the gated norm after it."""
import numpy as np
import pytest
import torch

import linear_ref
import oracle
from recurrent_kda_state_gb300 import kda as K
from test_gpu_linear import _ready, cumulate, f64, i32, rows, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [32, 128])
def test_a_kda_layer_from_projection_to_projection(d):
    """q, k, v and the gate from one projection's rows; keys of length 1 (rot_dim 0); a
    prompt, then speculative steps.  Each call against its definition on what the one
    before it gave, the layer against the oracle."""
    rng = np.random.default_rng(90)
    H, T, P, dt = 3, 4, 5, "bf16"
    bf16 = torch.bfloat16
    slots = i32([4, 1])
    pool, ring = K.StatePool.zeros(P, H, d), K.ReplayRing(P, H, d, T, bf16)
    session = oracle.OracleSession(P, H, d, d)
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(d)).to("cuda", bf16)

    def layer(n, cu, call, expected):
        q, k, v, gate = (p.unflatten(1, (H, d)) for p in rows(rng, n, (4 * H * d,), dt).split(H * d, 1))
        alpha = torch.from_numpy(rng.uniform(0.6, 1.0, (n, H, d))).to("cuda", bf16)
        beta = torch.from_numpy(rng.uniform(0.0, 1.0, (n, H))).to("cuda", bf16)
        norms = K.QKBatch(q, k, norm="l2", q_scale=d ** -0.5)
        K.kda_qk_norm(norms)
        for x, got, s in ((q, norms.q_out, d ** -0.5), (k, norms.k_out, 1.0)):
            within(got, *linear_ref.qk_norm(f64(x), None, "l2", 1e-6, None, None, False, s, dt), "qk")
        tok = K.TokenBatch(norms.q_out, norms.k_out, v.contiguous(), alpha, beta, i32(cu))
        call(tok)
        host = dict(q=f64(norms.q_out), k=f64(norms.k_out), v=f64(v), alpha=f64(alpha), beta=f64(beta),
                    cu_seqlens=cu)
        assert np.abs(f64(tok.o) - expected(host)).max() <= 2e-3
        out = K.GateBatch(tok.o, gate, w, "silu", 1e-6)
        assert out.y.dtype == bf16
        K.kda_gated_norm(out)
        within(out.y, *linear_ref.gated_norm(f64(tok.o), f64(gate), f64(w), True, 1e-6, dt), "y")

    cu = cumulate([70, 33])
    layer(103, cu, lambda tok: K.kda_prefill_chunked(tok, pool, slots, 16 if d < 64 else 64),
          lambda host: session.prefill(host, [4, 1])[0])
    cu = cumulate([T, T])
    for _ in range(4):
        layer(2 * T, cu, lambda tok: K.kda_verify(tok, T, pool, slots, ring),
              lambda host: session.verify(host, [4, 1]))
        accepted = rng.integers(0, T + 1, 2).astype(np.int32)
        K.kda_commit(i32(accepted), slots, pool, ring)
        session.commit(accepted, [4, 1])
    K.kda_materialize(slots, pool, ring)
    for s in (4, 1):
        got = np.swapaxes(f64(pool.data[s]), -1, -2)
        assert np.linalg.norm(got - session.pool[s]) <= 1e-3 * np.linalg.norm(session.pool[s])
