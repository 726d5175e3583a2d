"""Refusals of linear attention and of the head norms, on the host before any
CUDA call."""
import ctypes

import pytest
import torch

import linear_dispatch
from recurrent_kda_state_gb300 import kda as K
from recurrent_kda_state_gb300._build import build_library

by = ctypes.byref
PTR = ctypes.c_void_p(0x40000)


@pytest.fixture(scope="module")
def L():
    build_library()
    return K.lib()


def tok(**kw):
    f = dict(dtype=K.KDA_BF16, q=0x10000, k=0x11000, v=0x12000, o=0x13000, q_stride=64, k_stride=64,
             v_stride=256, o_stride=256, g=0x14000, g_stride=4, scale=1.0, cu_seqlens=0x50000,
             num_seqs=2, num_tokens=5, num_heads=4, num_qk_heads=2, d_k=32, d_v=64)
    f.update(kw)
    return K.kda_linear_tokens(**f)


def pool(**kw):
    f = dict(base=0x60000, num_slots=4, num_heads=4, d_k=32, d_v=64)
    f.update(kw)
    return K.kda_state_pool(**f)


LINEAR = [(dict(dtype=7), {}, K.KDA_EDTYPE), (dict(d_k=48), dict(d_k=48), K.KDA_ESHAPE),
          (dict(d_v=256), dict(d_v=256), K.KDA_ESHAPE), (dict(d_v=0), dict(d_v=0), K.KDA_ESHAPE),
          ({}, dict(d_k=64), K.KDA_ESHAPE), ({}, dict(num_heads=2), K.KDA_ESHAPE),
          (dict(num_qk_heads=3), {}, K.KDA_ESHAPE), (dict(num_qk_heads=0), {}, K.KDA_ESHAPE),
          (dict(num_qk_heads=8), {}, K.KDA_ESHAPE), (dict(num_heads=0), dict(num_heads=0), K.KDA_ESHAPE),
          (dict(num_heads=2 ** 20), dict(num_heads=2 ** 20), K.KDA_ESHAPE),
          ({}, dict(num_slots=0), K.KDA_ESHAPE), ({}, dict(base=None), K.KDA_EINVAL),
          ({}, dict(base=0x60008), K.KDA_EALIGN), (dict(q_stride=63), {}, K.KDA_ESHAPE),
          (dict(k_stride=0), {}, K.KDA_ESHAPE), (dict(v_stride=255), {}, K.KDA_ESHAPE),
          (dict(o_stride=255), {}, K.KDA_ESHAPE), (dict(o_stride=2 ** 30), {}, K.KDA_ESHAPE),
          (dict(g_stride=3), {}, K.KDA_ESHAPE), (dict(g_stride=-4), {}, K.KDA_ESHAPE),
          (dict(g=None), {}, K.KDA_EINVAL), (dict(g=0x14002), {}, K.KDA_EALIGN),
          (dict(q=None), {}, K.KDA_EINVAL), (dict(v=0x12001), {}, K.KDA_EALIGN),
          (dict(o=0x12000), {}, K.KDA_EINVAL), (dict(o=0x10000), {}, K.KDA_EINVAL),
          (dict(num_seqs=-1), {}, K.KDA_EINVAL), (dict(num_tokens=-1), {}, K.KDA_EINVAL),
          (dict(num_seqs=65536), {}, K.KDA_ESHAPE), (dict(num_tokens=2 ** 31 - 1), {}, K.KDA_ESHAPE),
          (dict(cu_seqlens=0x50002), {}, K.KDA_EALIGN)]


@pytest.mark.parametrize("t,p,want", LINEAR)
def test_linear_refusals(L, t, p, want):
    t, p = tok(**t), pool(**p)
    assert L.kda_linear_prefill(by(t), by(p), PTR, None, 0, 0, None, None, 0, None) == want
    assert L.kda_linear_step(by(t), by(p), PTR, None, None) == want


def test_linear_tables(L):
    t, p, call = tok(), pool(), L.kda_linear_prefill
    assert call(None, by(p), PTR, None, 0, 0, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), None, PTR, None, 0, 0, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), None, None, 0, 0, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), PTR, None, 2, 64, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), PTR, PTR, 2, 32, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), PTR, PTR, 2, -64, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), PTR, None, 0, 0, ctypes.c_void_p(0x70002), None, 0, None) == K.KDA_EALIGN
    assert call(by(t), by(p), PTR, None, 0, 0, None, ctypes.c_void_p(0x70010), 1 << 30,
                None) == K.KDA_EALIGN
    none = tok(cu_seqlens=None)
    assert call(by(none), by(p), PTR, None, 0, 0, None, None, 0, None) == K.KDA_EINVAL
    assert L.kda_linear_step(by(none), by(p), PTR, None, None) == K.KDA_EINVAL  # 5 tokens of 2 rows
    for empty in (tok(num_seqs=0, num_tokens=0), tok(num_tokens=0, q=None, k=None, v=None, o=None)):
        assert call(by(empty), by(p), PTR, None, 0, 0, None, None, 0, None) == K.KDA_OK
        assert L.kda_linear_step(by(empty), by(p), PTR, None, None) == K.KDA_OK


@pytest.mark.parametrize("dt,H,dk,dv", [("bf16", 32, 128, 128), ("bf16", 1, 64, 64), ("bf16", 64, 128, 64),
                                        ("bf16", 500, 64, 64), ("f32", 6, 64, 32), ("f32", 32, 128, 128),
                                        ("bf16", 3, 16, 16), ("f32", 4000, 16, 128)])
def test_workspace_of_a_batch_serves_smaller_ones(L, dt, H, dk, dv):
    """More tokens or more segments never need less, and what a batch is cut into
    fits."""
    tokens = [1, 64, 65, 128, 129, 200, 333, 1000, 3000, 4096, 8191, 8192, 16384, 100003, 2 ** 24]
    seqs = [1, 2, 3, 4, 7, 16, 37, 64, 500, 1024, 1025, 65535]
    code = {"f32": K.KDA_F32, "bf16": K.KDA_BF16}[dt]
    size = {(n, b): K.kda_linear_workspace_size(n, b, H, dk, dv, code) for n in tokens for b in seqs}
    for n, m in zip(tokens, tokens[1:]):
        assert all(size[n, b] <= size[m, b] for b in seqs)
    for b, c in zip(seqs, seqs[1:]):
        assert all(size[n, b] <= size[n, c] for n in tokens)
    for (n, b), bytes_ in size.items():
        assert bytes_ >= linear_dispatch.workspace(n, b, dt, H, dk, dv)


def test_workspace_too_small(L):
    n = 8192
    big = dict(num_tokens=n, num_seqs=1, num_heads=32, num_qk_heads=32, d_k=128, d_v=128, q_stride=4096,
               k_stride=4096, v_stride=4096, o_stride=4096, g_stride=32)
    need = linear_dispatch.workspace(n, 1, "bf16", 32, 128, 128)
    assert need and linear_dispatch.part_chunks(n, 1, "bf16", 32, 128, 128) == 15
    t, p = tok(**big), pool(num_heads=32, d_k=128, d_v=128)
    assert L.kda_linear_prefill(by(t), by(p), PTR, None, 0, 0, None, ctypes.c_void_p(0x70000), need - 1,
                                None) == K.KDA_ENOSPC
    for bad in ((-1, 1, 4, 64, 64, 1), (8192, 0, 4, 64, 64, 1), (8192, 65536, 4, 64, 64, 1), (8192, 1, 0, 64, 64, 1),
                (8192, 1, 4, 48, 64, 1), (8192, 1, 4, 64, 256, 1), (8192, 1, 4, 64, 64, 2), (16, 1, 4, 64, 64, 0)):
        assert K.kda_linear_workspace_size(*bad) == 0


def qk(**kw):
    f = dict(dtype=K.KDA_BF16, q=0x10000, k=0x11000, q_out=0x12000, k_out=0x13000, q_stride=256,
             k_stride=128, q_out_stride=256, k_out_stride=128, q_weight=None, k_weight=None,
             cos_sin=0x14000, positions=0x15000, num_tokens=5, num_q_heads=4, num_k_heads=2,
             head_dim=64, rot_dim=32, max_pos=8, interleaved=0, norm=K.KDA_NORM_RMS, eps=1e-6,
             q_scale=1.0)
    f.update(kw)
    return K.kda_qk_tokens(**f)


QK = [(dict(dtype=2), K.KDA_EDTYPE), (dict(num_tokens=-1), K.KDA_EINVAL), (dict(norm=3), K.KDA_EINVAL),
      (dict(norm=-1), K.KDA_EINVAL), (dict(head_dim=63), K.KDA_ESHAPE), (dict(head_dim=0), K.KDA_ESHAPE),
      (dict(head_dim=258), K.KDA_ESHAPE), (dict(rot_dim=66), K.KDA_ESHAPE), (dict(rot_dim=31), K.KDA_ESHAPE),
      (dict(rot_dim=-2), K.KDA_ESHAPE), (dict(max_pos=0), K.KDA_ESHAPE), (dict(num_q_heads=-1), K.KDA_EINVAL),
      (dict(num_k_heads=2 ** 20), K.KDA_ESHAPE), (dict(q_stride=255), K.KDA_ESHAPE),
      (dict(k_out_stride=127), K.KDA_ESHAPE), (dict(q=None), K.KDA_EINVAL), (dict(k_out=None), K.KDA_EINVAL),
      (dict(k=0x11001), K.KDA_EALIGN), (dict(q_weight=0x16008), K.KDA_EALIGN),
      (dict(cos_sin=None), K.KDA_EINVAL), (dict(cos_sin=0x14004), K.KDA_EALIGN),
      (dict(positions=None), K.KDA_EINVAL), (dict(positions=0x15002), K.KDA_EALIGN),
      (dict(q_out=0x10000, q_out_stride=512), K.KDA_EINVAL),   # in place with another stride
      (dict(k_out=0x12000), K.KDA_EINVAL), (dict(q_out=0x11000), K.KDA_EINVAL),
      (dict(num_tokens=0), K.KDA_OK), (dict(num_q_heads=0, num_k_heads=0, q=None), K.KDA_OK)]


@pytest.mark.parametrize("kw,want", QK)
def test_qk_refusals(L, kw, want):
    assert L.kda_qk_norm(by(qk(**kw)), None) == want


def gate(**kw):
    f = dict(x_dtype=K.KDA_F32, dtype=K.KDA_BF16, x=0x10000, gate=0x11000, weight=None, y=0x12000,
             x_stride=256, gate_stride=256, y_stride=256, num_tokens=5, num_heads=4, head_dim=64,
             silu=0, eps=1e-6)
    f.update(kw)
    return K.kda_gate_tokens(**f)


GATE = [(dict(dtype=2), K.KDA_EDTYPE), (dict(x_dtype=2), K.KDA_EDTYPE), (dict(num_tokens=-1), K.KDA_EINVAL),
        (dict(head_dim=257), K.KDA_ESHAPE), (dict(head_dim=0), K.KDA_ESHAPE), (dict(num_heads=0), K.KDA_ESHAPE),
        (dict(num_heads=2 ** 20), K.KDA_ESHAPE), (dict(x_stride=255), K.KDA_ESHAPE),
        (dict(gate_stride=255), K.KDA_ESHAPE), (dict(y_stride=0), K.KDA_ESHAPE), (dict(x=None), K.KDA_EINVAL),
        (dict(y=None), K.KDA_EINVAL), (dict(x=0x10002), K.KDA_EALIGN), (dict(gate=0x11001), K.KDA_EALIGN),
        (dict(weight=0x13004), K.KDA_EALIGN), (dict(y=0x10000), K.KDA_EINVAL),
        (dict(y=0x11000, y_stride=512), K.KDA_EINVAL), (dict(num_tokens=2 ** 30), K.KDA_ESHAPE),
        (dict(num_tokens=0), K.KDA_OK)]


@pytest.mark.parametrize("kw,want", GATE)
def test_gate_refusals(L, kw, want):
    assert L.kda_gated_norm(by(gate(**kw)), None) == want


def test_binding_refuses_tensors_that_do_not_fit():
    q, v, g = torch.zeros(4, 2, 16), torch.zeros(4, 4, 32), torch.zeros(4, 4)
    K.LinearBatch(q, q.clone(), v, g)
    K.LinearBatch(q, q.clone(), v, g[0].clone())
    for bad in (dict(k=q[:3]), dict(k=q.bfloat16()), dict(v=v[:3]), dict(g=g.double()), dict(g=g[:, :3]),
                dict(g=g[:1].expand(4, 4)), dict(o=torch.zeros(4, 4, 16)), dict(g=torch.zeros(8)[::2]),
                dict(cu_seqlens=torch.zeros(2, dtype=torch.int64)), dict(v=v.transpose(1, 2))):
        with pytest.raises(ValueError):
            K.LinearBatch(**dict(dict(q=q, k=q.clone(), v=v, g=g), **bad))
    pos, table = torch.zeros(4, dtype=torch.int32), torch.zeros(9, 16)
    for bad in (dict(norm="max"), dict(cos_sin=table), dict(positions=pos), dict(k=q[:, :, :8]),
                dict(q_weight=torch.ones(8)), dict(q_weight=torch.ones(16).bfloat16()),
                dict(q_out=q[:3]), dict(cos_sin=table.double(), positions=pos)):
        with pytest.raises(ValueError):
            K.QKBatch(**dict(dict(q=q, k=q.clone()), **bad))
    for bad in (dict(activation="relu"), dict(gate=v[:3]), dict(weight=torch.ones(32).bfloat16()),
                dict(y=v[:, :2]), dict(weight=torch.ones(16))):
        with pytest.raises(ValueError):
            K.GateBatch(**dict(dict(x=v, gate=v.clone()), **bad))


def test_binding_refuses_tensors_off_the_gpu():
    """Host memory in a kernel's arguments would fault, so it goes no further."""
    i32, q, v = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 16), torch.zeros(4, 4, 32)
    batch = K.LinearBatch(q, q.clone(), v, torch.zeros(4, 4))
    states = K.StatePool.zeros(4, 4, 16, device="cpu", d_v=32)
    qkb, gb = K.QKBatch(q, q.clone()), K.GateBatch(v, v.clone())
    for call in (lambda: K.kda_linear_step(batch, states, i32), lambda: K.kda_qk_norm(qkb),
                 lambda: K.kda_linear_prefill(batch, states, i32), lambda: K.kda_gated_norm(gb)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_binding_refuses_tensors_of_several_devices():
    """One tensor on the host among those on the GPU, at every argument."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    i32, q, v, g = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 16), torch.zeros(4, 4, 32), torch.zeros(4, 4)
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32)

    def refused(call, **kw):
        """With each argument on the host in turn, the others on the GPU."""
        on = {k: t.cuda() for k, t in kw.items()}
        for k in kw:
            with pytest.raises(ValueError):
                call(**dict(on, **{k: kw[k]}))
    refused(K.LinearBatch, q=q, k=q, v=v, g=g, cu_seqlens=cu, o=v)
    refused(K.QKBatch, q=q, k=q, q_weight=torch.ones(16), k_weight=torch.ones(16), positions=i32,
            cos_sin=torch.zeros(9, 16), q_out=q, k_out=q)
    refused(K.GateBatch, x=v, gate=v, weight=torch.ones(32), y=v)
    batch = K.LinearBatch(q.cuda(), q.cuda(), v.cuda(), g.cuda(), cu.cuda())
    states = K.StatePool.zeros(4, 4, 16, d_v=32)
    refused(lambda **kw: K.kda_linear_step(batch, states, **kw), state_slots=i32, commit_len=i32)
    refused(lambda **kw: K.kda_linear_prefill(batch, states, ckpt_every=64, **kw), state_slots=i32,
            ckpt_slots=i32.view(4, 1), start_pos=i32)
    with pytest.raises(ValueError):
        K.kda_linear_prefill(batch, states, i32.cuda(), workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        K.kda_linear_step(batch, K.StatePool.zeros(4, 4, 16, device="cpu", d_v=32), i32.cuda())
