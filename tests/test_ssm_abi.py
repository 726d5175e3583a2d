"""Refusals of the state space layers' calls, on the host before any CUDA call."""
import ctypes

import pytest
import torch

import ssm_dispatch
from recurrent_kda_state_gb300 import kda as K
from recurrent_kda_state_gb300._build import build_library

by = ctypes.byref
PTR = ctypes.c_void_p(0x40000)


@pytest.fixture(scope="module")
def L():
    build_library()
    return K.lib()


def conv_tok(**kw):
    f = dict(dtype=K.KDA_BF16, x=0x10000, y=0x20000, x_stride=64, y_stride=64, weight=0x30000,
             bias=None, cu_seqlens=0x50000, num_seqs=2, num_tokens=5, channels=64, width=4, silu=1)
    f.update(kw)
    return K.kda_conv_tokens(**f)


def conv_pool(**kw):
    f = dict(base=0x60000, dtype=K.KDA_BF16, num_slots=4, channels=64, width=4)
    f.update(kw)
    return K.kda_conv_pool(**f)


def scan_tok(**kw):
    f = dict(dtype=K.KDA_BF16, x=0x10000, dt=0x11000, z=None, B=0x12000, C=0x13000, y=0x20000,
             x_stride=64, dt_stride=64, z_stride=0, b_stride=16, c_stride=16, y_stride=64,
             A=0x30000, D=None, dt_bias=None, cu_seqlens=0x50000, num_seqs=2, num_tokens=5,
             channels=64, state=16, groups=1, dt_softplus=1)
    f.update(kw)
    return K.kda_scan_tokens(**f)


def scan_pool(**kw):
    f = dict(base=0x60000, num_slots=4, channels=64, state=16)
    f.update(kw)
    return K.kda_scan_pool(**f)


CONV = [(dict(dtype=7), {}, K.KDA_EDTYPE), ({}, dict(dtype=K.KDA_F32), K.KDA_EDTYPE),
        (dict(width=5), dict(width=5), K.KDA_ESHAPE), ({}, dict(width=3), K.KDA_ESHAPE),
        (dict(channels=0), dict(channels=0), K.KDA_ESHAPE), ({}, dict(channels=32), K.KDA_ESHAPE),
        (dict(x_stride=63), {}, K.KDA_ESHAPE), (dict(y_stride=8), {}, K.KDA_ESHAPE),
        (dict(x=0x10001), {}, K.KDA_EALIGN), (dict(weight=0x30008), {}, K.KDA_EALIGN),
        (dict(bias=0x30004), {}, K.KDA_EALIGN), ({}, dict(base=0x60008), K.KDA_EALIGN),
        (dict(x=None), {}, K.KDA_EINVAL), (dict(weight=None), {}, K.KDA_EINVAL),
        (dict(y=0x10000), {}, K.KDA_EINVAL), ({}, dict(base=None), K.KDA_EINVAL),
        (dict(num_seqs=-1), {}, K.KDA_EINVAL), (dict(num_tokens=-1), {}, K.KDA_EINVAL),
        (dict(num_seqs=65536), {}, K.KDA_ESHAPE), ({}, dict(num_slots=0), K.KDA_ESHAPE),
        (dict(num_tokens=2 ** 31 - 1), {}, K.KDA_ESHAPE), (dict(x_stride=2 ** 30), {}, K.KDA_ESHAPE),
        (dict(cu_seqlens=0x50002), {}, K.KDA_EALIGN)]


@pytest.mark.parametrize("tok,pool,want", CONV)
def test_conv_refusals(L, tok, pool, want):
    t, p = conv_tok(**tok), conv_pool(**pool)
    assert L.kda_conv_prefill(by(t), by(p), PTR, None, 0, 0, None, None) == want
    assert L.kda_conv_step(by(t), by(p), PTR, None, None) == want


def test_conv_tables(L):
    t, p = conv_tok(), conv_pool()
    assert L.kda_conv_prefill(None, by(p), PTR, None, 0, 0, None, None) == K.KDA_EINVAL
    assert L.kda_conv_prefill(by(t), None, PTR, None, 0, 0, None, None) == K.KDA_EINVAL
    assert L.kda_conv_prefill(by(t), by(p), None, None, 0, 0, None, None) == K.KDA_EINVAL
    assert L.kda_conv_prefill(by(t), by(p), PTR, None, 2, 16, None, None) == K.KDA_EINVAL
    assert L.kda_conv_prefill(by(t), by(p), PTR, PTR, 2, -1, None, None) == K.KDA_EINVAL
    assert L.kda_conv_prefill(by(conv_tok(cu_seqlens=None)), by(p), PTR, None, 0, 0, None,
                              None) == K.KDA_EINVAL          # prompts need their table
    assert L.kda_conv_step(by(conv_tok(cu_seqlens=None)), by(p), PTR, None,
                           None) == K.KDA_EINVAL             # 5 tokens of 2 rows
    for none in (conv_tok(num_seqs=0, num_tokens=0), conv_tok(num_tokens=0, x=None, y=None)):
        assert L.kda_conv_prefill(by(none), by(p), PTR, None, 0, 0, None, None) == K.KDA_OK
        assert L.kda_conv_step(by(none), by(p), PTR, None, None) == K.KDA_OK


SCAN = [(dict(dtype=7), {}, K.KDA_EDTYPE), (dict(state=24), dict(state=24), K.KDA_ESHAPE),
        ({}, dict(state=32), K.KDA_ESHAPE), ({}, dict(channels=32), K.KDA_ESHAPE),
        (dict(groups=3), {}, K.KDA_ESHAPE), (dict(groups=0), {}, K.KDA_ESHAPE),
        (dict(groups=2), {}, K.KDA_ESHAPE),                  # rows of B shorter than G * S
        (dict(dt_stride=63), {}, K.KDA_ESHAPE), (dict(z=0x14000, z_stride=63), {}, K.KDA_ESHAPE),
        (dict(c_stride=15), {}, K.KDA_ESHAPE), (dict(dt=0x11001), {}, K.KDA_EALIGN),
        (dict(A=0x30004), {}, K.KDA_EALIGN), (dict(D=0x30004), {}, K.KDA_EALIGN),
        (dict(dt_bias=0x30004), {}, K.KDA_EALIGN), ({}, dict(base=0x60008), K.KDA_EALIGN),
        (dict(A=None), {}, K.KDA_EINVAL), (dict(B=None), {}, K.KDA_EINVAL),
        (dict(dt=None), {}, K.KDA_EINVAL), (dict(y=0x11000), {}, K.KDA_EINVAL),
        (dict(num_seqs=-1), {}, K.KDA_EINVAL), (dict(num_seqs=65536), {}, K.KDA_ESHAPE),
        (dict(num_tokens=2 ** 31 - 1), {}, K.KDA_ESHAPE), (dict(b_stride=2 ** 30), {}, K.KDA_ESHAPE)]


@pytest.mark.parametrize("tok,pool,want", SCAN)
def test_scan_refusals(L, tok, pool, want):
    t, p = scan_tok(**tok), scan_pool(**pool)
    assert L.kda_scan_prefill(by(t), by(p), PTR, None, 0, 0, None, None, 0, None) == want
    assert L.kda_scan_step(by(t), by(p), PTR, None, None) == want


def test_scan_tables_and_workspace(L):
    t, p = scan_tok(), scan_pool()
    call = L.kda_scan_prefill
    assert call(None, by(p), PTR, None, 0, 0, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), None, None, 0, 0, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), PTR, PTR, 1, 24, None, None, 0, None) == K.KDA_EINVAL
    assert call(by(t), by(p), PTR, None, 0, 0, None, ctypes.c_void_p(0x70010), 1 << 30,
                None) == K.KDA_EALIGN
    big = scan_tok(num_tokens=8192, channels=4096, x_stride=4096, dt_stride=4096, y_stride=4096)
    need = K.kda_scan_workspace_size(8192, 2, 4096, 16)
    if need:
        assert call(by(big), by(scan_pool(channels=4096)), PTR, None, 0, 0, None,
                    ctypes.c_void_p(0x70000), need - 1, None) == K.KDA_ENOSPC
    for bad in ((-1, 1, 64, 16, 1), (8, 0, 64, 16, 1), (8, 1, 0, 16, 1), (8, 1, 64, 24, 1),
                (8, 1, 64, 16, 3), (8, 65536, 64, 16, 1)):
        assert K.kda_scan_workspace_size(*bad) == 0
    wide = scan_tok(num_seqs=65535, channels=2 ** 20, state=128, x_stride=2 ** 20, b_stride=128,
                    dt_stride=2 ** 20, y_stride=2 ** 20, c_stride=128)
    assert call(by(wide), by(scan_pool(channels=2 ** 20, state=128)), PTR, None, 0, 0, None, None,
                0, None) == K.KDA_ESHAPE                      # more blocks than a grid has
    assert K.kda_scan_workspace_size(2 ** 30, 65535, 2 ** 20, 128) == 0
    none = scan_tok(num_seqs=0, num_tokens=0)
    assert call(by(none), by(p), None, None, 0, 0, None, None, 0, None) == K.KDA_OK


def test_move_refusals(L):
    def arr(base=0x10000, nbytes=64):
        return (K.kda_slot_array * 1)(K.kda_slot_array(base, nbytes))

    def call(a, na=1, P=4, src=PTR, dst=PTR, n=1, ws=None, nbytes=0):
        return L.kda_move_slots(a, na, P, src, dst, n, ws, nbytes, None)
    assert call(None) == K.KDA_EINVAL
    assert call(arr(), na=65) == K.KDA_EINVAL
    assert call(arr(), na=-1) == K.KDA_EINVAL
    assert call(arr(), n=-1) == K.KDA_EINVAL
    assert call(arr(), src=None) == K.KDA_EINVAL
    assert call(arr(), dst=None) == K.KDA_EINVAL
    assert call(arr(base=None)) == K.KDA_EINVAL
    assert call(arr(base=0x10008)) == K.KDA_EALIGN
    assert call(arr(nbytes=6)) == K.KDA_ESHAPE
    assert call(arr(nbytes=0)) == K.KDA_ESHAPE
    assert call(arr(), P=0) == K.KDA_ESHAPE
    assert call(arr(), n=3, ws=ctypes.c_void_p(0x70010), nbytes=1 << 20) == K.KDA_EALIGN
    assert call(arr(), n=3, ws=ctypes.c_void_p(0x70000), nbytes=191) == K.KDA_ENOSPC
    assert call(arr(), n=0, src=None, dst=None) == K.KDA_OK
    assert L.kda_move_workspace_size(arr(), 1, 3) == 192
    assert L.kda_move_workspace_size(arr(nbytes=20), 1, 3) == 96
    assert L.kda_move_workspace_size(arr(nbytes=6), 1, 3) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    x, w = torch.zeros(4, 8), torch.zeros(8, 4)
    K.ConvBatch(x, w)
    with pytest.raises(ValueError):
        K.ConvBatch(x, w.bfloat16())
    with pytest.raises(ValueError):
        K.ConvBatch(x, torch.zeros(7, 4))
    with pytest.raises(ValueError):
        K.ConvBatch(x.t(), torch.zeros(4, 4))             # channels not contiguous
    with pytest.raises(ValueError):
        K.ConvBatch(x, w, activation="relu")
    with pytest.raises(ValueError):
        K.ConvBatch(x, w, cu_seqlens=torch.zeros(2, dtype=torch.int64))
    A, b = torch.zeros(8, 16), torch.zeros(4, 1, 16)
    K.ScanBatch(x, x.clone(), A, b, b)
    with pytest.raises(ValueError):
        K.ScanBatch(x, x.clone()[:3], A, b, b)
    with pytest.raises(ValueError):
        K.ScanBatch(x, x.clone(), A.double(), b, b)
    with pytest.raises(ValueError):
        K.ScanBatch(x, x.clone(), A, b, torch.zeros(4, 2, 16))
    with pytest.raises(ValueError):
        K.ScanPool(torch.zeros(2, 8, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        K.SlotArrays([torch.zeros(4, 3), torch.zeros(5, 3)])
    batch = K.ConvBatch(x, w)
    with pytest.raises(ValueError):                       # a table of the wrong length or type
        K.kda_conv_step(batch, K.ConvPool(torch.zeros(2, 3, 8)), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        K.kda_conv_step(batch, K.ConvPool(torch.zeros(2, 3, 8)), torch.zeros(4))


@pytest.mark.parametrize("D,S,G", [(4096, 16, 1), (4096, 128, 1), (500, 64, 2), (33, 16, 1),
                                   (50, 64, 25), (2 ** 16, 16, 1), (2 ** 20, 16, 2 ** 10)])
def test_scan_workspace_of_a_batch_serves_smaller_ones(D, S, G):
    """More tokens or more segments never need less, and what a batch is cut into
    fits: a carry slot of 18 x 128 floats for each part and block of channels."""
    tokens = [1, 32, 33, 100, 1000, 3000, 4096, 8191, 8192, 16384, 100003, 2 ** 24]
    seqs = [1, 2, 3, 14, 15, 18, 19, 37, 64, 500]
    size = {(n, b): K.kda_scan_workspace_size(n, b, D, S, G) for n in tokens for b in seqs}
    for n, m in zip(tokens, tokens[1:]):
        assert all(size[n, b] <= size[m, b] for b in seqs)
    for b, c in zip(seqs, seqs[1:]):
        assert all(size[n, b] <= size[n, c] for n in tokens)
    nblk = ssm_dispatch.scan_blocks(D, S, G)
    for (n, b), bytes_ in size.items():
        part = ssm_dispatch.scan_part(n, b, D, S, G)
        slots = n // part + 2 * b if part else 0
        assert bytes_ >= slots * (nblk * 18 * 128 * 4 + 8)


def test_scan_workspace_stays_near_the_need():
    """One more part than two waves hold at most, beside two of every segment."""
    slot = 32 * 18 * 128 * 4
    for n, b in ((8192, 1), (16384, 37), (100000, 200)):
        assert K.kda_scan_workspace_size(n, b, 4096, 16, 1) <= (2 * 760 // 32 + 2 * b + 1) * slot


def test_move_workspace_that_cannot_be_counted(L):
    """2^30 moves of 2^39 bytes are 2^69: no workspace is large enough."""
    arr = (K.kda_slot_array * 1)(K.kda_slot_array(0x10000, 2 ** 39))
    for n in (2 ** 30, 2 ** 31 - 1):
        assert L.kda_move_workspace_size(arr, 1, n) == 0
        assert L.kda_move_slots(arr, 1, 4, PTR, PTR, n, ctypes.c_void_p(0x70000), 2 ** 20,
                                None) == K.KDA_ENOSPC
    assert L.kda_move_workspace_size(arr, 1, 2 ** 20) == 2 ** 59


def test_binding_refuses_tensors_off_the_gpu():
    """Host memory in a kernel's arguments would fault, so it goes no further."""
    i32, x = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)
    conv, scan = K.ConvPool(torch.zeros(4, 3, 8)), K.ScanPool(torch.zeros(4, 8, 16))
    b = torch.zeros(4, 1, 16)
    cb, sb = K.ConvBatch(x, torch.zeros(8, 4)), K.ScanBatch(x, x.clone(), torch.zeros(8, 16), b, b)
    arrays = K.SlotArrays([conv.data, scan.data])
    for call in (lambda: K.kda_conv_step(cb, conv, i32), lambda: K.kda_scan_step(sb, scan, i32),
                 lambda: K.kda_conv_prefill(cb, conv, i32), lambda: K.kda_scan_prefill(sb, scan, i32),
                 lambda: K.kda_move_slots(arrays, i32, i32)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_binding_refuses_tensors_of_several_devices():
    """One tensor on the host among those on the GPU, at every argument."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    i32, x, w = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8), torch.zeros(8, 4)
    b, A, v = torch.zeros(4, 1, 16), torch.zeros(8, 16), torch.zeros(8)
    conv, scan = torch.zeros(4, 3, 8), torch.zeros(4, 8, 16)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)

    def refused(call, *args, **kw):
        """With each argument on the host in turn, the others on the GPU."""
        on = {k: t.cuda() for k, t in kw.items()}
        for k in kw:
            with pytest.raises(ValueError):
                call(*args, **dict(on, **{k: kw[k]}))
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32)
    refused(K.ConvBatch, x=x, weight=w, bias=v, cu_seqlens=cu, y=x)
    refused(K.ScanBatch, x=x, dt=x, A=A, B=b, C=b, D=v, z=x, dt_bias=v, cu_seqlens=cu, y=x)
    cb = K.ConvBatch(x.cuda(), w.cuda(), cu_seqlens=cu.cuda())
    sb = K.ScanBatch(x.cuda(), x.cuda(), A.cuda(), b.cuda(), b.cuda(), cu_seqlens=cu.cuda())
    cp, sp = K.ConvPool(conv.cuda()), K.ScanPool(scan.cuda())
    ckpt = i32.view(4, 1)
    refused(K.kda_conv_step, cb, cp, state_slots=i32, commit_len=i32)
    refused(K.kda_scan_step, sb, sp, state_slots=i32, commit_len=i32)
    for call, batch, pool, host in ((K.kda_conv_prefill, cb, cp, conv),
                                    (K.kda_scan_prefill, sb, sp, scan)):
        refused(lambda **kw: call(batch, pool, ckpt_every=16, **kw), state_slots=i32,
                ckpt_slots=ckpt, start_pos=i32)
        with pytest.raises(ValueError):
            call(batch, type(pool)(host), i32.cuda())
    with pytest.raises(ValueError):
        K.kda_scan_prefill(sb, sp, i32.cuda(), workspace=ws)
    with pytest.raises(ValueError):
        K.SlotArrays([conv.cuda(), scan])
    arrays = K.SlotArrays([conv.cuda(), scan.cuda()])
    refused(lambda **kw: K.kda_move_slots(arrays, **kw), src=i32, dst=i32, workspace=ws)
