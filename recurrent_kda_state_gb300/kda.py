"""ctypes binding of libkda.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does
nothing but turn torch tensors into pointers and sizes; all arithmetic of the
path runs in the library's CUDA kernels.  The library must have been built
(``recurrent_kda_state_gb300._build.build_library``); if it is missing the
first call raises, there is no fallback.
"""
import ctypes
import os

import torch

from ._build import LIB

KDA_OK, KDA_EINVAL, KDA_EDTYPE, KDA_ESHAPE, KDA_EALIGN = 0, -1, -2, -3, -4
KDA_EPROTO, KDA_ECUDA, KDA_EDEVICE, KDA_ENOSPC = -5, -6, -7, -8
KDA_DERR_SLOT, KDA_DERR_ACCEPT, KDA_DERR_DEPTH = 1, 2, 4
KDA_DERR_SEGMENT, KDA_DERR_RING, KDA_DERR_RANGE = 8, 16, 32
KDA_DERR_TIMEOUT, KDA_DERR_UNSAFE, KDA_DERR_POSITION = 64, 128, 256
KDA_F32, KDA_BF16 = 0, 1
KDA_NORM_NONE, KDA_NORM_RMS, KDA_NORM_L2 = 0, 1, 2

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64


class kda_tokens(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("q", _P), ("k", _P), ("v", _P),
                ("alpha", _P), ("beta", _P), ("o", _P), ("cu_seqlens", _P),
                ("num_seqs", _I32), ("num_tokens", _I32), ("num_heads", _I32),
                ("d_k", _I32), ("d_v", _I32)]


class kda_state_pool(ctypes.Structure):
    _fields_ = [("base", _P), ("num_slots", _I32), ("num_heads", _I32),
                ("d_k", _I32), ("d_v", _I32)]


class kda_replay_ring(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("alpha", _P), ("beta", _P),
                ("ctrl", _P), ("depth", _I32), ("dtype", ctypes.c_int)]


class kda_conv_tokens(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("x", _P), ("y", _P), ("x_stride", _I64),
                ("y_stride", _I64), ("weight", _P), ("bias", _P), ("cu_seqlens", _P),
                ("num_seqs", _I32), ("num_tokens", _I32), ("channels", _I32),
                ("width", _I32), ("silu", _I32)]


class kda_conv_pool(ctypes.Structure):
    _fields_ = [("base", _P), ("dtype", ctypes.c_int), ("num_slots", _I32),
                ("channels", _I32), ("width", _I32)]


class kda_scan_tokens(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("x", _P), ("dt", _P), ("z", _P), ("B", _P),
                ("C", _P), ("y", _P), ("x_stride", _I64), ("dt_stride", _I64),
                ("z_stride", _I64), ("b_stride", _I64), ("c_stride", _I64),
                ("y_stride", _I64), ("A", _P), ("D", _P), ("dt_bias", _P),
                ("cu_seqlens", _P), ("num_seqs", _I32), ("num_tokens", _I32),
                ("channels", _I32), ("state", _I32), ("groups", _I32),
                ("dt_softplus", _I32)]


class kda_scan_pool(ctypes.Structure):
    _fields_ = [("base", _P), ("num_slots", _I32), ("channels", _I32), ("state", _I32)]


class kda_slot_array(ctypes.Structure):
    _fields_ = [("base", _P), ("slot_bytes", ctypes.c_size_t)]


class kda_linear_tokens(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("q", _P), ("k", _P), ("v", _P), ("o", _P),
                ("q_stride", _I64), ("k_stride", _I64), ("v_stride", _I64),
                ("o_stride", _I64), ("g", _P), ("g_stride", _I64), ("scale", ctypes.c_float),
                ("cu_seqlens", _P), ("num_seqs", _I32), ("num_tokens", _I32),
                ("num_heads", _I32), ("num_qk_heads", _I32), ("d_k", _I32), ("d_v", _I32)]


class kda_qk_tokens(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("q", _P), ("k", _P), ("q_out", _P), ("k_out", _P),
                ("q_stride", _I64), ("k_stride", _I64), ("q_out_stride", _I64),
                ("k_out_stride", _I64), ("q_weight", _P), ("k_weight", _P), ("cos_sin", _P),
                ("positions", _P), ("num_tokens", _I32), ("num_q_heads", _I32),
                ("num_k_heads", _I32), ("head_dim", _I32), ("rot_dim", _I32),
                ("max_pos", _I32), ("interleaved", _I32), ("norm", ctypes.c_int),
                ("eps", ctypes.c_float), ("q_scale", ctypes.c_float)]


class kda_gate_tokens(ctypes.Structure):
    _fields_ = [("x_dtype", ctypes.c_int), ("dtype", ctypes.c_int), ("x", _P), ("gate", _P),
                ("weight", _P), ("y", _P), ("x_stride", _I64), ("gate_stride", _I64),
                ("y_stride", _I64), ("num_tokens", _I32), ("num_heads", _I32),
                ("head_dim", _I32), ("silu", _I32), ("eps", ctypes.c_float)]


EXPORTS = ("kda_prefill_chunked", "kda_prefill_chunked_raw", "kda_prefill_chunked_noalloc",
           "kda_prefill_workspace_size", "kda_verify", "kda_verify_raw",
           "kda_commit", "kda_commit_layers", "kda_materialize", "kda_ring_reset",
           "kda_gather_states", "kda_copy_slots", "kda_verify_snapshot",
           "kda_commit_snapshot", "kda_forward_mixed", "kda_conv_prefill", "kda_conv_step",
           "kda_scan_prefill", "kda_scan_step", "kda_scan_workspace_size",
           "kda_move_slots", "kda_move_workspace_size", "kda_linear_prefill",
           "kda_linear_step", "kda_linear_workspace_size", "kda_qk_norm", "kda_gated_norm",
           "kda_get_device_error", "kda_set_wait_limit",
           "kda_status_string", "kda_version")

_lib = None


def lib():
    """The loaded libkda.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(
                "libkda.so is not built (%s); run __graft_entry__.build()" % LIB)
        L = ctypes.CDLL(LIB)
        tp, pp, rp = (ctypes.POINTER(kda_tokens), ctypes.POINTER(kda_state_pool),
                      ctypes.POINTER(kda_replay_ring))
        L.kda_prefill_chunked.argtypes = [tp, pp, _P, _P, _I32, _I32, _I32, _P,
                                          _P, ctypes.c_size_t, _P]
        L.kda_prefill_chunked_raw.argtypes = [tp, pp, _P, _P, _I32, _I32, _I32, _P,
                                              _P, ctypes.c_size_t, _P]
        L.kda_prefill_chunked_noalloc.argtypes = [tp, pp, _P, _P, _I32, _I32,
                                                  _I32, _P, _P]
        L.kda_prefill_workspace_size.argtypes = [_I32] * 6 + [ctypes.c_int]
        L.kda_prefill_workspace_size.restype = ctypes.c_size_t
        L.kda_verify.argtypes = [tp, _I32, pp, _P, rp, _P, _P]
        L.kda_verify_raw.argtypes = [tp, _I32, pp, _P, rp, _P, _P]
        L.kda_commit.argtypes = [_P, _P, _I32, pp, rp, _P]
        L.kda_commit_layers.argtypes = [_P, _P, _I32, pp, rp, _I32, _P]
        L.kda_materialize.argtypes = [_P, _I32, pp, rp, _P]
        L.kda_ring_reset.argtypes = [_P, _I32, pp, rp, _P]
        L.kda_gather_states.argtypes = [pp, _P, _I32, _P, _P]
        L.kda_copy_slots.argtypes = [pp, _P, _P, _I32, _P]
        L.kda_verify_snapshot.argtypes = [tp, _I32, pp, _P, _P, _P]
        L.kda_forward_mixed.argtypes = [tp, _I32, _I32, pp, _P, _P, _I32, _I32, _I32,
                                        _P, _P, ctypes.c_size_t, _I32, rp, _P, _P, _P]
        L.kda_commit_snapshot.argtypes = [_P, _P, _I32, pp, _P, _I32, _P]
        ct, cp = ctypes.POINTER(kda_conv_tokens), ctypes.POINTER(kda_conv_pool)
        st, sp = ctypes.POINTER(kda_scan_tokens), ctypes.POINTER(kda_scan_pool)
        ap, size = ctypes.POINTER(kda_slot_array), ctypes.c_size_t
        L.kda_conv_prefill.argtypes = [ct, cp, _P, _P, _I32, _I32, _P, _P]
        L.kda_conv_step.argtypes = [ct, cp, _P, _P, _P]
        L.kda_scan_prefill.argtypes = [st, sp, _P, _P, _I32, _I32, _P, _P, size, _P]
        L.kda_scan_step.argtypes = [st, sp, _P, _P, _P]
        L.kda_scan_workspace_size.argtypes = [_I32] * 5
        L.kda_scan_workspace_size.restype = size
        L.kda_move_slots.argtypes = [ap, _I32, _I32, _P, _P, _I32, _P, size, _P]
        L.kda_move_workspace_size.argtypes = [ap, _I32, _I32]
        L.kda_move_workspace_size.restype = size
        lt = ctypes.POINTER(kda_linear_tokens)
        L.kda_linear_prefill.argtypes = [lt, pp, _P, _P, _I32, _I32, _P, _P, size, _P]
        L.kda_linear_step.argtypes = [lt, pp, _P, _P, _P]
        L.kda_linear_workspace_size.argtypes = [_I32] * 5 + [ctypes.c_int]
        L.kda_linear_workspace_size.restype = size
        L.kda_qk_norm.argtypes = [ctypes.POINTER(kda_qk_tokens), _P]
        L.kda_gated_norm.argtypes = [ctypes.POINTER(kda_gate_tokens), _P]
        L.kda_get_device_error.argtypes = [ctypes.POINTER(_I32), _P]
        L.kda_set_wait_limit.argtypes = [_I32]
        L.kda_status_string.argtypes = [ctypes.c_int]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_version.restype = ctypes.c_int
        for name in EXPORTS:
            getattr(L, name).restype = getattr(L, name).restype or ctypes.c_int
        _lib = L
    return _lib


class KdaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().kda_status_string(status).decode()
        super().__init__("%s: %s" % (where, msg))


def _check(status, where):
    if status != KDA_OK:
        raise KdaError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without building a Stream object: a single-token
# step takes the GPU 2 us, and torch.cuda.current_stream() the host 3 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_ready = False  # the first call goes through torch, which sets CUDA up


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, dev=-1):
    """The stream's handle (None: the current one's) for a call on tensors of GPU dev:
    its kernels run on the current device, which has to be that one, as has the
    stream's.  dev -1: a call without tensors on a GPU."""
    global _raw_ready
    if dev >= 0 and _current_device() != dev:
        raise ValueError("the tensors are on GPU %d, the current device is GPU %d"
                         % (dev, _current_device()))
    if stream is not None:
        if dev >= 0 and stream.device_index != dev:
            raise ValueError("the tensors are on GPU %d, the stream is of GPU %d"
                             % (dev, stream.device_index))
        return stream.cuda_stream
    if _raw_ready:
        return _raw_stream(torch._C._cuda_getDevice())
    handle = torch.cuda.current_stream().cuda_stream
    _raw_ready = _raw_stream is not None
    return handle


def _dtype_code(dt):
    if dt == torch.float32:
        return KDA_F32
    if dt == torch.bfloat16:
        return KDA_BF16
    raise ValueError("unsupported input dtype %s" % dt)


class StatePool:
    """fp32 states [num_slots][H][d_v][d_k] (each column of S contiguous)."""

    def __init__(self, data):
        assert data.dtype == torch.float32 and data.dim() == 4
        assert data.is_contiguous()
        self.data, self.dev = data, data.get_device()
        P, H, dv, dk = data.shape
        self.c = kda_state_pool(data.data_ptr(), P, H, dk, dv)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def zeros(cls, num_slots, H, d, device="cuda", d_v=None):
        return cls(torch.zeros(num_slots, H, d if d_v is None else d_v, d,
                               dtype=torch.float32, device=device))


class ReplayRing:
    """ReplaySSM ring for one pool: payload [P][H][depth][d] + ctrl [P][H][2]."""

    def __init__(self, num_slots, H, d, depth, dtype, device="cuda"):
        self.k = torch.zeros(num_slots, H, depth, d, dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.alpha = torch.zeros_like(self.k)
        self.beta = torch.zeros(num_slots, H, depth, dtype=dtype, device=device)
        self.ctrl = torch.zeros(num_slots, H, 2, dtype=torch.int32, device=device)
        self.depth = depth
        self.c = kda_replay_ring(self.k.data_ptr(), self.v.data_ptr(),
                                 self.alpha.data_ptr(), self.beta.data_ptr(),
                                 self.ctrl.data_ptr(), depth, _dtype_code(dtype))


class TokenBatch:
    """Packed tokens q, k, alpha [N][H][d_k], v [N][H][d_v], beta [N][H],
    fp32 outputs o [N][H][d_v] and cu_seqlens [B + 1] (int32, device)."""

    def __init__(self, q, k, v, alpha, beta, cu_seqlens, o=None):
        self.q, self.k, self.v, self.alpha, self.beta = q, k, v, alpha, beta
        self.cu_seqlens = cu_seqlens
        N, H, dk = k.shape
        dv = v.shape[2]
        self.o = o if o is not None else torch.empty(
            N, H, dv, dtype=torch.float32, device=k.device)
        for t in (q, k, v, alpha, beta, self.o, cu_seqlens):
            assert t.is_contiguous()
        self.c = kda_tokens(_dtype_code(k.dtype), q.data_ptr(), k.data_ptr(),
                            v.data_ptr(), alpha.data_ptr(), beta.data_ptr(),
                            self.o.data_ptr(), cu_seqlens.data_ptr(),
                            cu_seqlens.numel() - 1, N, H, dk, dv)


def kda_prefill_workspace_size(num_tokens, num_seqs, H, d_k, d_v, chunk, dtype):
    """Workspace bytes for these sizes and input dtype (KDA_F32 / KDA_BF16);
    0 when the call needs none."""
    return int(lib().kda_prefill_workspace_size(num_tokens, num_seqs, H, d_k,
                                                d_v, chunk, dtype))


def kda_prefill_chunked(tok, pool, state_slots, chunk, ckpt_every=0,
                        ckpt_slots=None, start_pos=None, workspace=None,
                        stream=None, single_pass=False, raw=False):
    """Chunked prefill; ckpt_slots [B][max_ckpt] int32 (device) or None.
    workspace None: one of the required size is allocated here;
    single_pass: pass no workspace (the tensor-core shape's single pass);
    raw: projection-space inputs, prep fused (kda_prefill_chunked_raw)."""
    max_ckpt = 0 if ckpt_slots is None else int(ckpt_slots.shape[1])
    if single_pass:
        workspace = None
    elif workspace is None:
        nbytes = kda_prefill_workspace_size(tok.c.num_tokens, tok.c.num_seqs,
                                            tok.c.num_heads, tok.c.d_k,
                                            tok.c.d_v, chunk, tok.c.dtype)
        if nbytes > 0:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=tok.k.device)
    fn, name = ((lib().kda_prefill_chunked_raw, "kda_prefill_chunked_raw") if raw
                else (lib().kda_prefill_chunked, "kda_prefill_chunked"))
    _check(fn(
        ctypes.byref(tok.c), ctypes.byref(pool.c), _ptr(state_slots),
        _ptr(ckpt_slots), max_ckpt, ckpt_every, chunk, _ptr(start_pos),
        _ptr(workspace), 0 if workspace is None else workspace.numel(),
        _stream(stream, pool.dev)), name)
    return workspace


KDA_NOALLOC_SCRATCH_BYTES = 64 << 20


def kda_prefill_chunked_noalloc(tok, pool, state_slots, chunk, ckpt_every=0,
                                ckpt_slots=None, start_pos=None, stream=None):
    """kda_prefill_chunked with the library's own fixed scratch instead of a
    workspace argument, for callers that cannot allocate device memory."""
    max_ckpt = 0 if ckpt_slots is None else int(ckpt_slots.shape[1])
    _check(lib().kda_prefill_chunked_noalloc(
        ctypes.byref(tok.c), ctypes.byref(pool.c), _ptr(state_slots),
        _ptr(ckpt_slots), max_ckpt, ckpt_every, chunk, _ptr(start_pos),
        _stream(stream, pool.dev)), "kda_prefill_chunked_noalloc")


def kda_verify(tok, max_T, pool, state_slots, ring, is_spec=None, stream=None,
               raw=False):
    """raw: projection-space keys, decay and beta logits, prep fused
    (kda_verify_raw)."""
    fn, name = ((lib().kda_verify_raw, "kda_verify_raw") if raw
                else (lib().kda_verify, "kda_verify"))
    _check(fn(ctypes.byref(tok.c), max_T, ctypes.byref(pool.c), _ptr(state_slots),
              ctypes.byref(ring.c), _ptr(is_spec), _stream(stream, pool.dev)), name)


def kda_forward_mixed(tok, num_prefill, prefill_tokens, pool, state_slots, chunk,
                      max_T, ring, ckpt_every=0, ckpt_slots=None, start_pos=None,
                      is_spec=None, workspace=None, single_pass=False, stream=None,
                      side_stream=None):
    """Prefill segments (the first num_prefill sequences, token rows
    [0, prefill_tokens)) and verify/decode segments of one packed batch in one
    call; side_stream: run the prefill part there, forked and joined."""
    max_ckpt = 0 if ckpt_slots is None else int(ckpt_slots.shape[1])
    if single_pass or num_prefill == 0:
        workspace = None
    elif workspace is None:
        nbytes = kda_prefill_workspace_size(prefill_tokens, num_prefill,
                                            tok.c.num_heads, tok.c.d_k, tok.c.d_v,
                                            chunk, tok.c.dtype)
        if nbytes > 0:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=tok.k.device)
    side = None if side_stream is None else ctypes.c_void_p(_stream(side_stream, pool.dev))
    _check(lib().kda_forward_mixed(
        ctypes.byref(tok.c), num_prefill, prefill_tokens, ctypes.byref(pool.c),
        _ptr(state_slots), _ptr(ckpt_slots), max_ckpt, ckpt_every, chunk,
        _ptr(start_pos), _ptr(workspace),
        0 if workspace is None else workspace.numel(), max_T,
        ctypes.byref(ring.c), _ptr(is_spec), _stream(stream, pool.dev), side),
        "kda_forward_mixed")
    return workspace


def kda_commit(accepted_len, state_slots, pool, ring, stream=None):
    _check(lib().kda_commit(_ptr(accepted_len), _ptr(state_slots),
                            state_slots.numel(), ctypes.byref(pool.c),
                            ctypes.byref(ring.c), _stream(stream, pool.dev)), "kda_commit")


def kda_commit_layers(accepted_len, state_slots, pool, rings, stream=None):
    """kda_commit on several layers' rings (same pool geometry), one launch."""
    arr = (kda_replay_ring * len(rings))(*[r.c for r in rings])
    _check(lib().kda_commit_layers(_ptr(accepted_len), _ptr(state_slots),
                                   state_slots.numel(), ctypes.byref(pool.c),
                                   arr, len(rings), _stream(stream, pool.dev)),
           "kda_commit_layers")


def kda_materialize(state_slots, pool, ring, stream=None):
    _check(lib().kda_materialize(_ptr(state_slots), state_slots.numel(),
                                 ctypes.byref(pool.c), ctypes.byref(ring.c),
                                 _stream(stream, pool.dev)), "kda_materialize")


def kda_ring_reset(slots, pool, ring, stream=None):
    _check(lib().kda_ring_reset(_ptr(slots), slots.numel(), ctypes.byref(pool.c),
                                ctypes.byref(ring.c), _stream(stream, pool.dev)),
           "kda_ring_reset")


def kda_gather_states(pool, slots, out=None, stream=None):
    if out is None:
        P, H, dv, dk = pool.data.shape
        out = torch.empty(slots.numel(), H, dv, dk, dtype=torch.float32,
                          device=pool.data.device)
    _check(lib().kda_gather_states(ctypes.byref(pool.c), _ptr(slots),
                                   slots.numel(), _ptr(out), _stream(stream, pool.dev)),
           "kda_gather_states")
    return out


def kda_copy_slots(pool, src, dst, stream=None):
    _check(lib().kda_copy_slots(ctypes.byref(pool.c), _ptr(src), _ptr(dst),
                                src.numel(), _stream(stream, pool.dev)), "kda_copy_slots")


def snapshot_buffer(num_seqs, max_T, pool):
    """Per-position snapshots [num_seqs][max_T][H][d_v][d_k] fp32 for
    kda_verify_snapshot (the direct design's extra state cache)."""
    P, H, dv, dk = pool.data.shape
    return torch.empty(num_seqs, max_T, H, dv, dk, dtype=torch.float32,
                       device=pool.data.device)


def kda_verify_snapshot(tok, max_T, pool, state_slots, snapshots, stream=None):
    _check(lib().kda_verify_snapshot(ctypes.byref(tok.c), max_T,
                                     ctypes.byref(pool.c), _ptr(state_slots),
                                     _ptr(snapshots), _stream(stream, pool.dev)),
           "kda_verify_snapshot")


def kda_commit_snapshot(accepted_len, state_slots, pool, snapshots, stream=None):
    _check(lib().kda_commit_snapshot(_ptr(accepted_len), _ptr(state_slots),
                                     state_slots.numel(), ctypes.byref(pool.c),
                                     _ptr(snapshots), int(snapshots.shape[1]),
                                     _stream(stream, pool.dev)), "kda_commit_snapshot")


def _row_view(t, dt, what):
    """Row stride of a token tensor [N][...] whose rows are contiguous."""
    if t.dtype != dt:
        raise ValueError("%s is %s, the batch %s" % (what, t.dtype, dt))
    inner = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != inner:
            raise ValueError("the rows of %s are not contiguous" % what)
        inner *= size
    return t.stride(0) if t.shape[0] > 1 else inner


def _same(what, got, want):
    if tuple(got) != tuple(want):
        raise ValueError("%s has shape %s, expected %s" % (what, tuple(got), tuple(want)))


def _param(t, shape, dt, what):
    if t is not None:
        _same(what, t.shape, shape)
        if t.dtype != dt or not t.is_contiguous():
            raise ValueError("%s must be contiguous %s" % (what, dt))
    return None if t is None else t.data_ptr()


def _together(home, tensors):
    """The device index of tensor `home`; all others (None: skipped) are there too."""
    dev = home.get_device()  # -1: not on a GPU, which the calls refuse
    for t, what in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("%s is on %s, the others on %s" % (what, t.device, home.device))
    return dev


def _cu(cu_seqlens, N):
    """Pointer and segments of cu_seqlens; None: one token a row (steps)."""
    if cu_seqlens is None:
        return None, N
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous int32")
    return cu_seqlens.data_ptr(), cu_seqlens.numel() - 1


def _table(t, n, what, dev):
    """Pointer of an int32 table of n entries on device dev (None: NULL)."""
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != n:
        raise ValueError("%s must be contiguous int32 with %d entries" % (what, n))
    if t.get_device() != dev or dev < 0:
        raise ValueError("%s is on %s, the call on GPU %d" % (what, t.device, dev))
    return t.data_ptr()


def _call_device(tok, pool):
    if tok.dev != pool.dev or tok.dev < 0:
        raise ValueError("the batch is on device %d, the pool on %d; both must be on one GPU"
                         % (tok.dev, pool.dev))
    return tok.dev


def _workspace(ws, dev):
    """Pointer and bytes of a workspace (None: NULL)."""
    if ws is None:
        return None, 0
    if not ws.is_contiguous() or ws.get_device() != dev or dev < 0:
        raise ValueError("a workspace is a contiguous tensor on the call's GPU")
    return ws.data_ptr(), ws.numel() * ws.element_size()


class ConvPool:
    """Convolution states [num_slots][W - 1][D]: each slot's last W - 1 inputs."""

    def __init__(self, data):
        if data.dim() != 3 or not data.is_contiguous():
            raise ValueError("a convolution pool is a contiguous [num_slots][W - 1][D]")
        self.data = data
        self.dev = data.get_device()
        P, taps, D = data.shape
        self.c = kda_conv_pool(data.data_ptr(), _dtype_code(data.dtype), P, D, taps + 1)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def zeros(cls, num_slots, width, D, dtype, device="cuda"):
        return cls(torch.zeros(num_slots, width - 1, D, dtype=dtype, device=device))


class ConvBatch:
    """Packed rows x [N][D] (a row stride is fine), weight [D][W], bias [D] or
    None, outputs y [N][D]; cu_seqlens [B + 1] int32, or None for steps of one
    token a row; activation None or "silu"."""

    def __init__(self, x, weight, bias=None, cu_seqlens=None, activation="silu", y=None):
        if activation not in (None, "silu"):
            raise ValueError("activation must be None or 'silu'")
        N, D = x.shape
        dt = x.dtype
        self.x, self.weight, self.bias, self.cu_seqlens = x, weight, bias, cu_seqlens
        self.y = y if y is not None else torch.empty(N, D, dtype=dt, device=x.device)
        _same("y", self.y.shape, (N, D))
        self.dev = _together(x, ((weight, "weight"), (bias, "bias"), (cu_seqlens, "cu_seqlens"),
                                 (self.y, "y")))
        W = weight.shape[1]
        cu, B = _cu(cu_seqlens, N)
        self.c = kda_conv_tokens(
            _dtype_code(dt), x.data_ptr(), self.y.data_ptr(), _row_view(x, dt, "x"),
            _row_view(self.y, dt, "y"), _param(weight, (D, W), dt, "weight"),
            _param(bias, (D,), dt, "bias"), cu, B, N, D, W, 1 if activation else 0)
        self.ref, self.num_seqs = ctypes.byref(self.c), B


class ScanPool:
    """Scan states fp32 [num_slots][D][S]."""

    def __init__(self, data):
        if data.dtype != torch.float32 or data.dim() != 3 or not data.is_contiguous():
            raise ValueError("a scan pool is a contiguous fp32 [num_slots][D][S]")
        self.data, self.dev = data, data.get_device()
        self.c = kda_scan_pool(data.data_ptr(), *data.shape)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def zeros(cls, num_slots, D, S, device="cuda"):
        return cls(torch.zeros(num_slots, D, S, dtype=torch.float32, device=device))


class ScanBatch:
    """Packed rows x, dt, z [N][D] and B, C [N][G][S] (row strides are fine),
    fp32 A [D][S], D [D], dt_bias [D], outputs y [N][D]; D, z, dt_bias may be
    None; cu_seqlens [B + 1] int32, or None for steps of one token a row."""

    def __init__(self, x, dt, A, B, C, D=None, z=None, dt_bias=None, cu_seqlens=None,
                 dt_softplus=True, y=None):
        N, Dm = x.shape
        _, G, S = B.shape
        ty, f32 = x.dtype, torch.float32
        self.x, self.dt, self.A, self.B, self.C = x, dt, A, B, C
        self.D, self.z, self.dt_bias, self.cu_seqlens = D, z, dt_bias, cu_seqlens
        self.y = y if y is not None else torch.empty(N, Dm, dtype=ty, device=x.device)
        for t, shape, what in ((dt, (N, Dm), "dt"), (z, (N, Dm), "z"), (B, (N, G, S), "B"),
                               (C, (N, G, S), "C"), (self.y, (N, Dm), "y")):
            if t is not None:
                _same(what, t.shape, shape)
        self.dev = _together(x, ((dt, "dt"), (A, "A"), (B, "B"), (C, "C"), (D, "D"), (z, "z"),
                                 (dt_bias, "dt_bias"), (cu_seqlens, "cu_seqlens"), (self.y, "y")))
        cu, nseq = _cu(cu_seqlens, N)
        self.c = kda_scan_tokens(
            _dtype_code(ty), x.data_ptr(), dt.data_ptr(),
            None if z is None else z.data_ptr(), B.data_ptr(), C.data_ptr(),
            self.y.data_ptr(), _row_view(x, ty, "x"), _row_view(dt, ty, "dt"),
            0 if z is None else _row_view(z, ty, "z"), _row_view(B, ty, "B"),
            _row_view(C, ty, "C"), _row_view(self.y, ty, "y"), _param(A, (Dm, S), f32, "A"),
            _param(D, (Dm,), f32, "D"), _param(dt_bias, (Dm,), f32, "dt_bias"), cu, nseq,
            N, Dm, S, G, 1 if dt_softplus else 0)
        self.ref, self.num_seqs = ctypes.byref(self.c), nseq


def _ckpt(ckpt_slots, B, dev):
    if ckpt_slots is None:
        return None, 0
    if ckpt_slots.dim() != 2:
        raise ValueError("ckpt_slots is [B][max_ckpt]")
    n = int(ckpt_slots.shape[1])
    return _table(ckpt_slots, B * n, "ckpt_slots", dev), n


def kda_conv_prefill(tok, pool, state_slots, ckpt_every=0, ckpt_slots=None, start_pos=None,
                     stream=None):
    """Causal convolution of packed prompts; ckpt_slots [B][max_ckpt] int32."""
    B, dev = tok.num_seqs, _call_device(tok, pool)
    ckpt, max_ckpt = _ckpt(ckpt_slots, B, dev)
    _check(lib().kda_conv_prefill(
        tok.ref, pool.ref, _table(state_slots, B, "state_slots", dev), ckpt, max_ckpt, ckpt_every,
        _table(start_pos, B, "start_pos", dev), _stream(stream, dev)), "kda_conv_prefill")


def kda_conv_step(tok, pool, state_slots, commit_len=None, stream=None):
    """Steps of one or a few tokens a row; commit_len [B] int32: how many of a
    row's tokens the stored state takes in (None: all)."""
    B, dev = tok.num_seqs, _call_device(tok, pool)
    st = (_lib or lib()).kda_conv_step(
        tok.ref, pool.ref, _table(state_slots, B, "state_slots", dev),
        None if commit_len is None else _table(commit_len, B, "commit_len", dev),
        _stream(stream, dev))
    if st:
        _check(st, "kda_conv_step")


def kda_scan_workspace_size(num_tokens, num_seqs, channels, state, groups=1):
    """Workspace bytes with which kda_scan_prefill splits long segments, enough
    for every batch of at most these tokens and segments; 0 when none is split."""
    return int(lib().kda_scan_workspace_size(num_tokens, num_seqs, channels, state, groups))


def scan_workspace(tok):
    """A workspace tensor for kda_scan_prefill of this batch and of smaller ones
    (None: not needed)."""
    n = kda_scan_workspace_size(tok.c.num_tokens, tok.c.num_seqs, tok.c.channels, tok.c.state,
                                tok.c.groups)
    return torch.empty(n, dtype=torch.uint8, device=tok.x.device) if n else None


def kda_scan_prefill(tok, pool, state_slots, ckpt_every=0, ckpt_slots=None, start_pos=None,
                     workspace=None, stream=None):
    """Selective scan of packed prompts; workspace: from scan_workspace(tok),
    or None: no segment is split."""
    B, dev = tok.num_seqs, _call_device(tok, pool)
    ckpt, max_ckpt = _ckpt(ckpt_slots, B, dev)
    ws, size = _workspace(workspace, dev)
    _check(lib().kda_scan_prefill(
        tok.ref, pool.ref, _table(state_slots, B, "state_slots", dev), ckpt, max_ckpt, ckpt_every,
        _table(start_pos, B, "start_pos", dev), ws, size, _stream(stream, dev)), "kda_scan_prefill")


def kda_scan_step(tok, pool, state_slots, commit_len=None, stream=None):
    """The scan's steps, commit_len as in kda_conv_step."""
    B, dev = tok.num_seqs, _call_device(tok, pool)
    st = (_lib or lib()).kda_scan_step(
        tok.ref, pool.ref, _table(state_slots, B, "state_slots", dev),
        None if commit_len is None else _table(commit_len, B, "commit_len", dev),
        _stream(stream, dev))
    if st:
        _check(st, "kda_scan_step")


class LinearBatch:
    """Packed rows q, k [N][Hk][d_k] and v [N][H][d_v] (row strides are fine), fp32
    log decays g [N][H] or [H] (every token's), outputs o [N][H][d_v], times scale;
    cu_seqlens [B + 1] int32, or None for steps of one token a row.  The states
    are a StatePool's."""

    def __init__(self, q, k, v, g, cu_seqlens=None, scale=1.0, o=None):
        N, Hk, dk = q.shape
        _, H, dv = v.shape
        ty = q.dtype
        self.q, self.k, self.v, self.g, self.cu_seqlens = q, k, v, g, cu_seqlens
        self.o = o if o is not None else torch.empty(N, H, dv, dtype=ty, device=q.device)
        _same("k", k.shape, q.shape)
        _same("v", v.shape, (N, H, dv))
        _same("o", self.o.shape, (N, H, dv))
        _same("g", g.shape, (H,) if g.dim() == 1 else (N, H))
        if g.dim() == 1:
            if g.dtype != torch.float32 or not g.is_contiguous():
                raise ValueError("g must be fp32, and contiguous where it is [H]")
            g_stride = 0
        else:
            g_stride = _row_view(g, torch.float32, "g")
            if g_stride < H:
                raise ValueError("g of one row for all tokens is passed as [H]")
        self.dev = _together(q, ((k, "k"), (v, "v"), (g, "g"), (cu_seqlens, "cu_seqlens"),
                                 (self.o, "o")))
        cu, nseq = _cu(cu_seqlens, N)
        self.c = kda_linear_tokens(
            _dtype_code(ty), q.data_ptr(), k.data_ptr(), v.data_ptr(), self.o.data_ptr(),
            _row_view(q, ty, "q"), _row_view(k, ty, "k"), _row_view(v, ty, "v"),
            _row_view(self.o, ty, "o"), g.data_ptr(), g_stride, scale, cu, nseq, N, H, Hk, dk, dv)
        self.ref, self.num_seqs = ctypes.byref(self.c), nseq


def kda_linear_workspace_size(num_tokens, num_seqs, H, d_k, d_v, dtype):
    """Workspace bytes with which kda_linear_prefill splits long segments, enough
    for every batch of at most these tokens and segments (dtype KDA_F32 or
    KDA_BF16); 0 when none is split."""
    return int(lib().kda_linear_workspace_size(num_tokens, num_seqs, H, d_k, d_v, dtype))


def linear_workspace(tok):
    """A workspace tensor for kda_linear_prefill of this batch and of smaller ones
    (None: not needed).  A few prompts of like lengths whose heads fill the GPU are
    faster without one."""
    c = tok.c
    n = kda_linear_workspace_size(c.num_tokens, c.num_seqs, c.num_heads, c.d_k, c.d_v, c.dtype)
    return torch.empty(n, dtype=torch.uint8, device=tok.q.device) if n else None


def kda_linear_prefill(tok, pool, state_slots, ckpt_every=0, ckpt_slots=None, start_pos=None,
                       workspace=None, stream=None):
    """Linear attention of packed prompts; workspace: from linear_workspace(tok),
    or None: no segment is split."""
    B, dev = tok.num_seqs, _call_device(tok, pool)
    ckpt, max_ckpt = _ckpt(ckpt_slots, B, dev)
    ws, size = _workspace(workspace, dev)
    _check(lib().kda_linear_prefill(
        tok.ref, pool.ref, _table(state_slots, B, "state_slots", dev), ckpt, max_ckpt, ckpt_every,
        _table(start_pos, B, "start_pos", dev), ws, size, _stream(stream, dev)),
        "kda_linear_prefill")


def kda_linear_step(tok, pool, state_slots, commit_len=None, stream=None):
    """Steps of one or a few tokens a row, commit_len as in kda_conv_step."""
    B, dev = tok.num_seqs, _call_device(tok, pool)
    st = (_lib or lib()).kda_linear_step(
        tok.ref, pool.ref, _table(state_slots, B, "state_slots", dev),
        None if commit_len is None else _table(commit_len, B, "commit_len", dev),
        _stream(stream, dev))
    if st:
        _check(st, "kda_linear_step")


_NORMS = {None: KDA_NORM_NONE, "rms": KDA_NORM_RMS, "l2": KDA_NORM_L2}


class QKBatch:
    """Queries q [N][Hq][d] and keys k [N][Hk][d] (row strides are fine; either may
    be None), weights [d] or None, norm "rms", "l2" or None; cos_sin fp32
    [max_pos][rot_dim] (cosines, then sines) with positions [N] int32, or None: no
    rotation; interleaved: neighbours turn, else halves; the queries times q_scale.
    Outputs q_out, k_out may be the inputs."""

    def __init__(self, q, k, q_weight=None, k_weight=None, norm="rms", eps=1e-6, cos_sin=None,
                 positions=None, interleaved=False, q_scale=1.0, q_out=None, k_out=None):
        if norm not in _NORMS:
            raise ValueError("norm must be 'rms', 'l2' or None")
        if (cos_sin is None) != (positions is None):
            raise ValueError("cos_sin and positions go together")
        one = q if q is not None else k
        N, _, d = one.shape
        ty = one.dtype
        if q is not None and k is not None:
            _same("k", k.shape, (N, k.shape[1], d))

        def rows(x, out, weight, what):
            if x is None:
                return None, (None, 0, None, 0, None, 0)
            if out is None:
                out = torch.empty(x.shape, dtype=ty, device=x.device)
            _same(what + "_out", out.shape, x.shape)
            return out, (x.data_ptr(), _row_view(x, ty, what), out.data_ptr(),
                         _row_view(out, ty, what + "_out"),
                         _param(weight, (d,), ty, what + "_weight"), x.shape[1])

        self.q, self.k, self.q_weight, self.k_weight = q, k, q_weight, k_weight
        self.cos_sin, self.positions = cos_sin, positions
        self.q_out, a = rows(q, q_out, q_weight, "q")
        self.k_out, b = rows(k, k_out, k_weight, "k")
        rot = max_pos = 0
        if cos_sin is not None:
            max_pos, rot = cos_sin.shape
            _param(cos_sin, (max_pos, rot), torch.float32, "cos_sin")
        self.dev = _together(one, ((q, "q"), (k, "k"), (self.q_out, "q_out"),
                                   (self.k_out, "k_out"), (q_weight, "q_weight"),
                                   (k_weight, "k_weight"), (cos_sin, "cos_sin")))
        self.c = kda_qk_tokens(
            _dtype_code(ty), a[0], b[0], a[2], b[2], a[1], b[1], a[3], b[3], a[4], b[4],
            None if cos_sin is None else cos_sin.data_ptr(),
            _table(positions, N, "positions", self.dev), N, a[5], b[5], d, rot, max_pos,
            1 if interleaved else 0, _NORMS[norm], eps, q_scale)
        self.ref = ctypes.byref(self.c)


def _on_gpu(tok):
    if tok.dev < 0:
        raise ValueError("the batch is not on a GPU")


def kda_qk_norm(tok, stream=None):
    """Norm, rotation and scale of queries and keys: into tok.q_out, tok.k_out."""
    _on_gpu(tok)
    st = (_lib or lib()).kda_qk_norm(tok.ref, _stream(stream, tok.dev))
    if st:
        _check(st, "kda_qk_norm")


class GateBatch:
    """A layer's outputs x [N][H][d], their gate [N][H][d] or None, weight [d] or
    None, activation "sigmoid" or "silu", outputs y [N][H][d] in the gate's dtype
    (without a gate: the weight's, else x's); row strides are fine, and y may be
    the gate, or x of the same dtype."""

    def __init__(self, x, gate, weight=None, activation="sigmoid", eps=1e-6, y=None):
        if activation not in ("sigmoid", "silu"):
            raise ValueError("activation must be 'sigmoid' or 'silu'")
        N, H, d = x.shape
        like = next(t for t in (gate, weight, x) if t is not None)
        ty = like.dtype
        self.x, self.gate, self.weight = x, gate, weight
        self.y = y if y is not None else torch.empty(N, H, d, dtype=ty, device=x.device)
        _same("y", self.y.shape, (N, H, d))
        if gate is not None:
            _same("gate", gate.shape, (N, H, d))
        self.dev = _together(x, ((gate, "gate"), (weight, "weight"), (self.y, "y")))
        self.c = kda_gate_tokens(
            _dtype_code(x.dtype), _dtype_code(ty), x.data_ptr(),
            None if gate is None else gate.data_ptr(), _param(weight, (d,), ty, "weight"),
            self.y.data_ptr(), _row_view(x, x.dtype, "x"),
            0 if gate is None else _row_view(gate, ty, "gate"), _row_view(self.y, ty, "y"),
            N, H, d, 1 if activation == "silu" else 0, eps)
        self.ref = ctypes.byref(self.c)


def kda_gated_norm(tok, stream=None):
    """Norm of each head's outputs times the gate's activation: into tok.y."""
    _on_gpu(tok)
    st = (_lib or lib()).kda_gated_norm(tok.ref, _stream(stream, tok.dev))
    if st:
        _check(st, "kda_gated_norm")


class SlotArrays:
    """The per-slot tensors [num_slots][...] of a model (pools, rings, of all
    layers) that kda_move_slots moves together: up to 64, whose slots are each a
    multiple of 4 bytes.  A model of more takes one SlotArrays for each 64."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        if not self.tensors or self.tensors[0].shape[0] < 1:
            raise ValueError("no arrays, or no slots")
        self.num_slots = int(self.tensors[0].shape[0])
        self.dev = _together(self.tensors[0], [(t, "an array") for t in self.tensors])
        for t in self.tensors:
            if not t.is_contiguous() or t.shape[0] != self.num_slots:
                raise ValueError("every array is a contiguous [num_slots][...]")
        self.c = (kda_slot_array * len(self.tensors))(
            *[kda_slot_array(t.data_ptr(), t.numel() // self.num_slots * t.element_size())
              for t in self.tensors])


def kda_move_workspace_size(arrays, n):
    return int(lib().kda_move_workspace_size(arrays.c, len(arrays.tensors), n))


def move_workspace(arrays, n):
    """A workspace tensor for kda_move_slots of up to n moves."""
    return torch.empty(max(1, kda_move_workspace_size(arrays, n)), dtype=torch.uint8,
                       device=arrays.tensors[0].device)


def kda_move_slots(arrays, src, dst, workspace=None, stream=None):
    """In every array: slot dst[i] receives slot src[i] (src < 0: zeros, dst < 0:
    nothing).  workspace None: src and dst must be disjoint."""
    n, dev = dst.numel(), arrays.dev
    ws, size = _workspace(workspace, dev)
    st = (_lib or lib()).kda_move_slots(
        arrays.c, len(arrays.tensors), arrays.num_slots, _table(src, n, "src", dev),
        _table(dst, n, "dst", dev), n, ws, size, _stream(stream, dev))
    if st:
        _check(st, "kda_move_slots")


def kda_get_device_error(stream=None):
    """Synchronize, read and clear the device error word; returns its bits."""
    bits = _I32(0)
    st = lib().kda_get_device_error(ctypes.byref(bits), _stream(stream))
    if st not in (KDA_OK, KDA_EDEVICE):
        raise KdaError(st, "kda_get_device_error")
    return int(bits.value)


def kda_set_wait_limit(polls):
    """Testing hook: bounded device waits give up after `polls` polls
    (KDA_DERR_TIMEOUT); a negative value restores the default."""
    _check(lib().kda_set_wait_limit(int(polls)), "kda_set_wait_limit")
