"""Calls launch on the current device: tensors or a stream of another one are refused
before anything is enqueued.  The library and the devices are stand-ins here."""
import types

import pytest
import torch

from recurrent_kda_state_gb300 import kda as K


class Library:
    """Counts the calls that reach it; every one succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    """The calls under GPU 0 as the current device; tables and workspaces pass."""
    stub = Library()
    monkeypatch.setattr(K, "_lib", stub)
    monkeypatch.setattr(K, "lib", lambda: stub)
    monkeypatch.setattr(K, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(K, "_table", lambda *a: None)
    monkeypatch.setattr(K, "_workspace", lambda *a: (None, 0))
    monkeypatch.setattr(K, "_raw_ready", True)
    monkeypatch.setattr(K, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return stub


def calls():
    """(name, call(dev, stream)): each call with all its tensors on GPU dev."""
    i32, q, v = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 16), torch.zeros(4, 2, 16)
    x, f = torch.zeros(4, 32), torch.zeros
    linear, norm, gate = K.LinearBatch(q, q.clone(), v, f(4, 2)), K.QKBatch(q, q.clone()), K.GateBatch(v, v.clone())
    conv, taps = K.ConvBatch(x, f(32, 4)), K.ConvPool.zeros(4, 4, 32, torch.float32, device="cpu")
    scan = K.ScanBatch(x, x.clone(), f(32, 16), f(4, 1, 16), f(4, 1, 16))
    hidden, states = K.ScanPool.zeros(4, 32, 16, device="cpu"), K.StatePool.zeros(4, 2, 16, device="cpu")
    arrays, cu = K.SlotArrays([f(4, 8)]), torch.tensor([0, 4], dtype=torch.int32)
    tok = K.TokenBatch(q, q.clone(), v, q.clone(), f(4, 2), cu)
    ring = K.ReplayRing(4, 2, 16, 4, torch.float32, device="cpu")
    snaps = f(4, 2, 2, 16, 16)
    owners = (linear, norm, gate, conv, taps, scan, hidden, states, arrays)

    def on(call):
        def run(dev, stream):
            for o in owners:
                o.dev = dev
            return call(stream)
        return run
    for name, call in (
            ("kda_linear_prefill", lambda s: K.kda_linear_prefill(linear, states, i32, stream=s)),
            ("kda_linear_step", lambda s: K.kda_linear_step(linear, states, i32, stream=s)),
            ("kda_qk_norm", lambda s: K.kda_qk_norm(norm, stream=s)),
            ("kda_gated_norm", lambda s: K.kda_gated_norm(gate, stream=s)),
            ("kda_conv_prefill", lambda s: K.kda_conv_prefill(conv, taps, i32, stream=s)),
            ("kda_conv_step", lambda s: K.kda_conv_step(conv, taps, i32, stream=s)),
            ("kda_scan_prefill", lambda s: K.kda_scan_prefill(scan, hidden, i32, stream=s)),
            ("kda_scan_step", lambda s: K.kda_scan_step(scan, hidden, i32, stream=s)),
            ("kda_move_slots", lambda s: K.kda_move_slots(arrays, i32, i32, stream=s)),
            ("kda_prefill_chunked", lambda s: K.kda_prefill_chunked(tok, states, i32, 64, single_pass=True, stream=s)),
            ("kda_prefill_chunked_noalloc", lambda s: K.kda_prefill_chunked_noalloc(tok, states, i32, 64, stream=s)),
            ("kda_verify", lambda s: K.kda_verify(tok, 4, states, i32, ring, stream=s)),
            ("kda_forward_mixed", lambda s: K.kda_forward_mixed(tok, 0, 0, states, i32, 64, 4, ring, stream=s)),
            ("kda_forward_mixed", lambda s: K.kda_forward_mixed(tok, 0, 0, states, i32, 64, 4, ring, stream=s,
                                                                side_stream=s)),
            ("kda_commit", lambda s: K.kda_commit(i32, i32, states, ring, stream=s)),
            ("kda_commit_layers", lambda s: K.kda_commit_layers(i32, i32, states, [ring], stream=s)),
            ("kda_materialize", lambda s: K.kda_materialize(i32, states, ring, stream=s)),
            ("kda_ring_reset", lambda s: K.kda_ring_reset(i32, states, ring, stream=s)),
            ("kda_gather_states", lambda s: K.kda_gather_states(states, i32, stream=s)),
            ("kda_copy_slots", lambda s: K.kda_copy_slots(states, i32, i32, stream=s)),
            ("kda_verify_snapshot", lambda s: K.kda_verify_snapshot(tok, 2, states, i32, snaps, stream=s)),
            ("kda_commit_snapshot", lambda s: K.kda_commit_snapshot(i32, i32, states, snaps, stream=s))):
        yield name, on(call)


def stream(dev):
    return types.SimpleNamespace(cuda_stream=0, device_index=dev)


def test_tensors_of_another_device_are_refused(lib):
    for name, call in calls():
        for s in (None, stream(0), stream(1)):
            with pytest.raises(ValueError, match="current device"):
                call(1, s)
        assert not lib.calls, name


def test_streams_of_another_device_are_refused(lib):
    for name, call in calls():
        with pytest.raises(ValueError, match="stream"):
            call(0, stream(1))
        assert not lib.calls, name


def test_calls_on_the_current_device_pass(lib):
    for name, call in calls():
        for s in (None, stream(0)):
            call(0, s)
            assert lib.calls == [name]
            lib.calls.clear()
