"""Every call runs with its tensors' device current and, where no stream is named, on that device's current
stream: a plan and the decode behind it must not part when another device is current."""

from __future__ import annotations

import contextlib

import pytest
import torch

import mla_decode_attention_etap_b200 as m

BF16, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


class _Device:
    def __init__(self, index):
        self.index = index

    def __eq__(self, other):
        return isinstance(other, _Device) and other.index == self.index


class _Stream:
    def __init__(self, address, device=None):
        self.cuda_stream = address
        if device is not None:
            self.device = device


@pytest.fixture
def fake_cuda(monkeypatch):
    """A process whose current device is 0; device i's current stream has the address 100 + i."""
    now = [0]

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d.index
        yield
        now[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    return now


@pytest.mark.parametrize("index", [0, 1])
def test_launch_follows_the_tensors_device(fake_cuda, index):
    seen = []
    m._launch(_Device(index), None, lambda s: seen.append((fake_cuda[0], s)) or 0, "call")
    m._launch(_Device(index), _Stream(7, _Device(index)), lambda s: seen.append((fake_cuda[0], s)) or 0, "call")
    m._launch(_Device(index), _Stream(8), lambda s: seen.append((fake_cuda[0], s)) or 0, "call")  # names no device
    assert seen == [(index, 100 + index), (index, 7), (index, 8)] and fake_cuda[0] == 0


def test_launch_refuses_another_devices_stream(fake_cuda):
    with pytest.raises(ValueError, match="stream on"):
        m._launch(_Device(1), _Stream(7, _Device(0)), lambda s: 0, "call")


def _calls():
    B, q_len, h = 2, 4, 16
    q = torch.zeros(B, q_len, h, 576, dtype=BF16)
    kv, kv8, scale = torch.zeros(B, 64, 576, dtype=BF16), torch.zeros(B, 64, 576, dtype=U8), torch.ones(B, 64)
    lens, mask = torch.full((B,), 9, dtype=I32), torch.zeros(B, q_len, 1, dtype=I32)
    o, lse = torch.zeros(B, q_len, h, 512, dtype=BF16), torch.zeros(B, q_len, h)
    ws, err = torch.zeros(1 << 20, dtype=U8), torch.zeros(1, dtype=I32)
    return {
        "mla_decode_plan": lambda s: m.mla_decode_plan(lens, q_len, h, ws, 148, s),
        "mla_decode_fwd": lambda s: m.mla_decode_fwd(q, kv, lens, None, 0.1, 0, o, lse, ws, 148, 0, s),
        "mla_decode_fwd_ragged": lambda s: m.mla_decode_fwd(q, kv, lens, None, 0.1, 0, o, lse, ws, 148, 0, s, lens),
        "mla_decode_fwd_fp8": lambda s: m.mla_decode_fwd_fp8(q, kv8, scale, lens, None, 0.1, 0, o, lse, ws, 148, 0, s),
        "mla_decode_fwd_untransposed":
            lambda s: m.mla_decode_fwd_untransposed(q, kv, lens, None, 0.1, 0, o, lse, ws, 148, 0, s),
        "mla_decode_fwd_trace": lambda s: m.mla_decode_fwd_trace(q, kv, lens, None, 0.1, 0, o, lse, ws, 148,
                                                                 m.trace_buffer(8, 148), s),
        "mla_decode_fwd_tree": lambda s: m.mla_decode_fwd_tree(q, kv, lens, None, 0.1, mask, o, lse, ws, 148, 0, s),
        "mla_decode_fwd_tree_fp8":
            lambda s: m.mla_decode_fwd_tree_fp8(q, kv8, scale, lens, None, 0.1, mask, o, lse, ws, 148, 0, s),
        "mla_combine": lambda s: m.mla_combine(ws, B, q_len, h, 148, o, lse, s),
        "mla_decode_read_status": lambda s: m.mla_decode_read_status(ws, s),
        "mla_stream_probe": lambda s: m.mla_stream_probe(kv, 2, err, s),
        "mla_form_ablation": lambda s: m.mla_form_ablation(0, 16, 1, 1, torch.zeros(2, dtype=I64), err, s),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_every_call_goes_through_the_launch(monkeypatch, name):
    seen = []
    monkeypatch.setattr(m, "_require_cuda", lambda t, what: None)
    monkeypatch.setattr(m, "_launch", lambda device, stream, call, what: seen.append((device, stream, what)))
    _calls()[name]("a stream")
    assert seen == [(torch.device("cpu"), "a stream", name)]
