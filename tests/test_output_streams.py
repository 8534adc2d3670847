"""Outputs that a call makes for itself belong to the stream that it runs on (host tensors, recorded calls)."""
from __future__ import annotations

import contextlib

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from test_products_devices import _On, _on


class _Stream:
    """Something with a stream's handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def made(monkeypatch):
    """(the four wrappers, the list of the streams under which torch.empty was called)."""
    under, log = ["current"], []

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield
        under.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    g = moe.GroupedExperts(_on(torch.zeros(2, 16, 32, dtype=torch.bfloat16)))
    w = moe.W4Experts(_on(torch.zeros(2, 16, 16, dtype=torch.uint8)), _on(torch.zeros(2, 16, 1, dtype=torch.float16)), group=32)
    for op in (g, w):
        op._matmul = lambda *a: None
    layer = moe.MoeLayer.__new__(moe.MoeLayer)
    layer.plan, layer.H, layer.ws, layer.ws_T = 0, 32, None, -1
    layer.workspace_bytes = lambda T: 64
    monkeypatch.setattr(moe.layer.N, "moe_norm_residual", lambda *a: None)
    monkeypatch.setattr(moe.layer.N, "moe_layer", lambda *a: None)
    monkeypatch.setattr(moe.layer.N, "_stream", lambda s: 5 if s is None else getattr(s, "cuda_stream", s))
    monkeypatch.setattr(_On, "record_stream", lambda self, s: log.append(("used by", s)), raising=False)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (log.append(under[-1]), _on(empty(*a, **kw)))[1])
    return dict(grouped=g, w4=w, norm=moe.NormResidual(32, gamma_pre=_on(torch.ones(32))), layer=layer), log


def _call(name, op, stream):
    x = _on(torch.zeros(4, 32, dtype=torch.float32 if name == "norm" else torch.bfloat16))
    if name == "norm":
        op(x, x, stream=stream)
    elif name == "layer":
        op(x, stream=stream)
    else:
        op(x, _on(torch.zeros(3, dtype=torch.int32)), stream=stream)


@pytest.mark.parametrize("name, n", [("grouped", 1), ("w4", 1), ("norm", 2), ("layer", 2)])
def test_outputs_are_made_under_the_call_s_stream(made, name, n):
    ops, log = made
    s = _Stream(77)
    for stream, want in ((None, "current"), (s, s), (77, ("external", 77)), (0, "default"), (1, "default")):
        log.clear()
        ops["layer"].ws = None
        _call(name, ops[name], stream)
        assert log == [want] * n, (stream, log)


def test_a_workspace_of_another_stream_is_kept_from_its_memory_until_the_call_is_done(made):
    ops, log = made
    layer, x = ops["layer"], _on(torch.zeros(4, 32, dtype=torch.bfloat16))
    layer(x)
    log.clear()
    layer(x, stream=77)
    layer(x)
    assert log == [("external", 77), ("used by", ("external", 77)), "current"]
