"""The wrappers of the dense product, layer norm and balance loss: devices, shapes and the streams of what a call makes for
itself, with host tensors that report a device of their own; the library's calls are recorded."""
from __future__ import annotations

import contextlib

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe
from test_products_devices import _On, _on

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def ops(monkeypatch):
    """(linear, norm, balance, recorded calls, streams under which torch.empty was called); GPU 0 is the current device."""
    under, made, calls = ["current"], [], []

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield
        under.pop()

    N = moe.layer.N
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(N, "_stream", lambda s: 5 if s is None else getattr(s, "cuda_stream", s))
    for name in ("moe_linear", "moe_layer_norm", "moe_layer_norm_backward", "moe_balance_loss"):
        monkeypatch.setattr(N, name, lambda *a, _n=name: calls.append((_n, a)))
    linear = moe.Linear(_on(torch.zeros(16, 32, dtype=BF)), _on(torch.zeros(16)))
    norm = moe.LayerNorm(32, gamma=_on(torch.ones(32)), beta=_on(torch.ones(32)))
    balance = moe.BalanceLoss(8, 2, device="cpu")
    balance._status = _on(balance._status)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (made.append(under[-1]), _on(empty(*a, **kw)))[1])
    return linear, norm, balance, calls, made


def _x(dtype=F32, index=0, width=32):
    return _on(torch.zeros(4, width, dtype=dtype), index)


def _calls(ops, stream=None, **other):
    linear, norm, balance, _, _ = ops
    i = lambda name: other.get(name, 0)  # noqa: E731
    return {
        "linear": lambda: linear(_x(BF, i("x")), residual=_x(F32, i("residual"), 16), stream=stream),
        "norm": lambda: norm(_x(F32, i("x")), stream=stream),
        "backward": lambda: norm.backward(_x(BF, i("dy")), _x(F32, i("x")), _on(torch.zeros(4), i("mean")), _on(torch.zeros(4)),
                                          add=_x(F32, i("add")), stream=stream),
        "balance": lambda: balance(_x(F32, i("x"), 8), _on(torch.zeros(4, 2, dtype=I32), i("ids")), dlogits=True,
                                   mask=_on(torch.ones(4, dtype=torch.bool), i("mask")), stream=stream),
    }


@pytest.mark.parametrize("name, made", [("linear", 1), ("norm", 3), ("backward", 4), ("balance", 4)])
def test_what_a_call_makes_is_of_its_stream(ops, name, made):
    s = _Stream(77)
    for stream, want in ((None, "current"), (s, s), (77, ("external", 77)), (0, "default"), (1, "default")):
        ops[4].clear()
        _calls(ops, stream)[name]()
        assert ops[4] == [want] * made, (stream, ops[4])
    assert len(ops[3]) == 5 and ops[3][2][1][-1] == 77


@pytest.mark.parametrize("name, tensor", [("linear", "x"), ("linear", "residual"), ("norm", "x"), ("backward", "x"), ("backward", "dy"),
                                          ("backward", "mean"), ("backward", "add"), ("balance", "x"), ("balance", "ids"),
                                          ("balance", "mask")])
def test_tensors_of_another_device_are_refused(ops, monkeypatch, name, tensor):
    with pytest.raises(ValueError, match="device 1"):
        _calls(ops, **{tensor: 1})[name]()
    assert not ops[3]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        _calls(ops)[name]()
    assert not ops[3]


def test_wrong_shapes_and_types_are_named(ops):
    linear, norm, balance, calls, _ = ops
    for fn, word in [
        (lambda: linear(_x(F32)), "x must be"), (lambda: linear(_x(BF, width=24)), "x must be"),
        (lambda: linear(_x(BF), residual=_x(F32, width=15)), "residual"), (lambda: linear(_x(BF), residual=_x(I32, width=16)), "residual"),
        (lambda: linear(_x(BF), out=_x(F32, width=16)), "out"), (lambda: linear(_x(BF), status=_x(F32)), "status"),
        (lambda: norm(_x(F32, width=31)), "x must be"), (lambda: norm(_x(), out=_x(I32)), "out must be"),
        (lambda: norm(_x(), mean=_on(torch.zeros(5))), "mean"), (lambda: norm.backward(_x(), _x(), None, None), "forward call"),
        (lambda: norm.backward(_x(), _x(), _on(torch.zeros(4)), _on(torch.zeros(4)), add=_x(BF)), "x's type"),
        (lambda: norm.backward(_x(), _x(), _on(torch.zeros(4)), _on(torch.zeros(4)), dx=_x(BF)), "x's type"),
        (lambda: norm.backward(_x(), _x(), _on(torch.zeros(4)), _on(torch.zeros(4)), accumulate=True), "given"),
        (lambda: norm.backward(_x(), _x(), _on(torch.zeros(4)), _on(torch.zeros(4)), dgamma=_on(torch.zeros(31))), "dgamma"),
        (lambda: balance(_x(BF, width=8), None), "logits"), (lambda: balance(_x(width=8), None), "ids"),
        (lambda: balance(_x(width=8), _on(torch.zeros(4, 3, dtype=I32))), "ids"),
        (lambda: balance(_x(width=8), _on(torch.zeros(4, 2, dtype=I32)), offsets=_on(torch.zeros(1, dtype=I32))), "offsets"),
        (lambda: balance(_x(width=8), _on(torch.zeros(4, 2, dtype=I32)), mask=_on(torch.zeros(3, dtype=torch.bool))), "mask"),
        (lambda: balance(_x(width=8), _on(torch.zeros(4, 2, dtype=I32)), upstream=_on(torch.zeros(2))), "upstream"),
        (lambda: balance(_x(width=8), _on(torch.zeros(4, 2, dtype=I32)), dlogits=True, accumulate=True), "given"),
        (lambda: balance(_x(width=8), _on(torch.zeros(4, 2, dtype=I32)), dlogits=_x(width=7)), "dlogits"),
    ]:
        with pytest.raises(ValueError, match=word):
            fn()
    assert not calls


def test_a_calls_own_word_unless_one_is_given(ops):
    linear, _, balance, calls, _ = ops
    given = _on(torch.zeros(1, dtype=I32))
    linear(_x(BF))
    linear(_x(BF), status=given)
    balance(_x(width=8), _on(torch.zeros(4, 2, dtype=I32)), status=given)
    assert calls[0][1][9] is linear._status and calls[1][1][9] is given and calls[2][1][13] is given
