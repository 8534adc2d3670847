"""Refusals of the products' and norms' wrappers that depend on devices and counts, with host tensors that
report a device of their own; no call gets past the wrapper."""

import pytest
import torch

import quantized_routed_expert_sigmoid_gb300 as moe


class _On(torch.Tensor):
    """A host tensor that says that it lies on GPU `index`."""

    index = 0
    is_cuda = True

    def get_device(self):
        return self.index


def _on(t, index=0):
    t = t.as_subclass(_On)
    t.index = index
    return t


@pytest.fixture
def ops(monkeypatch):
    """The three operators over tensors of GPU 0, which is current; their C calls are recorded, not made."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    calls = []
    monkeypatch.setattr(moe.layer.N, "moe_norm_residual",
                        lambda *a: calls.append(a))
    g = moe.GroupedExperts(_on(torch.zeros(2, 16, 32, dtype=torch.bfloat16)))
    w = moe.W4Experts(_on(torch.zeros(2, 16, 16, dtype=torch.uint8)), _on(torch.zeros(2, 16, 1, dtype=torch.float16)), group=32)
    for op in (g, w):
        op._matmul = lambda *a: calls.append(a)
    return g, w, moe.NormResidual(32, gamma_pre=_on(torch.ones(32))), calls


def _args(**index):
    at = lambda name: index.get(name, 0)
    return dict(x=_on(torch.zeros(4, 32, dtype=torch.bfloat16), at("x")),
                offsets=_on(torch.zeros(3, dtype=torch.int32), at("offsets")),
                sorted_pairs=_on(torch.zeros(8, dtype=torch.int32), at("sorted_pairs")), k=2,
                out=_on(torch.zeros(8, 16), at("out")), status=_on(torch.zeros(1, dtype=torch.int32), at("status")))


@pytest.mark.parametrize("which", [0, 1])
def test_products_on_one_device_are_called(ops, which):
    ops[which](**_args())
    assert len(ops[3]) == 1


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("name", ["x", "offsets", "sorted_pairs", "out", "status"])
def test_products_refuse_a_tensor_of_another_device(ops, which, name):
    with pytest.raises(ValueError, match=name):
        ops[which](**_args(**{name: 1}))
    assert not ops[3]


@pytest.mark.parametrize("which", [0, 1])
def test_products_refuse_weights_of_a_device_that_is_not_current(ops, which, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        ops[which](**_args())
    assert not ops[3]


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("k", [0, -1])
def test_products_refuse_a_count_of_experts_below_one(ops, which, k):
    with pytest.raises(ValueError, match="k = "):
        ops[which](**dict(_args(), k=k))
    with pytest.raises(ValueError, match="k = "):
        ops[which](_args()["x"], k=k)
    assert not ops[3]


def test_plans_refuse_matrices_of_two_devices(ops):
    w = torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="w_up"):
        moe.GroupedExperts(_on(w), _on(w.clone(), 1))
    q, s = torch.zeros(2, 16, 16, dtype=torch.uint8), torch.zeros(2, 16, 1, dtype=torch.float16)
    with pytest.raises(ValueError, match="scales"):
        moe.W4Experts(_on(q), _on(s, 1), group=32)
    with pytest.raises(ValueError, match="gamma"):
        moe.NormResidual(32, gamma_post=_on(torch.ones(32)), gamma_pre=_on(torch.ones(32), 1))


def _norm_args(**index):
    at = lambda name: index.get(name, 0)
    return dict(x=_on(torch.zeros(4, 32), at("x")), y=_on(torch.zeros(4, 32), at("y")),
                gate=_on(torch.zeros(32), at("gate")), x_out=_on(torch.zeros(4, 32), at("x_out")),
                u=_on(torch.zeros(4, 32, dtype=torch.bfloat16), at("u")))


def test_norm_on_one_device_is_called(ops):
    ops[2](**_norm_args())
    assert len(ops[3]) == 1


@pytest.mark.parametrize("name", ["x", "y", "gate", "x_out", "u"])
def test_norm_refuses_a_tensor_of_another_device(ops, name):
    with pytest.raises(ValueError, match="device" if name == "y" else name):
        ops[2](**_norm_args(**{name: 1}))
    assert not ops[3]


def test_norm_refuses_a_device_that_is_not_current(ops, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        ops[2](**_norm_args())
    with pytest.raises(ValueError, match="gamma"):       # all of the call's on the current one, the gains are not
        ops[2](**_norm_args(x=1, y=1, gate=1, x_out=1, u=1))
    assert not ops[3]
