"""Calls of the operators around the routed experts that the binding refuses (no GPU needed)."""
import pytest
import torch

import dequant_iqk_moe_amd as q
from test_block_host import Fake

F32, I8, I32 = torch.float32, torch.int8, torch.int32


def _weights():
    w = q.Int8Weights(torch.zeros(2, 4, 16, dtype=I8), torch.zeros(2, 4))
    w.codes, w.scales = Fake((2, 4, 16), I8), Fake((2, 4), F32)
    return w


@pytest.mark.parametrize("grouped,which", [(g, m) for g in (False, True) for m in
                                           ("codes", "scales", "x", "x_scales", "workspace", "y") + ("offsets",) * g])
def test_products_refuse_another_device(grouped, which, monkeypatch):
    """Each tensor of the call, those that the weights consist of among them."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    w = _weights()
    given = dict(x=Fake((3, 16), I8), x_scales=Fake((3,), F32), workspace=Fake((1 << 20,), torch.uint8), y=Fake((3, 4), F32))
    if grouped:
        given["offsets"] = Fake((3,), I32)
    for t in (*given.values(), w.codes, w.scales):
        t.at = 0
    (given[which] if which in given else getattr(w, which)).at = 1
    with pytest.raises(q.IqkValueError, match="cuda:1"):
        (q.int8_grouped if grouped else q.int8_linear)(w, **given)


class FakeDual(Fake):
    """a dual tensor of forward-mode differentiation"""

    tangent = 1


@pytest.fixture
def dual_level(monkeypatch):
    """An open level in which FakeDual has a tangent; ordinary tensors are looked at as they are."""
    real = q._forward_ad.unpack_dual
    fake = lambda t: t if isinstance(t, FakeDual) else real(t) if isinstance(t, torch.Tensor) else FakeNone()
    monkeypatch.setattr(q._forward_ad, "unpack_dual", fake)
    with q._forward_ad.dual_level():
        yield


class FakeNone:
    tangent = None


def _calls(x):
    """Calls that carry gradients, with x in each place that one is carried from."""
    like = lambda *shape, dtype=F32: Fake(shape, dtype)
    ids, place = like(4, 2, dtype=I32), like(2, 2, dtype=I32)
    return (lambda: q.moe_sort(x, ids, 4), lambda: q.moe_unsort(x, place), lambda: q.moe_unsort(like(4, 64), place, x),
            lambda: q.block_norm(x, next_weight=like(64)), lambda: q.block_norm(like(4, 64), x), lambda: q.block_norm(like(4, 64), like(4, 64), x),
            lambda: q.block_norm(like(4, 64), like(4, 64), gate=x), lambda: q.block_norm(like(4, 64), next_weight=x), lambda: q.router_topk(x, 2))


@pytest.mark.parametrize("which", range(9))
def test_forward_mode_is_refused(which, dual_level):
    """A tangent would be lost without a word, with gradients switched off too."""
    for context in (torch.enable_grad, torch.no_grad):
        with context(), pytest.raises(q.IqkValueError, match="tangent"):
            _calls(FakeDual((4, 64), F32))[which]()


def test_forward_mode_of_real_tensors():
    x, v = torch.randn(4, 64), torch.randn(4, 64)
    with q._forward_ad.dual_level():
        dual = q._forward_ad.make_dual(x, v)
        for call in (lambda: q.block_norm(dual, dual), lambda: q.moe_unsort(dual, torch.zeros(2, 2, dtype=I32))):
            with pytest.raises(q.IqkValueError, match="tangent"):
                call()
        assert not q._wants_grad(x, None, dual.detach())  # (what has none is no one's loss)
        assert q._wants_grad(x, v.clone().requires_grad_())
        with torch.inference_mode():
            assert not q._wants_grad(dual)  # (no operation carries one there)
    assert not q._wants_grad(x)


class FakeLeaf(Fake):
    requires_grad = True


@pytest.mark.parametrize("which", ["x", "x_scales", "scales"])
@pytest.mark.parametrize("grouped", [False, True])
def test_products_refuse_what_requires_a_gradient(which, grouped, monkeypatch):
    """They have none to give, and a result without one would pass for a constant."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    w = _weights()
    given = dict(x=Fake((3, 16), I8), x_scales=Fake((3,), F32), workspace=Fake((1 << 20,), torch.uint8), y=Fake((3, 4), F32))
    if grouped:
        given["offsets"] = Fake((3,), I32)
    if which == "scales":
        w.scales = FakeLeaf((2, 4), F32)
    else:
        given[which] = FakeLeaf(given[which].shape, F32)
    call = q.int8_grouped if grouped else q.int8_linear
    with pytest.raises(q.IqkValueError, match="no gradient"):
        call(w, **given)
    given["y"] = Fake((3, 5), F32)  # where gradients are off the call goes on, to the next mistake
    with torch.no_grad(), pytest.raises(q.IqkValueError) as e:
        call(w, **given)
    assert "no gradient" not in str(e.value)


def test_quantization_refuses_what_requires_a_gradient():
    x = torch.randn(3, 32, requires_grad=True)
    with pytest.raises(q.IqkValueError, match="no gradient"):
        q.int8_quantize(x)
    for context, v in ((torch.no_grad, x), (torch.enable_grad, x.detach())):
        with context(), pytest.raises(q.IqkValueError, match="device tensor"):
            q.int8_quantize(v)


def test_products_refuse_forward_mode(dual_level):
    with torch.no_grad():
        for call in (lambda: q.int8_linear(_weights(), FakeDual((3, 16), F32)), lambda: q.int8_quantize(FakeDual((3, 16), F32)),
                     lambda: q.int8_grouped(_weights(), FakeDual((3, 16), F32), Fake((3,), I32))):
            with pytest.raises(q.IqkValueError, match="tangent"):
                call()
