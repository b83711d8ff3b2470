"""Logits that require a gradient: the weights carry it (no silent detaching)."""
import pytest
import torch

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu


def _logits(dtype=torch.float32):
    return torch.randn(37, 60, generator=torch.Generator().manual_seed(1)).to(dtype).cuda().requires_grad_()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_is_the_gradient_call(scoring, renorm, dtype):
    l = _logits(dtype)
    bias = torch.linspace(-0.1, 0.1, 60, device="cuda")
    args = dict(scoring=scoring, renorm=renorm, scale=2.5)
    ids, w = q.router_topk(l, 5, bias=bias, n_group=4, topk_group=2, **args)
    plain_ids, plain = q.router_topk(l.detach(), 5, bias=bias, n_group=4, topk_group=2, **args)
    assert torch.equal(ids, plain_ids) and torch.equal(w.detach(), plain)
    assert w.requires_grad and not ids.requires_grad and not plain.requires_grad
    dw = torch.randn(37, 5, device="cuda")
    (w * dw).sum().backward()
    assert l.grad.dtype == dtype
    assert torch.equal(l.grad, q.router_topk_grad(l.detach(), ids, dw, **args))


def test_expanded_gradient_and_caller_buffers():
    l = _logits()
    ids = torch.empty(37, 6, dtype=torch.int32, device="cuda")
    buf = torch.empty(37, 6, device="cuda")
    i, w = q.router_topk(l, 6, renorm=False, ids=ids, weights=buf)
    assert i is ids and w.data_ptr() == buf.data_ptr()
    w.sum().backward()
    assert torch.equal(l.grad, q.router_topk_grad(l.detach(), ids, torch.ones_like(buf), renorm=False))


def test_ids_that_a_later_call_overwrote_are_refused():
    l = _logits()
    ids = torch.empty(37, 6, dtype=torch.int32, device="cuda")
    _, w = q.router_topk(l, 6, ids=ids)
    q.router_topk(l.detach() * -1, 6, ids=ids)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        w.sum().backward()


def test_without_gradients_nothing_is_recorded():
    l = _logits()
    with torch.no_grad():
        assert not q.router_topk(l, 6)[1].requires_grad
    assert not q.router_topk(l.detach(), 6)[1].requires_grad


def test_inference_mode_with_caller_buffers():
    with torch.inference_mode():
        l = torch.randn(3, 60, device="cuda")
        ids = torch.empty(3, 6, dtype=torch.int32, device="cuda")
        assert torch.equal(q.router_topk(l, 6, ids=ids)[1], q.router_topk(l, 6)[1])


def test_the_same_buffers_in_every_step():
    l = _logits()
    ids = torch.empty(37, 6, dtype=torch.int32, device="cuda")
    buf = torch.empty(37, 6, device="cuda")
    dw = torch.randn(37, 6, device="cuda")
    for step in range(3):
        l.grad = None
        _, w = q.router_topk(l, 6, ids=ids, weights=buf)
        (w * dw).sum().backward()
        assert torch.equal(l.grad, q.router_topk_grad(l.detach(), ids, dw))
        with torch.no_grad():
            l -= l.grad
    assert not buf.requires_grad
    # a step whose weights are needed after the next call overwrote them
    _, w = q.router_topk(l, 6, ids=ids, weights=buf)
    loss = (w * w).sum()
    q.router_topk(l.detach() * -1, 6, weights=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
