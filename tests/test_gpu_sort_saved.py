"""What the gradient of moe_unsort keeps alive: only what it reads."""
import pytest
import torch

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu

T, K, E, N = 40, 3, 6, 130


def _case(dtype=torch.float32):
    g = torch.Generator().manual_seed(0)
    ids = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(T, N, generator=g).to(dtype).cuda()
    ys, _, place = q.moe_sort(x, ids, E)
    return ys, place, torch.rand(T, K, generator=g).cuda(), torch.randn(T, N, generator=g).cuda()


def _saved(call):
    """Addresses of the tensors that a forward call keeps for its gradient"""
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t.data_ptr()) or t, lambda t: t):
        call()
    return kept


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weighted", [False, True])
def test_rows_may_be_overwritten_where_no_weight_needs_a_gradient(dtype, weighted):
    ys, place, w, dy = _case(dtype)
    w = w if weighted else None
    leaf = ys.clone().requires_grad_()
    rows = leaf * 1  # (a leaf itself may not be written)
    assert rows.data_ptr() not in _saved(lambda: q.moe_unsort(rows, place, w))
    y = q.moe_unsort(rows, place, w)
    want = q.moe_unsort_grad(dy, ys, place, w, want_weights=False)[0]
    with torch.no_grad():
        rows.fill_(float("nan"))
    y.backward(dy)
    assert leaf.grad.dtype == dtype and torch.equal(leaf.grad, want)


def test_rows_are_kept_for_the_weights_gradient():
    ys, place, w, dy = _case()
    leaf, rows = w.clone().requires_grad_(), ys.clone()
    assert rows.data_ptr() in _saved(lambda: q.moe_unsort(rows, place, leaf))
    y = q.moe_unsort(rows, place, leaf)
    rows.zero_()
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward(dy)


def test_weights_may_be_overwritten_where_no_row_needs_a_gradient():
    ys, place, w, dy = _case()
    leaf = w.clone().requires_grad_()
    weights = leaf * 1
    assert weights.data_ptr() not in _saved(lambda: q.moe_unsort(ys, place, weights))
    y = q.moe_unsort(ys, place, weights)
    want = q.moe_unsort_grad(dy, ys, place, w, want_ys=False)[1]
    with torch.no_grad():
        weights.fill_(float("nan"))
    y.backward(dy)
    assert torch.equal(leaf.grad, want)


def test_both_gradients():
    ys, place, w, dy = _case()
    leaves = ys.clone().requires_grad_(), w.clone().requires_grad_()
    q.moe_unsort(leaves[0], place, leaves[1]).backward(dy)
    want = q.moe_unsort_grad(dy, ys, place, w)
    assert torch.equal(leaves[0].grad, want[0]) and torch.equal(leaves[1].grad, want[1])
    flat = w.reshape(-1).clone().requires_grad_()  # weights of another shape: their gradient is of theirs
    q.moe_unsort(ys, place, flat).backward(dy)
    assert torch.equal(flat.grad, want[1].reshape(-1))


def test_no_tokens():
    ys, place = torch.empty(0, N, device="cuda", requires_grad=True), torch.empty(0, K, dtype=torch.int32, device="cuda")
    q.moe_unsort(ys, place).backward(torch.empty(0, N, device="cuda"))
    assert ys.grad.shape == (0, N)
