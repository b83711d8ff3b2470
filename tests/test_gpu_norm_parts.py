"""Norms' calls whose results must not depend on what has no part in them."""
import pytest
import torch

import dequant_iqk_moe_amd as q
from test_gpu_norm import BF16, F32, _args, _cuda, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [33, 520, 4096, 8192])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token", "element"])
def test_next_weight_has_no_part_without_dh(n, post, gate):
    """A norm whose result no gradient comes from, whatever its weight holds."""
    v, a = _cuda(_inputs(4, n, F32, post=post, gate=gate)), _args(0.5, 2.0)
    dr = torch.randn(4, n, device="cuda")
    args = dict(post_weight=v["post_weight"], gate=v["gate"], **a)
    want = q.block_norm_grad(v["x"], v["y"], dr, None, next_weight=v["next_weight"], **args)
    w = v["next_weight"].clone()
    w[1], w[n // 2], w[n - 1] = float("inf"), float("nan"), float("-inf")
    got = q.block_norm_grad(v["x"], v["y"], dr, None, next_weight=w, **args)
    assert torch.equal(got[0], 0.5 * dr) and (got[4] == 0).all()
    assert all(s is None and t is None or torch.equal(s, t) for s, t in zip(got, want))
    # through autograd, where only r goes on
    leaf = {m: None if t is None else t.clone().requires_grad_() for m, t in dict(v, next_weight=w).items()}
    r, _ = q.block_norm(**leaf, **a)
    r.backward(dr)
    assert all(t is None or torch.equal(t.grad, s) for t, s in zip(leaf.values(), got))


def _shifted(t):
    """t at no multiple of 16 bytes"""
    v = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")[1:t.numel() + 1].view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 16
    return v


@pytest.mark.parametrize("n", [72, 1024, 2056, 4096, 8192])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_gate_of_tokens_lies_anywhere(n, dtype):
    """Its values are read one by one, so its address changes no bit of any result."""
    v, a = _cuda(_inputs(6, n, dtype, gate="token", gate_dtype=dtype)), _args(0.75, 0.22)
    w = dict(v, gate=_shifted(v["gate"]))
    dr, dh = (_inputs(6, n, dtype, seed=s)["x"].cuda() for s in (1, 2))
    assert all(torch.equal(s, t) for s, t in zip(q.block_norm(**v, **a), q.block_norm(**w, **a)))
    grads = [q.block_norm_grad(c["x"], c["y"], dr, dh, post_weight=c["post_weight"], gate=c["gate"],
                               next_weight=c["next_weight"], **a) for c in (v, w)]
    assert all(torch.equal(s, t) for s, t in zip(*grads))


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("n", [72, 1024, 4096, 8192])
def test_a_gates_summed_gradient_lies_anywhere(gate, n, monkeypatch):
    """It is written one value at a time."""
    v, a = _cuda(_inputs(6, n, BF16, gate=gate)), _args(0.75, 0.22)
    dr, dh = (_inputs(6, n, BF16, seed=s)["x"].cuda() for s in (1, 2))
    call = lambda: q.block_norm_grad(v["x"], v["y"], dr, dh, post_weight=v["post_weight"], gate=v["gate"],
                                     next_weight=v["next_weight"], **a)
    want, like = call(), q._like
    monkeypatch.setattr(q, "_like", lambda t, stream: _shifted(t) if t is v["gate"] else like(t, stream))
    got = call()
    assert got[3].data_ptr() % 16 and all(torch.equal(s, t) for s, t in zip(got, want))
