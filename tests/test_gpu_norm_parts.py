"""Norms' calls whose results must not depend on what has no part in them."""
import pytest
import torch

import dequant_iqk_moe_amd as q
from test_gpu_norm import F32, _args, _cuda, _inputs

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
