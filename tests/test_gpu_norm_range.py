"""The gradient of the norms far from unit scale: rows up to the largest values whose squares' sum is a float32
number, and rows that are small or zero beside the smallest eps.  The oracle and the bounds of test_gpu_norm; the
gradient comes through the norms alone (dr null), since beside dr it would not be seen."""
import pytest
import torch

import dequant_iqk_moe_amd as q
from test_gpu_norm import BF16, F32, _args, _check_forward, _check_grad, _inputs

pytestmark = pytest.mark.gpu


def _scaled(T, n, dtype, scale, **form):
    v = _inputs(T, n, dtype, **form)
    v["x"][:, n // 3] /= 20  # (its values of 20 would pass 1e17)
    unit = v["x"].float()
    for m in ("x", "y"):
        v[m] = None if v[m] is None else (v[m].double() * scale).to(v[m].dtype)
    return v, unit


@pytest.mark.parametrize("scale", [1e13, 1e16])
@pytest.mark.parametrize("n", [24, 513, 1000, 4096, 8192])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", [dict(with_y=False, post=False, gate=None), dict(post=False, gate=None), dict(gate=None),
                                  dict(gate="channel"), dict(gate="token"), dict(gate="element")])
def test_gradient_of_large_rows(scale, n, dtype, form):
    """h does not change along r, so what dh holds of that direction has to leave the gradient."""
    v, unit = _scaled(5, n, dtype, scale, **form)
    a = _args(1.0, 0.5)
    _check_forward(v, a)
    dh = (torch.randn(5, n, generator=torch.Generator().manual_seed(4)) + 2 * unit).to(dtype)
    got = _check_grad(v, a, None, dh)
    assert (got[0] != 0).any()


@pytest.mark.parametrize("n", [24, 513, 4096, 8192])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", [dict(with_y=False, post=False, gate=None), dict(gate=None), dict(gate="channel"), dict(gate="token")])
@pytest.mark.parametrize("eps", [1e-26, 1e-30])
def test_gradient_of_zero_and_small_rows_with_a_tiny_eps(n, dtype, form, eps):
    v, _ = _scaled(4, n, dtype, 1.0, **form)
    for m in ("x", "y"):
        if v[m] is not None:
            v[m][0] = 0
            v[m][1] *= 1e-14
    a = _args(1.0, 0.5, eps)
    _check_forward(v, a)
    got = _check_grad(v, a, None, _inputs(4, n, dtype, seed=2)["x"])
    assert all(torch.isfinite(t).all() for t in got if t is not None)


def test_gradient_of_a_norm_behind_the_block_alone():
    """dy through post_weight's norm where h is not asked for: rows of 1e16, and of zeros beside an eps of 1e-30."""
    for n in (72, 4096):
        v, unit = _scaled(4, n, F32, 1e16, nxt=False)
        v["y"][0] = 0
        dr = torch.randn(4, n, generator=torch.Generator().manual_seed(7)) + unit
        for eps in (1e-6, 1e-30):
            got = _check_grad(v, _args(0.5, 0.7, eps), dr, None)
            assert all(torch.isfinite(t).all() for t in got if t is not None)
