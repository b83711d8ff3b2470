"""Values at the ends of float32 in expert selection and its gradient, against
the 64-bit oracle.  Bars as in test_gpu_router."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from oracle import layer
from test_gpu_router import DT, _check, _dev

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu
INF = np.inf
LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("least", [-85.0, -60.0, -20.0])
def test_gradient_of_small_scores(least, dtype):
    """Sigmoid scores of e^-85 with weights divided by their sum: the gradient is
    w_j (1 - s_j) (g_j - sum g w), of the size of g, whatever the scores'."""
    announce(f"router grad of logits from {least} {dtype}")
    rng = np.random.default_rng(int(-least))
    T, E, k = 9, 40, 4
    l = least + rng.integers(0, 8, (T, E)) / 2
    dw = (rng.normal(size=(T, k)) * 10.0 ** rng.integers(0, 7, (T, 1))).astype(np.float32)
    ids, _ = layer.router(l, k, "sigmoid")
    ref = layer.router_grad(l, ids, dw, "sigmoid", True, 2.5)
    got = q.router_topk_grad(_dev(l, DT[dtype]), _dev(ids), _dev(dw), scoring="sigmoid", scale=2.5).double().cpu().numpy()
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    room = 1e-5 * 2.5 * np.abs(dw).max(1)[:, None] + half * np.abs(ref)
    assert (np.abs(got - ref) <= room).all()


@pytest.mark.parametrize("E,n_group", [(24, 4), (32, 4), (256, 8), (60, 4)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_masked_by_the_lowest_finite_bias(E, n_group, scoring):
    """A bias of float32's lowest value is no -inf: its experts stay in, last, and the sum of
    a group's best two does not leave float32."""
    announce(f"router lowest bias E={E} G={n_group} {scoring}")
    per = E // n_group
    rng = np.random.default_rng(E)
    l = np.stack([rng.permutation(E) - E // 2 for _ in range(5)]) / 64   # scores at least 4e-6 apart (softmax), 1e-3 (sigmoid)
    bias = np.zeros(E, np.float32)
    bias[per:] = LOWEST                    # one group is free, the others have the lowest bias throughout
    k = min(64, per + 3)                   # more slots than that group has experts
    for keep in (2, n_group):
        _check(l, "f32", k, scoring, bias=bias, n_group=n_group, topk_group=keep, group_top=2)
    bias[:] = -LOWEST                      # and the highest
    bias[per:] = 0
    _check(l, "f32", k, scoring, bias=bias, n_group=n_group, topk_group=2, group_top=2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_rows_without_a_choice(scoring, renorm, dtype):
    """Rows that chose nothing (ids -1) have the gradient zero, whatever their logits."""
    rng = np.random.default_rng(3)
    l = np.round(rng.normal(size=(6, 70)) * 16) / 16
    l[1, 5], l[2, 66], l[3], l[4, 9] = np.nan, INF, -INF, -INF
    ids, _ = layer.router(l, 4, "softmax")
    assert (ids[1:4] == -1).all()
    dw = rng.normal(size=(6, 4)).astype(np.float32)
    ref = layer.router_grad(l, ids, dw, scoring, renorm, 1.0)
    got = q.router_topk_grad(_dev(l, DT[dtype]), _dev(ids), _dev(dw), scoring=scoring, renorm=renorm).double().cpu().numpy()
    assert (got[1:4] == 0).all()
    rows = [0, 4, 5]
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    assert (np.abs(got - ref)[rows] <= 1e-5 * np.abs(dw).max() + half * np.abs(ref[rows]) + 2.0 ** -25).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradient_of_one_expert_by_its_own_score_is_zero(scoring, dtype):
    """One slot divided by itself is one whatever the logits."""
    rng = np.random.default_rng(1)
    l = rng.normal(size=(50, 64)) * 3
    ids, _ = q.router_topk(_dev(l, DT[dtype]), 1, scoring=scoring)
    dw = _dev(rng.normal(size=(50, 1)).astype(np.float32) * 1000)
    assert not q.router_topk_grad(_dev(l, DT[dtype]), ids, dw, scoring=scoring).any()
