"""Expert selection and its gradient on the GPU against the 64-bit oracle.

Tolerances.  Ids: equal, on logits whose choice no float32 rounding can move
(values a choice compares are equal or at least 1e-5 apart, checked).
Weights: the logit difference in exp is rounded to 2^-24 of at most 40
(2.4e-6 of a weight), exp, sums and quotients add a few 2^-24: 4e-6 relative,
and 1e-6 of the scale for weights near zero.  Gradients: the same relative
error in each term of a sum of k terms: 1e-5 of the row's largest term
scale * max |dw| (times 1 / D where the weights are divided by D), plus half a
unit of the result's type."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from oracle import layer

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = np.inf


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(dtype) if dtype is not None else t).cuda()


def _grid_logits(rng, T, E):
    """Multiples of 1/16 in [-6, 6]: exact in every type, with many ties."""
    return np.clip(np.round(rng.normal(size=(T, E)) * 24) / 16, -6, 6)


def _check(logits, dtype, k, scoring, **kw):
    bias = kw.get("bias")
    ref_ids, ref_w = layer.router(logits, k, scoring, **kw)
    args = dict(kw)
    if bias is not None:
        args["bias"] = _dev(bias.astype(np.float32))
    ids, w = q.router_topk(_dev(logits, DT[dtype]), k, scoring=scoring, **args)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    got = w.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref_w))
    np.testing.assert_allclose(np.nan_to_num(got), np.nan_to_num(ref_w), rtol=4e-6, atol=1e-6 * kw.get("scale", 1.0))


@pytest.mark.parametrize("E,k", [(1, 1), (7, 3), (8, 8), (60, 6), (64, 64), (65, 5), (128, 1), (160, 8), (256, 6),
                                 (384, 10), (512, 8), (1000, 7), (1024, 33)])
@pytest.mark.parametrize("scoring,dtype", [("softmax", "f32"), ("softmax", "bf16"), ("sigmoid", "f16")])
def test_choice_by_logit(E, k, scoring, dtype):
    announce(f"router E={E} k={k} {scoring} {dtype}")
    rng = np.random.default_rng(E * 100 + k)
    for T in (1, 5, 130):
        for renorm in (False, True):
            _check(_grid_logits(rng, T, E), dtype, k, scoring, renorm=renorm, scale=2.5)


def _apart(rng, T, E, scoring, groups):
    """Logits and bias whose choice hangs on no float32 rounding."""
    logits = np.zeros((T, E))
    bias = (rng.integers(-100, 101, E) * 0.001).astype(np.float32)
    for t in range(T):
        for _ in range(2000):
            logits[t] = np.clip(np.round(rng.normal(size=E) * 48) / 32, -6, 6)
            if layer.router_gap(logits[t:t + 1], 1, scoring, bias, **groups) > (1e-5 if scoring == "sigmoid" else 1e-6):
                break
        else:
            raise AssertionError("no such row found")
    return logits, bias


@pytest.mark.parametrize("E,k,groups", [
    (8, 2, {}), (24, 4, dict(n_group=4, topk_group=2, group_top=2)), (32, 5, dict(n_group=8, topk_group=3, group_top=1)),
    (66, 6, dict(n_group=3, topk_group=2, group_top=2)), (64, 6, dict(n_group=64, topk_group=9, group_top=1))])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_choice_with_a_bias(E, k, groups, scoring):
    announce(f"router bias E={E} k={k} {scoring} {groups}")
    rng = np.random.default_rng(E + k)
    logits, bias = _apart(rng, 6, E, scoring, groups)
    for renorm in (False, True):
        _check(logits, "f32", k, scoring, bias=bias, renorm=renorm, **groups)


@pytest.mark.parametrize("E,n_group", [(64, 8), (96, 3), (256, 8), (160, 16), (512, 2), (1020, 60)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_by_logit(E, n_group, group_top):
    """Group worth from the best logit is exact; from the best two scores the
    logits of a group's best two are kept apart between groups."""
    announce(f"router groups E={E} G={n_group} top={group_top}")
    rng = np.random.default_rng(E + n_group)
    T, per = 9, E // n_group
    logits = _grid_logits(rng, T, E)
    if group_top == 2:
        # the worth of group g falls by at least 1 % from one rank to the next
        logits = np.minimum(logits, -3.0)
        for t in range(T):
            for rank, g in enumerate(rng.permutation(n_group)):
                logits[t, g * per + rng.integers(per)] = 2.0 - rank / 16
    for scoring in ("softmax", "sigmoid"):
        _check(logits, "f32", 4, scoring, n_group=n_group, topk_group=max(1, n_group // 2), group_top=group_top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masks_and_special_values(scoring, dtype):
    announce(f"router masks {scoring} {dtype}")
    rng = np.random.default_rng(11)
    E, k = 70, 5
    lowest = torch.finfo(DT[dtype]).min
    l = _grid_logits(rng, 12, E)
    l[0, rng.permutation(E)[:50]] = -INF
    l[1] = -INF                      # nothing left
    l[2] = -INF
    l[2, 66] = 1.0                   # one expert left for five slots
    l[3, 5:] = -INF                  # exactly enough
    l[4] = lowest                    # finite masks only
    l[5, 3:] = lowest                # fewer unmasked than slots, the rest finite
    l[6, 9] = np.nan
    l[7, 69] = INF
    l[8, 2] = np.nan
    l[8, 3] = -INF
    l[9] = 0.0                       # all equal
    for renorm in (False, True):
        _check(l, dtype, k, scoring, renorm=renorm)
    _check(l, dtype, k, scoring, n_group=7, topk_group=2, group_top=1)
    groups = l.copy()
    groups[:, :10] = -INF            # a whole group masked
    _check(groups, dtype, k, scoring, n_group=7, topk_group=6, group_top=1)


def test_bias_special_values():
    rng = np.random.default_rng(12)
    l = _grid_logits(rng, 4, 16)
    l = l[:, np.argsort(l[0])]
    bias = np.zeros(16, np.float32)
    bias[3] = -INF                   # switched off
    bias[2] = INF                    # always chosen
    logits, b = _apart(rng, 4, 16, "sigmoid", {})
    b[3], b[2] = -INF, INF
    _check(logits, "f32", 4, "sigmoid", bias=b)
    b[2] = np.nan
    _check(logits, "f32", 4, "sigmoid", bias=b)


def test_scores_that_underflow():
    """Sigmoid scores that are all zero in float32: weights zero, not NaN."""
    l = np.full((1, 8), -1e4, np.float32)
    ids, w = q.router_topk(_dev(l), 3, scoring="sigmoid", renorm=True)
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0.0, 0.0, 0.0]]


@pytest.mark.parametrize("E,k", [(1, 1), (9, 4), (64, 6), (65, 6), (160, 8), (256, 6), (513, 11), (1024, 64)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient(E, k, scoring, renorm):
    announce(f"router grad E={E} k={k} {scoring} renorm={renorm}")
    rng = np.random.default_rng(E + k)
    scale = 2.5
    for T in (1, 37):
        for dtype in ("f32", "bf16", "f16"):
            l = _grid_logits(rng, T, E)
            dw = rng.normal(size=(T, k)).astype(np.float32)
            ids, _ = layer.router(l, k, scoring)
            ref = layer.router_grad(l, ids, dw, scoring, renorm, scale)
            got = q.router_topk_grad(_dev(l, DT[dtype]), _dev(ids), _dev(dw), scoring=scoring, renorm=renorm, scale=scale)
            assert got.dtype == DT[dtype]
            got = got.double().cpu().numpy()
            d = np.array([layer.scores(l[t], scoring)[ids[t]].sum() for t in range(T)]) if renorm else np.ones(T)
            top = scale * np.abs(dw).max(1) * (np.maximum(1, 1 / d) if scoring == "sigmoid" else 1)
            half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
            room = 1e-5 * top[:, None] + half * np.abs(ref) + (2.0 ** -25 if dtype == "f16" else 0)
            assert (np.abs(got - ref) <= room).all()


def test_gradient_against_differences_of_the_forward_call():
    """Central differences of the GPU's own weights: float32 weights near 1
    are off by 1e-7, over 2h = 2^-5 that is 4e-6 per slot; the truncation is
    h^2 / 6 of a third derivative below 1 (4e-5).  Bar 3e-4 over 4 slots."""
    rng = np.random.default_rng(21)
    E, k, h = 12, 4, 2.0 ** -6
    l = rng.permutation(E)[None].astype(np.float64) / 2 - 3   # choices further apart than h
    dw = rng.normal(size=(1, k)).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = q.router_topk(_dev(l, torch.float32), k, scoring=scoring, renorm=renorm)
            got = q.router_topk_grad(_dev(l, torch.float32), ids, _dev(dw), scoring=scoring, renorm=renorm).cpu().numpy()
            up = np.repeat(l, E, 0) + h * np.eye(E)
            down = np.repeat(l, E, 0) - h * np.eye(E)
            wu = q.router_topk(_dev(up, torch.float32), k, scoring=scoring, renorm=renorm)
            wd = q.router_topk(_dev(down, torch.float32), k, scoring=scoring, renorm=renorm)
            assert (wu[0] == ids).all() and (wd[0] == ids).all()
            diff = ((wu[1] - wd[1]).double().cpu().numpy() * dw).sum(1) / (2 * h)
            assert np.abs(got[0] - diff).max() < 3e-4


def test_gradient_of_slots_that_take_no_part():
    l = np.array([[0.5, 1.0, -INF, -0.5], [-INF] * 4, [0.0, 1.0, 2.0, 3.0]])
    ids = np.array([[1, 0, 1], [-1, -1, -1], [3, 9, -7]], np.int32)   # a repeat, an empty row, invalid ids
    dw = np.array([[1.0, -2.0, 5.0]] * 3, np.float32)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ref = layer.router_grad(l, ids, dw, scoring, renorm, 1.0)
            got = q.router_topk_grad(_dev(l, torch.float32), _dev(ids), _dev(dw), scoring=scoring, renorm=renorm)
            assert np.abs(got.cpu().numpy() - ref).max() <= 1e-5 * 5


def test_other_stream_and_caller_buffers():
    rng = np.random.default_rng(31)
    l = _grid_logits(rng, 300, 256)
    dev = _dev(l, torch.bfloat16)
    ids = torch.full((300, 6), 77, dtype=torch.int32, device="cuda")
    w = torch.zeros(300, 6, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, b = q.router_topk(dev, 6, ids=ids, weights=w, stream=s)
    s.synchronize()
    assert a is ids and b is w
    ref_ids, _ = layer.router(l, 6, "softmax")
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)


def test_no_tokens():
    ids, w = q.router_topk(torch.empty(0, 64, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert q.router_topk_grad(torch.empty(0, 64, device="cuda"), ids, w).shape == (0, 64)
