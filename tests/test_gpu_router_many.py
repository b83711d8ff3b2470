"""Expert selection for so many tokens that four of them share a wave (rows of
16 lanes; from 8192 tokens on, up to 16 values a lane and 16 slots).

Two checks: a sample of the rows against the 64-bit oracle, with the bars of
test_gpu_router; and every row against the same rows in calls of fewer tokens
(a wave per token).  Rows whose choice hangs on float32 rounding (two compared
values that differ by less than 1e-6 of their size, and 1e-9) are left out of
both; equal values stay in.  Both forms round the same sums in another order:
weights within 4e-6 relative, as against the oracle."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from oracle import layer
from test_gpu_router import DT, _dev

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu
INF = np.inf
PIECE = 4099  # tokens of a call that takes a wave per token


def _logits(rng, T, E, dtype):
    """Multiples of 1/16 with many ties; special rows between ordinary ones, each kind at every place of a wave."""
    l = np.clip(np.round(rng.normal(size=(T, E)) * 24) / 16, -6, 6)
    lowest = float(torch.finfo(DT[dtype]).min)
    kinds = [lambda r: np.full(E, -INF), lambda r: np.where(np.arange(E) == E // 2, 1.0, -INF),
             lambda r: np.where(rng.random(E) < 0.8, -INF, r), lambda r: np.full(E, lowest),
             lambda r: np.where(rng.random(E) < 0.9, lowest, r), lambda r: np.zeros(E),
             lambda r: np.where(np.arange(E) == E - 1, np.nan, r), lambda r: np.where(np.arange(E) == 0, INF, r),
             lambda r: np.where(np.arange(E) < E // 2, -INF, r)]
    special = list(range(0, T, 61)) + [T - 3, T - 1]
    for i, t in enumerate(special):
        l[t] = kinds[i % len(kinds)](l[t])
    return l, special


def _hangs(l, scoring, bias, n_group, group_top):
    """Rows in which two values that a choice compares differ by too little."""
    v = torch.from_numpy(l)
    s = torch.sigmoid(v) if scoring == "sigmoid" else torch.softmax(v, -1)
    c = v if bias is None else torch.where(torch.isinf(v), v, s + torch.from_numpy(bias).double())
    sets = [c] if bias is not None else []
    if n_group > 1:
        worth = (s if bias is None and group_top == 2 else c).view(l.shape[0], n_group, -1)
        worth = worth.sort(-1, descending=True).values
        if group_top == 2 and worth.shape[-1] > 1:
            second = worth[..., 1]
            sets.append(worth[..., 0] + torch.where(second == -INF, torch.zeros_like(second), second))
        elif bias is not None:
            sets.append(worth[..., 0])
    bad = torch.zeros(l.shape[0], dtype=torch.bool)
    for x in sets:
        x = x.sort(-1).values
        d = x[:, 1:] - x[:, :-1]
        bad |= ((d > 0) & (d < 1e-6 * x[:, 1:].abs() + 1e-9)).any(-1)
    return bad.numpy()


CASES = [
    # E, k, groups
    (7, 3, {}), (60, 16, {}), (64, 6, {}), (160, 8, {}), (200, 10, {}), (256, 6, {}), (256, 16, {}), (33, 1, {}),
    (64, 17, {}),                                                            # more slots than a row has lanes: a wave each
    (64, 4, dict(n_group=16, topk_group=5, group_top=2)),                    # groups of one lane (4 experts)
    (256, 8, dict(n_group=16, topk_group=3, group_top=1)),                   # of one lane (16 experts)
    (256, 6, dict(n_group=8, topk_group=4, group_top=2)),                    # of two lanes
    (160, 6, dict(n_group=5, topk_group=3, group_top=2)),                    # of two lanes, the row not full
    (256, 5, dict(n_group=4, topk_group=1, group_top=2)),                    # of four
    (128, 5, dict(n_group=2, topk_group=1, group_top=1)),                    # of eight
    (256, 12, dict(n_group=2, topk_group=2, group_top=2)),                   # of eight, all stay
    (200, 6, dict(n_group=8, topk_group=3, group_top=1)),                    # of no whole lanes: a wave each
]


@pytest.mark.parametrize("E,k,groups", CASES)
@pytest.mark.parametrize("T,scoring,dtype", [(8192, "softmax", "bf16"), (8195, "sigmoid", "f32"), (8193, "softmax", "f16")])
@pytest.mark.parametrize("biased", [False, True])
def test_rows_of_16_lanes(E, k, groups, T, scoring, dtype, biased):
    announce(f"router T={T} E={E} k={k} {scoring} {dtype} bias={biased} {groups}")
    rng = np.random.default_rng(E * 31 + k + T + biased)
    l, special = _logits(rng, T, E, dtype)
    bias = None
    if biased:
        bias = rng.choice(np.float32([-0.25, 0.0, 0.25]), E)
        bias[rng.integers(E)] = -INF
        l = np.round(l * 2) / 2          # few values, so that few rows hang
    clear = ~_hangs(l, scoring, bias, groups.get("n_group", 1), groups.get("group_top", 1))
    assert clear.mean() > 0.5
    dev = _dev(l, DT[dtype])
    kw = dict(scoring=scoring, bias=None if bias is None else _dev(bias), **groups)
    sample = np.unique(np.r_[0:24, special[::3], T - 8:T])
    sample = sample[clear[sample]]
    for renorm in (False, True):
        ids, w = q.router_topk(dev, k, renorm=renorm, scale=2.5, **kw)
        parts = [q.router_topk(dev[i:i + PIECE], k, renorm=renorm, scale=2.5, **kw) for i in range(0, T, PIECE)]
        ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
        few_ids, few_w = (torch.cat([p[j] for p in parts]).cpu().numpy() for j in (0, 1))
        np.testing.assert_array_equal(ids[clear], few_ids[clear])
        np.testing.assert_allclose(w[clear], few_w[clear].astype(np.float64), rtol=4e-6, atol=2.5e-6)
        ref_ids, ref_w = layer.router(l[sample], k, scoring, bias=bias, renorm=renorm, scale=2.5, **groups)
        np.testing.assert_array_equal(ids[sample], ref_ids)
        np.testing.assert_array_equal(np.isnan(w[sample]), np.isnan(ref_w))
        np.testing.assert_allclose(np.nan_to_num(w[sample]), np.nan_to_num(ref_w), rtol=4e-6, atol=2.5e-6)


@pytest.mark.parametrize("scoring,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("E,k", [(160, 8), (256, 6), (60, 17)])
def test_gradient_of_many_tokens(E, k, scoring, renorm):
    """Rows of one large call have the bits of the same rows in small calls, and the oracle's values."""
    announce(f"router grad many E={E} k={k} {scoring} {renorm}")
    T = 8195
    rng = np.random.default_rng(E + k)
    l, special = _logits(rng, T, E, "bf16")
    dev, dw = _dev(l, torch.bfloat16), rng.normal(size=(T, k)).astype(np.float32)
    ids = q.router_topk(dev, k, scoring=scoring)[0]
    args = dict(scoring=scoring, renorm=renorm, scale=2.5)
    got = q.router_topk_grad(dev, ids, _dev(dw), **args)
    parts = [q.router_topk_grad(dev[i:i + 777], ids[i:i + 777], _dev(dw[i:i + 777]), **args) for i in range(0, T, 777)]
    assert torch.equal(got, torch.cat(parts))
    rows = np.unique(np.r_[0:24, special[::3], T - 8:T])
    rows = rows[~np.isnan(l[rows]).any(1) & ~(l[rows] == INF).any(1)]
    hids = ids.cpu().numpy()[rows]
    ref = layer.router_grad(l[rows], hids, dw[rows], scoring, renorm, 2.5)
    room = 1e-5 * 2.5 * np.abs(dw[rows]).max(1)[:, None] + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(got.double().cpu().numpy()[rows] - ref) <= room).all()
