"""The norms around a block and their gradient against the 64-bit oracle, with
bounds that follow the formula step by step (see rounding.py).

Longest chains of additions: of a row's sum, 16 values of a thread, four
rotations, three sums of sixteen lanes and seven of waves: 30; of a parameter's
gradient, a team's rows (T / 256 and one more) and the join's (at most 128 teams a
run for up to 2048 of them, no more than T / 16 + 1, and 15 runs)."""
import numpy as np
import pytest
import torch

import dequant_iqk_moe_amd as q
from oracle import block
from rounding import Ev
from gpu_common import announce

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
ROW = 30


def _inputs(T, n, dtype=F32, y_dtype=None, w_dtype=F32, gate_dtype=F32, post=True, gate="channel", nxt=True, with_y=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    shape = {None: None, "channel": (n,), "token": (T, 1), "element": (T, n)}[gate]
    x = r(T, n)
    x[:, n // 3] *= 20
    return dict(x=x.to(dtype), y=(r(T, n) * 0.7).to(y_dtype or dtype) if with_y else None,
                post_weight=(1 + 0.3 * r(n)).to(w_dtype) if post else None, gate=None if shape is None else r(*shape).to(gate_dtype),
                next_weight=(1 + 0.3 * r(n)).to(w_dtype) if nxt else None)


def _cuda(v):
    return {m: None if t is None else t.cuda() for m, t in v.items()}


def _ev(t):
    return None if t is None else Ev(t.double().numpy())


def _scale(v, n, eps):
    """s(v), with the division by n and the addition of eps (a float32)."""
    return ((v * v).sum(1, ROW) * Ev(1.0 / n) + Ev(eps)).inv_sqrt()


def _forward(v, alpha, beta, eps):
    x, y, wp, g, wn = (_ev(v[m]) for m in ("x", "y", "post_weight", "gate", "next_weight"))
    n = x.v.shape[1]
    u = s = r = h = qs = None
    if y is not None:
        u = y
        if wp is not None:
            s = _scale(y, n, eps)
            u = y * s * wp
        gu = u if g is None else (Ev(beta) * g) * u
        if g is None:
            gu = Ev(beta) * u
        r = Ev(alpha) * x + gu
    else:
        r = x
    if wn is not None:
        qs = _scale(r, n, eps)
        h = r * qs * wn
    return dict(x=x, y=y, wp=wp, g=g, wn=wn, u=u, s=s, r=r, q=qs, h=h, n=n)


def _args(alpha, beta, eps=1e-6):
    """as the library gets them: float32 values"""
    return dict(alpha=float(np.float32(alpha)), beta=float(np.float32(beta)), eps=float(np.float32(eps)))


def _check_forward(v, a):
    f = _forward(v, **a)
    r, h = q.block_norm(**_cuda(v), **a)
    want = block.block_norm(*(None if v[m] is None else v[m].double().numpy() for m in ("x", "y", "post_weight", "gate", "next_weight")), **a)
    if v["y"] is None:
        assert torch.equal(r.cpu(), v["x"])
    else:
        np.testing.assert_allclose(f["r"].v, want[0], rtol=1e-9, atol=1e-12)
        f["r"].check(r)
    if v["next_weight"] is None:
        assert h is None
    else:
        np.testing.assert_allclose(f["h"].v, want[1], rtol=1e-9, atol=1e-12)
        f["h"].check(h)


def _check_grad(v, a, dr, dh, cuda=_cuda):
    f = _forward(v, **a)
    T, n = f["x"].v.shape
    columns = T / 256 + 1 + T / 16 + 1 + 16
    D = Ev(np.zeros((T, n))) if dr is None else _ev(dr)
    bounds = {}
    if v["next_weight"] is not None:
        e = Ev(np.zeros((T, n))) if dh is None else _ev(dh)
        back = (f["r"] * (f["wn"] * e)).sum(1, ROW + 1)
        cube = f["q"] * f["q"] * f["q"] * Ev(1.0 / n)
        D = D + (f["q"] * (f["wn"] * e) - cube * back * f["r"])
        bounds["next"] = (e * (f["r"] * f["q"])).sum(0, columns)
    bounds["x"] = Ev(a["alpha"]) * D
    if v["y"] is not None:
        D = Ev(a["beta"]) * D
        if f["g"] is not None:
            dg = D * f["u"]
            if v["gate"].dim() == 1:
                dg = dg.sum(0, columns)
            elif v["gate"].shape[1] != n:
                dg = dg.sum(1, ROW)
            bounds["gate"] = dg
            D = D * f["g"]
        if f["wp"] is not None:
            bounds["post"] = (D * (f["y"] * f["s"])).sum(0, columns)
            w = D * f["wp"]
            cube = f["s"] * f["s"] * f["s"] * Ev(1.0 / n)
            D = f["s"] * w - cube * (w * f["y"]).sum(1, ROW + 1) * f["y"]
        bounds["y"] = D
    c = cuda(v)
    got = q.block_norm_grad(c["x"], c["y"], None if dr is None else dr.cuda(), None if dh is None else dh.cuda(),
                            post_weight=c["post_weight"], gate=c["gate"], next_weight=c["next_weight"], **a)
    d = lambda t: None if t is None else t.double().numpy()
    want = block.block_norm_grad(d(v["x"]), d(v["y"]), d(dr), d(dh if v["next_weight"] is not None else None), d(v["post_weight"]),
                                 d(v["gate"]), d(v["next_weight"]), **a)
    if dh is None and v["next_weight"] is not None:
        want = (*want[:4], np.zeros(n))
    for name, t, ref in zip(("x", "y", "post", "gate", "next"), got, want):
        if ref is None:
            assert t is None and name not in bounds
            continue
        b = bounds[name]
        b = Ev(b.v.reshape(ref.shape), b.e.reshape(ref.shape))
        np.testing.assert_allclose(b.v, ref, rtol=1e-8, atol=1e-10)
        b.check(t)
    return got


WIDTHS = [1, 2, 7, 8, 9, 65, 511, 512, 513, 1000, 1024, 1025, 2047, 2048, 2056, 4095, 4096, 4097, 5001, 8191, 8192]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES)
def test_widths(n, dtype):
    announce(f"norm 5 x {n} {dtype}")
    v, a = _inputs(5, n, dtype, w_dtype=dtype, gate_dtype=dtype), _args(0.75, 0.22)
    _check_forward(v, a)
    dr, dh = (_inputs(5, n, dtype, seed=s)["x"] for s in (1, 2))
    _check_grad(v, a, dr, dh)


@pytest.mark.parametrize("T", [1, 3, 4, 63, 257, 600])
@pytest.mark.parametrize("n", [40, 900, 1500, 3000, 4500])
def test_tokens(T, n):
    announce(f"norm {T} x {n}")
    v, a = _inputs(T, n, BF16), _args(1.0, 0.5)
    _check_forward(v, a)
    dr, dh = (_inputs(T, n, BF16, seed=s)["x"] for s in (1, 2))
    _check_grad(v, a, dr, dh)


def test_more_tokens_than_teams():
    T, n = 2600, 72
    v, a = _inputs(T, n, F32), _args(1.0, 1.0)
    _check_forward(v, a)
    dr, dh = (_inputs(T, n, F32, seed=s)["x"] for s in (1, 2))
    _check_grad(v, a, dr, dh)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token", "element"])
@pytest.mark.parametrize("nxt", [False, True])
@pytest.mark.parametrize("n", [200, 4099])
def test_forms(post, gate, nxt, n):
    a = _args(1.5, -0.7, 1e-3)
    for dtype, y_dtype, w_dtype, gate_dtype in ((F32, F32, F16, BF16), (BF16, F32, F32, BF16), (F16, F32, F16, F32), (BF16, BF16, BF16, F16)):
        announce(f"norm {post} {gate} {nxt} {n} {dtype} {y_dtype} {w_dtype} {gate_dtype}")
        v = _inputs(6, n, dtype, y_dtype, w_dtype, gate_dtype, post, gate, nxt)
        _check_forward(v, a)
        dr, dh = (_inputs(6, n, dtype, seed=s)["x"] for s in (1, 2))
        _check_grad(v, a, dr, dh if nxt else None)
        if nxt:
            _check_grad(v, a, None, dh)
            _check_grad(v, a, dr, None)


@pytest.mark.parametrize("n", [1, 300, 2048, 4100])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_before_the_first_block(n, dtype):
    v, a = _inputs(7, n, dtype, post=False, gate=None, with_y=False), _args(1.0, 1.0)
    _check_forward(v, a)
    dr, dh = (_inputs(7, n, dtype, seed=s)["x"] for s in (1, 2))
    _check_grad(v, a, None, dh)
    _check_grad(v, a, dr, dh)


def test_rows_of_zeros_and_special_values():
    v, a = _inputs(6, 520, F32, gate=None), _args(1.0, 1.0)
    v["x"][0], v["y"][0] = 0, 0
    v["y"][1] = 0
    v["x"][2, 5] = float("nan")
    v["y"][3, 6] = float("inf")
    c = _cuda(v)
    r, h = q.block_norm(**c, **a)
    assert (r[0] == 0).all() and (h[0] == 0).all()
    assert torch.equal(r[1], c["x"][1])
    assert r[2].isnan().sum() == 1 and h[2].isnan().all() and h[3].isnan().any()
    assert torch.isfinite(r[4:]).all() and torch.isfinite(h[4:]).all()
    rest = {m: t if t is None or t.dim() == 1 else t[4:].contiguous() for m, t in c.items()}
    r2, h2 = q.block_norm(**rest, **a)
    assert torch.equal(r[4:], r2) and torch.equal(h[4:], h2)
    got = q.block_norm_grad(c["x"][:2].contiguous(), c["y"][:2].contiguous(), torch.ones(2, 520, device="cuda"),
                            torch.ones(2, 520, device="cuda"), post_weight=c["post_weight"], next_weight=c["next_weight"], **a)
    assert all(torch.isfinite(t).all() for t in got if t is not None)


def test_results_over_the_inputs():
    v, a = _cuda(_inputs(9, 4096, BF16)), _args(1.0, 0.5)
    r, h = q.block_norm(**v, **a)
    for over in ("x", "y"):
        w = dict(v)
        w[over] = v[over].clone()
        other = "y" if over == "x" else "x"
        r2, h2 = q.block_norm(**w, **a, r=w[over])
        assert r2 is w[over] and torch.equal(r2, r) and torch.equal(h2, h)
        w[over], w[other] = v[over].clone(), v[other].clone()
        r2, h2 = q.block_norm(**w, **a, r=w[over], h=w[other])
        assert torch.equal(r2, r) and torch.equal(h2, h)
    x = v["x"].clone()
    _, h = q.block_norm(x, next_weight=v["next_weight"])
    assert torch.equal(q.block_norm(x, next_weight=v["next_weight"], h=x)[1], h)


def test_only_the_asked_for_is_written():
    for n in (65, 4096, 8192):
        v, a = _cuda(_inputs(5, n, BF16)), _args(1.0, 0.5)
        buf = [torch.full((5 * n + 32,), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
        q.block_norm(**v, **a, r=buf[0][16:-16].view(5, n), h=buf[1][16:-16].view(5, n))
        for b in buf:
            assert (b[:16] == 7).all() and (b[-16:] == 7).all()
        dr = torch.randn(5, n, device="cuda").to(BF16)
        args = dict(post_weight=v["post_weight"], gate=v["gate"], next_weight=v["next_weight"], **a)
        full = q.block_norm_grad(v["x"], v["y"], dr, dr, **args)
        for i in range(5):
            want = tuple(j == i for j in range(5))
            got = q.block_norm_grad(v["x"], v["y"], dr, dr, want=want, **args)
            assert [t is not None for t in got] == list(want) and torch.equal(got[i], full[i])
        need = q.block_norm_grad_workspace_bytes(5, n, channel_gate=True)
        ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        got = q.block_norm_grad(v["x"], v["y"], dr, dr, workspace=ws[:need], **args)
        assert all(torch.equal(s, t) for s, t in zip(got, full)) and (ws[need:] == 0xA5).all()


def test_no_tokens():
    v = _cuda(_inputs(1, 40, F32))
    e = torch.empty(0, 40, device="cuda")
    r, h = q.block_norm(e, e, v["post_weight"], v["gate"], v["next_weight"])
    assert r.shape == h.shape == (0, 40)
    got = q.block_norm_grad(e, e, e, e, post_weight=v["post_weight"], gate=v["gate"], next_weight=v["next_weight"])
    assert got[0].shape == got[1].shape == (0, 40)
    assert all((t == 0).all() and t.shape == (40,) for t in got[2:])  # sums over no tokens


@pytest.mark.parametrize("gate", [None, "channel", "token", "element"])
def test_autograd_is_the_gradient_call(gate):
    v, a = _cuda(_inputs(2 * 5, 72, BF16, gate=gate)), _args(0.5, 0.22)
    shaped = {m: t if t is None or t.dim() == 1 else t.view(2, 5, t.shape[1]) for m, t in v.items()}
    leaf = {m: None if t is None else t.clone().requires_grad_() for m, t in shaped.items()}
    r, h = q.block_norm(**leaf, **a)
    assert r.shape == h.shape == (2, 5, 72)
    dr, dh = torch.randn(2, 5, 72, device="cuda").to(BF16), torch.randn(2, 5, 72, device="cuda").to(BF16)
    torch.autograd.backward([r, h], [dr, dh])
    want = q.block_norm_grad(v["x"], v["y"], dr, dh, post_weight=v["post_weight"], gate=v["gate"], next_weight=v["next_weight"], **a)
    for (m, t), w in zip(leaf.items(), want):
        assert t is None and w is None or torch.equal(t.grad, w.view(t.shape)), m
    # one result alone, and the norm before the first block
    for t in leaf.values():
        if t is not None:
            t.grad = None
    r, h = q.block_norm(**leaf, **a)
    (h.float() * 2).sum().backward()
    want = q.block_norm_grad(v["x"], v["y"], None, torch.full_like(dh, 2), post_weight=v["post_weight"], gate=v["gate"],
                             next_weight=v["next_weight"], **a)
    assert torch.equal(leaf["x"].grad, want[0].view(2, 5, 72)) and torch.equal(leaf["next_weight"].grad, want[4])
    x, h = q.block_norm(leaf["x"], next_weight=v["next_weight"])
    assert x is leaf["x"]
    leaf["x"].grad = None
    h.backward(dh)
    assert torch.equal(leaf["x"].grad.view(10, 72), q.block_norm_grad(v["x"], None, None, dh, next_weight=v["next_weight"])[0])
    with pytest.raises(q.IqkValueError):
        q.block_norm(**leaf, **a, r=torch.empty_like(r))


def test_the_same_leaf_twice():
    """One tensor as the stream and the block's output: its gradient is the sum of both."""
    x = torch.randn(6, 48, device="cuda", requires_grad=True)
    w = torch.randn(48, device="cuda")
    r, h = q.block_norm(x, x, post_weight=w, next_weight=w)
    (r.sum() + (h * h).sum()).backward()
    dx, dy, *_ = q.block_norm_grad(x.detach(), x.detach(), torch.ones_like(r), 2 * h.detach(), post_weight=w, next_weight=w)
    assert torch.equal(x.grad, dx + dy)


def test_results_are_the_same_every_time():
    v, a = _cuda(_inputs(3000, 520, BF16)), _args(1.0, 1.0)
    dr = torch.randn(3000, 520, device="cuda").to(BF16)
    args = dict(post_weight=v["post_weight"], gate=v["gate"], next_weight=v["next_weight"], **a)
    first = q.block_norm_grad(v["x"], v["y"], dr, dr, **args)
    for _ in range(3):
        assert all(torch.equal(s, t) for s, t in zip(first, q.block_norm_grad(v["x"], v["y"], dr, dr, **args)))


@pytest.mark.parametrize("n", [64, 1024, 2048, 4096, 8192])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tensors_that_begin_anywhere(n, dtype):
    """Rows of whole chunks whose first value lies at no multiple of 16 bytes, one tensor of the call at a time and all
    of them: each value as where it does, and nothing beside a result is written."""
    T = 5

    def shifted(t, fill=None):
        buf = torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device="cuda")
        v = buf[1:t.numel() + 1].view(t.shape)
        if fill is None:
            v.copy_(t)
        return buf, v

    v, a = _inputs(T, n, dtype, y_dtype=F32), _args(0.5, 0.7)
    c = _cuda(v)
    dr, dh = (_inputs(T, n, dtype, seed=s)["x"] for s in (1, 2))
    f = _forward(v, **a)
    for moved in (*[(m,) for m in c], tuple(c)):
        w = {m: shifted(t)[1] if m in moved else t for m, t in c.items()}
        (rb, r), (hb, h) = shifted(c["x"], 0), shifted(c["x"], 0)
        q.block_norm(**w, **a, r=r, h=h)
        f["r"].check(r)
        f["h"].check(h)
        for b in (rb, hb):
            assert b[0] == 7 and (b[-15:] == 7).all()
        _check_grad(v, a, dr, dh, cuda=lambda _: w)


@pytest.mark.parametrize("n", [33, 520, 4096, 8192])
@pytest.mark.parametrize("gate", [None, "channel", "token", "element"])
def test_no_gradient_through_values_without_a_norm(n, gate):
    """Without a norm behind them, infinities and NaN in x and y have no part in their gradients."""
    v, a = _cuda(_inputs(4, n, F32, post=False, gate=gate, nxt=False)), _args(0.5, 2.0)
    dr = torch.randn(4, n, device="cuda")
    args = dict(gate=v["gate"], **a)
    clean = q.block_norm_grad(v["x"], v["y"], dr, None, **args)
    x, y = v["x"].clone(), v["y"].clone()
    x[0, 3], x[1, 4], y[1, 5], y[2, 6], x[2, 6] = float("nan"), float("inf"), float("nan"), float("-inf"), float("inf")
    dx, dy, _, dg, _ = q.block_norm_grad(x, y, dr, None, **args)
    assert torch.equal(dx, 0.5 * dr) and torch.equal(dx, clean[0]) and torch.equal(dy, clean[1])
    if gate == "element":
        there = torch.isfinite(y)
        assert torch.equal(dg[there], clean[3][there])
    # a norm of y alone: a row of x has no part in dy, nor y in dx
    w = torch.ones(n, device="cuda")
    got = q.block_norm_grad(x, v["y"], dr, None, post_weight=w, **args)
    want = q.block_norm_grad(v["x"], v["y"], dr, None, post_weight=w, **args)
    assert all(torch.equal(s, t) for s, t in zip(got[:3], want[:3]))
    assert torch.equal(q.block_norm_grad(x, y, dr, None, post_weight=w, **args)[0], 0.5 * dr)
