"""Pins of the 64-bit oracle of the operators around the routed experts (CPU)."""
import numpy as np
import pytest
import torch

from oracle import block


def test_order_by_hand():
    ids = np.array([[2, 0], [7, 2], [0, -1]], np.int32)
    offsets, place = block.order(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert place.tolist() == [[2, 0], [-5, 3], [1, -6]]


def test_sort_and_unsort_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    ids = np.array([[1, 0], [0, 5]], np.int32)
    xs, offsets, place = block.sort(x, ids, 2)
    assert xs.tolist() == [[1, 2], [3, 4], [1, 2], [0, 0]] and offsets.tolist() == [0, 2, 3]
    w = np.array([[0.5, 2.0], [3.0, 9.0]])
    y, size = block.unsort(xs, place, w)
    assert y.tolist() == [[2.5, 5.0], [9.0, 12.0]] and np.array_equal(y, size)


def test_order_is_a_stable_argsort():
    ids = np.random.default_rng(1).integers(0, 9, (40, 3)).astype(np.int32)
    offsets, place = block.order(ids, 9)
    perm = np.argsort(ids.reshape(-1), kind="stable")
    assert np.array_equal(place.reshape(-1)[perm], np.arange(120))
    assert np.array_equal(np.diff(offsets), np.bincount(ids.reshape(-1), minlength=9))


def _difference(f, x, at, h=1e-6):
    up, down = x.copy(), x.copy()
    up[at] += h
    down[at] -= h
    return (f(up) - f(down)) / (2 * h)


def test_unsort_gradient_against_differences():
    rng = np.random.default_rng(2)
    ids = np.array([[0, 3], [1, 1], [9, 0]], np.int32)
    _, place = block.order(ids, 4)
    ys, w, dy = rng.normal(size=(6, 5)), rng.normal(size=(3, 2)), rng.normal(size=(3, 5))
    d_ys, d_w, _ = block.unsort_grad(dy, ys, place, w)
    for at in np.ndindex(6, 5):
        assert abs(d_ys[at] - _difference(lambda v: (block.unsort(v, place, w)[0] * dy).sum(), ys, at)) < 1e-8
    for at in np.ndindex(3, 2):
        assert abs(d_w[at] - _difference(lambda v: (block.unsort(ys, place, v)[0] * dy).sum(), w, at)) < 1e-8


def test_quantize_by_hand():
    q, s = block.quantize(np.array([[254.0, -1.0, 1.0, 3.0, -254.0], [0, 0, 0, 0, 0], [1, np.nan, 0, 0, 0], [1, np.inf, 0, 0, 0]]))
    assert q.tolist() == [[127, 0, 0, 2, -127], [0] * 5, [0] * 5, [0] * 5]  # ties to even: 0.5 and 1.5
    assert s[0] == 2.0 and s[1] == np.float32(2.0 ** -100) / np.float32(127) and np.isnan(s[2:]).all()


def test_int8_product_against_integers():
    rng = np.random.default_rng(3)
    w, x = rng.integers(-128, 128, (3, 40)).astype(np.int8), rng.integers(-128, 128, (2, 40)).astype(np.int8)
    sw, sx = np.array([1, 0.5, 2], np.float32), np.array([4, 0.25], np.float32)
    want = (x.astype(np.int64) @ w.astype(np.int64).T) * np.outer(sx, sw)
    np.testing.assert_array_equal(block.int8_product(w, sw, x, sx), want)  # (powers of two: exact)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("kind", [None, "channel", "token", "element"])
@pytest.mark.parametrize("nxt", [False, True])
def test_norm_gradient_against_differences_and_autograd(post, kind, nxt):
    rng = np.random.default_rng(4)
    T, n = 3, 5
    v = dict(x=rng.normal(size=(T, n)), y=rng.normal(size=(T, n)), post=rng.normal(size=n) if post else None,
             gate={None: None, "channel": rng.normal(size=n), "token": rng.normal(size=(T, 1)),
                   "element": rng.normal(size=(T, n))}[kind], nxt=rng.normal(size=n) if nxt else None)
    dr, dh = rng.normal(size=(T, n)), rng.normal(size=(T, n)) if nxt else None
    args = dict(alpha=0.7, beta=-1.3, eps=1e-3)

    def loss(**change):
        r, h = block.block_norm(**{**v, **change}, **args)
        return (r * dr).sum() + (0 if h is None else (h * dh).sum())

    got = dict(zip(v, block.block_norm_grad(v["x"], v["y"], dr, dh, v["post"], v["gate"], v["nxt"], **args)))
    for name, value in v.items():
        if value is None:
            assert got[name] is None
            continue
        for at in np.ndindex(value.shape):
            assert abs(got[name][at] - _difference(lambda z: loss(**{name: z}), value, at)) < 1e-7


def test_norm_before_the_first_block():
    x = np.array([[3.0, -4.0]])
    r, h = block.block_norm(x, nxt=np.array([1.0, 2.0]), eps=1e-12)
    np.testing.assert_allclose(h, [[3 / np.sqrt(12.5), -8 / np.sqrt(12.5)]])
    assert r is x or np.array_equal(r, x)
    t = torch.tensor(x, requires_grad=True)
    (t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-12) * torch.tensor([1.0, 2.0])).sum().backward()
    dx = block.block_norm_grad(x, None, None, np.ones((1, 2)), nxt=np.array([1.0, 2.0]), eps=1e-12)[0]
    np.testing.assert_allclose(dx, t.grad.numpy(), rtol=1e-12)
