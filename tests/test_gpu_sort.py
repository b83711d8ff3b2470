"""Rows sorted by expert and back, and their gradients, against the 64-bit oracle.

Sorted rows, offsets and places are equal.  Sums: each product rounds once and
each of k - 1 additions once, at most 2 k 2^-24 of the sum of the magnitudes; a dot
product's longest chain is a lane's 8 values in each piece of 2048, four
rotations, three sums of sixteen lanes and three of waves.  Then one rounding to the
result's type."""
import numpy as np
import pytest
import torch

import dequant_iqk_moe_amd as q
from oracle import block
from rounding import U, Ev
from gpu_common import announce

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _x(T, n, dtype, seed=0):
    return torch.randn(T, n, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _ids(T, k, E, seed=0, invalid=0.0):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    bad = rng.random((T, k)) < invalid
    return torch.from_numpy(np.where(bad, rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1], (T, k)), ids).astype(np.int32))


def _bits(t):
    return t.cpu().contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16).numpy()


def _check_sort(x, ids, E, got):
    xs, offsets, place = got
    want_offsets, want_place = block.order(ids.numpy(), E)
    assert np.array_equal(offsets.cpu().numpy(), want_offsets)
    assert np.array_equal(place.cpu().numpy(), want_place)
    T, k = ids.shape
    want = torch.zeros(T * k, x.shape[1], dtype=x.dtype)
    flat = torch.from_numpy(want_place.reshape(-1)).long()
    there = flat >= 0
    want[flat[there]] = x[torch.arange(T * k) // k][there]
    assert np.array_equal(_bits(xs), _bits(want))


@pytest.mark.parametrize("T,k,E,n,invalid", [
    (1, 1, 1, 1, 0), (1, 6, 256, 4096, 0), (1, 6, 256, 7, 1.0), (2, 64, 3, 33, 0.1), (5, 3, 2048, 8, 0), (37, 8, 60, 129, 0.3),
    (64, 2, 1, 2048, 0), (700, 5, 16, 24, 0.5), (8192, 1, 7, 5, 0.1), (1024, 8, 160, 10, 0),  # the last in one launch
    (1025, 8, 160, 10, 0), (8193, 1, 2048, 3, 0.2), (1500, 6, 256, 264, 0.9), (2049, 4, 3, 17, 1.0), (513, 64, 2, 6, 0),
    (96, 64, 300, 40, 0.2), (128, 64, 2048, 9, 0), (129, 64, 40, 130, 0.1), (2048, 2, 33, 12, 0.3), (2049, 2, 33, 12, 0.3), (2896, 1, 9, 17, 0),
    (2897, 1, 9, 17, 0)])
@pytest.mark.parametrize("dtype", TYPES)
def test_sort(T, k, E, n, invalid, dtype):
    announce(f"sort {T} x {k} of {E}, {n} {dtype}")
    x, ids = _x(T, n, dtype), _ids(T, k, E, T + k, invalid)
    _check_sort(x, ids, E, q.moe_sort(x.cuda(), ids.cuda(), E))


def test_sort_of_no_tokens():
    xs, offsets, place = q.moe_sort(torch.empty(0, 5, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda"), 9)
    assert xs.shape == (0, 5) and place.shape == (0, 3) and offsets.tolist() == [0] * 10
    assert q.moe_unsort(xs, place).shape == (0, 5)


def test_sort_writes_every_value_and_no_more():
    x, ids = _x(700, 13, torch.bfloat16), _ids(700, 13, 40, 5, 0.2)  # 9100 pairs: three launches
    for T in (700, 20):
        P = T * 13
        buf = [torch.full((P * 13 + 32,), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((41 + 32,), 77, dtype=torch.int32, device="cuda"),
               torch.full((P + 32,), 77, dtype=torch.int32, device="cuda")]
        part = [b[16:-16] for b in buf]
        ws = torch.full((q.moe_sort_workspace_bytes(T, 13, 40),), 0xA5, dtype=torch.uint8, device="cuda")
        got = q.moe_sort(x[:T].cuda(), ids[:T].cuda(), 40, xs=part[0].view(P, 13), offsets=part[1], place=part[2].view(T, 13), workspace=ws)
        _check_sort(x[:T], ids[:T], 40, got)
        for b, v in zip(buf, (7.0, 77, 77)):
            assert (b[:16] == v).all() and (b[-16:] == v).all()


def test_special_values_are_copied():
    x = _x(9, 8, torch.float32)
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = float("nan"), float("inf"), -float("inf"), -0.0
    x.view(torch.int32)[4, 4] = 0x7F800001  # a signalling NaN
    ids = _ids(9, 4, 5, 3, 0.2)
    _check_sort(x, ids, 5, q.moe_sort(x.cuda(), ids.cuda(), 5))


def test_rows_beyond_32_bits():
    """8 rows of each of 40000 tokens, 16 KiB a row: 5.2 GB of sorted rows."""
    T, k, n = 40000, 8, 8192
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].expand(T, n).to(torch.bfloat16).contiguous()
    ids = torch.randint(0, 64, (T, k), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    xs, offsets, place = q.moe_sort(x, ids, 64)
    perm = ids.view(-1).long().argsort(stable=True)
    want = torch.empty_like(perm)
    want[perm] = torch.arange(T * k, device="cuda")
    assert torch.equal(place.view(-1).long(), want)
    for c in (0, 4095, 8191):
        assert torch.equal(xs[:, c], x[:, c][perm // k])
    w = torch.full((T, k), 0.25, device="cuda")
    y = q.moe_unsort(xs, place, w, out_dtype=torch.bfloat16)
    assert torch.equal(y, 2 * x)
    d_ys, d_w = q.moe_unsort_grad(x, xs, place, w)
    assert torch.equal(d_ys[:, 77], (0.25 * x[:, 77])[perm // k])
    one = (x[-1].double() ** 2).sum()
    assert float((d_w[-1].double() - one).abs().max() / one) < 1e-5


@pytest.mark.parametrize("T,k,n", [(1, 1, 1), (1, 6, 4096), (3, 8, 2047), (5, 9, 8), (2, 64, 130), (40, 3, 2056), (333, 5, 31)])
@pytest.mark.parametrize("ys_dtype,y_dtype", [(a, b) for a in TYPES for b in TYPES])
def test_unsort_and_its_gradient(T, k, n, ys_dtype, y_dtype):
    announce(f"unsort {T} x {k}, {n} {ys_dtype} {y_dtype}")
    rng = np.random.default_rng(T + n)
    ids = _ids(T, k, 12, T, 0.15)
    _, place = block.order(ids.numpy(), 12)
    ys, dy = _x(T * k, n, ys_dtype, 1), _x(T, n, y_dtype, 2)
    w = rng.normal(size=(T, k)).astype(np.float32)
    dev = [torch.from_numpy(place).cuda(), torch.from_numpy(w).cuda()]
    for weights in (w, None):
        y, size = block.unsort(ys.double().numpy(), place, weights)
        given = None if weights is None else dev[1]
        Ev(y, 2 * k * U * size).check(q.moe_unsort(ys.cuda(), dev[0], given, out_dtype=y_dtype))
        d_ys, d_w, size = block.unsort_grad(dy.double().numpy(), ys.double().numpy(), place, weights)
        got_ys, got_w = q.moe_unsort_grad(dy.cuda(), ys.cuda(), dev[0], given)
        Ev(d_ys, U * np.abs(d_ys)).check(got_ys)
        if weights is None:
            assert got_w is None
        else:
            chain = 8 * -(-n // 2048) + 4 + 3 + 4
            Ev(d_w, chain * U * size).check(got_w)
            again = q.moe_unsort_grad(dy.cuda(), ys.cuda(), dev[0], given, want_ys=False)
            assert again[0] is None and torch.equal(again[1], got_w)
            again = q.moe_unsort_grad(dy.cuda(), ys.cuda(), dev[0], given, want_weights=False)
            assert again[1] is None and torch.equal(again[0], got_ys)


def test_unsort_is_combine():
    """Where rows lie in the order of their pairs the two are one."""
    T, k, n = 50, 6, 512
    ys, w = torch.randn(T * k, n, device="cuda"), torch.randn(T, k, device="cuda")
    place = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    assert torch.equal(q.moe_unsort(ys, place, w), q.combine(ys.view(T, k, n), w))


def test_pairs_of_no_expert_count_as_zeros():
    T, k, n = 4, 3, 40
    ids = torch.tensor([[-1, -1, -1], [0, -1, 1], [1, 0, 9], [0, 0, 0]], dtype=torch.int32)
    place = torch.from_numpy(block.order(ids.numpy(), 2)[1]).cuda()
    ys = torch.randn(T * k, n, device="cuda")
    ys[0] = float("nan")  # a row that is not theirs
    rows_of_none = [int(-1 - p) for p in place.flatten().tolist() if p < 0]
    ys[rows_of_none] = float("inf")
    w = torch.ones(T, k, device="cuda")
    y = q.moe_unsort(ys, place, w)
    assert (y[0] == 0).all() and y[1:3].isnan().any(1).tolist() == [True, False] and torch.isfinite(y[3]).all()
    w[0, 1] = float("nan")  # what expert selection gives a row it could not choose for
    assert q.moe_unsort(ys, place, w)[0].isnan().all()
    dy = torch.randn(T, n, device="cuda")
    dy[0, 3] = float("inf")
    d_ys, d_w = q.moe_unsort_grad(dy, ys, place, w)
    assert (d_w[0] == 0).all() and (d_ys[rows_of_none] == 0).all()


def test_places_outside_the_rows_are_not_followed():
    ys = torch.randn(6, 16, device="cuda")
    place = torch.tensor([[0, 6, 2 ** 31 - 1], [-7, -2 ** 31, 5]], dtype=torch.int32, device="cuda")
    w = torch.ones(2, 3, device="cuda")
    assert torch.equal(q.moe_unsort(ys, place, w), ys[[0, 5]])
    guard = torch.full((8, 16), 3.0, device="cuda")
    q.moe_unsort_grad(torch.ones(2, 16, device="cuda"), ys, place, w, d_ys=guard[1:7])
    assert (guard[[1, 6]] == 1).all() and (guard[[0, 2, 3, 4, 5, 7]] == 3).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_autograd(dtype):
    """x -> sorted rows -> rows of a function -> y: gradients of x and the weights are the calls'."""
    T, k, E, n = 30, 4, 7, 65
    x, w = _x(T, n, dtype).cuda().requires_grad_(), torch.randn(T, k, device="cuda", requires_grad=True)
    ids = _ids(T, k, E, 9, 0.1).cuda()
    xs, offsets, place = q.moe_sort(x, ids, E)
    assert not offsets.requires_grad and not place.requires_grad
    ys = xs * 2
    y = q.moe_unsort(ys, place, w, out_dtype=dtype)
    dy = torch.randn(T, n, device="cuda").to(dtype)
    y.backward(dy)
    d_ys, d_w = q.moe_unsort_grad(dy, ys.detach(), place, w.detach())
    assert torch.equal(w.grad, d_w)
    assert torch.equal(x.grad, q.moe_unsort(d_ys * 2, place, out_dtype=dtype))
    with torch.no_grad():
        assert not q.moe_sort(x, ids, E)[0].requires_grad and not q.moe_unsort(ys, place, w).requires_grad
    # without gradients of the rows, and without weights
    q.moe_unsort(ys.detach(), place, w).sum().backward()
    assert not q.moe_unsort(ys.detach(), place).requires_grad
    with pytest.raises(q.IqkValueError):
        q.moe_sort(x, ids, E, xs=torch.empty_like(xs))
    with pytest.raises(q.IqkValueError):
        q.moe_unsort(ys, place, w, y=torch.empty_like(y))


def test_autograd_against_differences():
    T, k, E, n = 6, 3, 4, 5
    ids = _ids(T, k, E, 2, 0.2).cuda()
    x, w = torch.randn(T, n, device="cuda"), torch.randn(T, k, device="cuda")
    dy = torch.randn(T, n, device="cuda")

    def loss(x, w):
        xs, _, place = q.moe_sort(x, ids, E)
        return (q.moe_unsort(xs, place, w) * dy).double().sum()

    leaf = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss(*leaf).backward()
    h = 2.0 ** -6  # the loss is linear in each: no truncation; sums of 30 values round by 30 * 2^-24 of about 10, over 2 h
    for which, t in enumerate((x, w)):
        for at in np.ndindex(*t.shape):
            v = [x.clone(), w.clone()]
            v[which][at] += h
            up = loss(*v)
            v[which][at] -= 2 * h
            assert abs(float(up - loss(*v)) / (2 * h) - float(leaf[which].grad[at])) < 2e-3


def test_place_that_a_later_call_overwrote_is_refused():
    x, ids = torch.randn(5, 8, device="cuda", requires_grad=True), _ids(5, 2, 3).cuda()
    place = torch.empty(5, 2, dtype=torch.int32, device="cuda")
    xs = q.moe_sort(x, ids, 3, place=place)[0]
    q.moe_sort(x.detach(), ids, 3, place=place)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        xs.sum().backward()
