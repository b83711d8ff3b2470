"""8-bit integer quantization and products against the oracle: codes and scales bit
for bit, and results too, since sums are exact and the definition fixes the three
float32 roundings behind them and the one to the result's type."""
import numpy as np
import pytest
import torch

import dequant_iqk_moe_amd as q
from oracle import block
from gpu_common import announce

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _x(rows, n, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g)
    x[:, torch.randint(0, n, (max(1, n // 200),), generator=g)] *= 20
    return x.to(dtype)


def _w(E, out, n, seed=0):
    rng = np.random.default_rng(seed)
    codes = rng.integers(-128, 128, (E, out, n)).astype(np.int8)
    return codes, rng.uniform(1e-3, 1e-2, (E, out)).astype(np.float32)


def _dev(codes, scales):
    return q.Int8Weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def _same(got: torch.Tensor, want: np.ndarray):
    """Equal bits, NaNs aside (which have to be there)."""
    want = torch.from_numpy(want).to(got.dtype)
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    off = (got != want) & ~want.isnan()
    assert not off.any(), (int(off.sum()), got[off][:4], want[off][:4])


# ---------------------------------------------------------------------------
# quantization
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("rows,n", [(1, 16), (3, 512), (5, 2048), (2, 2064), (3, 8192), (2, 8208), (1, 65536), (1000, 48)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize(rows, n, dtype):
    announce(f"quantize {rows} x {n} {dtype}")
    x = _x(rows, n, dtype)
    x[0, -1] *= 30
    codes, scales = q.int8_quantize(x.cuda())
    want_codes, want_scales = block.quantize(x.float().numpy())
    assert np.array_equal(codes.cpu().numpy(), want_codes) and np.array_equal(scales.cpu().numpy(), want_scales)


def test_quantize_ties_and_special_rows():
    n = 32
    x = np.zeros((9, n), np.float32)
    x[0, :8] = [127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -127]  # factor 1: ties to even
    x[2, 5], x[3, 5], x[4, 5] = np.nan, np.inf, -np.inf
    x[2:5, 6] = 3
    x[5] = 2.0 ** -120  # below the floor: codes of zero
    x[6, 0] = 3.4e38
    x[7, :2] = [2.0 ** -100, -2.0 ** -101]
    x[8] = -np.float32(1e-40)  # subnormal
    codes, scales = q.int8_quantize(torch.from_numpy(x).cuda())
    want_codes, want_scales = block.quantize(x)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    assert np.array_equal(scales.cpu().numpy(), want_scales, equal_nan=True)
    assert want_codes[0, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, -127] and np.isnan(want_scales[2:5]).all()


def test_quantize_shapes_and_no_rows():
    codes, scales = q.int8_quantize(torch.randn(2, 3, 64, device="cuda"))
    assert codes.shape == (2, 3, 64) and scales.shape == (2, 3)
    codes, scales = q.int8_quantize(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0,)


# ---------------------------------------------------------------------------
# dense product
# ---------------------------------------------------------------------------

# sizes (rows, out, in) at which each kernel of the dense product runs
DENSE = [((1, 33, 16), ("few",)), ((4, 64, 4096), ("few",)), ((3, 17, 1040), ("few",)), ((1, 20, 32992), ("few",)),
         ((1, 20, 65536), ("rows",)), ((5, 257, 144), ("rows",)), ((16, 40, 2064), ("rows",)), ((17, 100, 4096), ("rows",)),
         ((32, 33, 16), ("rows",)), ((7, 9000, 64), ("tiles", 16, 128)), ((34, 116, 64), ("tiles", 16, 128)),
         ((77, 130, 528), ("tiles", 16, 128)), ((48, 16391, 144), ("tiles", 32, 128)), ((2980, 131, 80), ("tiles", 32, 128)),
         ((1869, 516, 64), ("tiles", 64, 128)), ((300, 4001, 2064), ("tiles", 64, 128)), ((2000, 1290, 272), ("tiles", 128, 128)),
         ((1301, 2101, 128), ("tiles", 128, 128)), ((2382, 1743, 64), ("tiles", 128, 256)), ((2048, 4096, 272), ("tiles", 128, 256)),
         ((2600, 4100, 400), ("tiles", 256, 256)), ((3202, 2505, 272), ("tiles", 256, 256))]


@pytest.mark.parametrize("size,path", DENSE)
def test_dense_paths(size, path):
    M, out, n = size
    assert q.int8_path(1, out, n, M) == path


@pytest.mark.parametrize("size,path", DENSE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16, torch.int8])
def test_linear(size, path, dtype):
    M, out, n = size
    codes, scales = _w(1, out, n, M)
    if dtype == torch.int8:
        rng = np.random.default_rng(n)
        xq, xs = rng.integers(-128, 128, (M, n)).astype(np.int8), rng.uniform(0.5, 2, M).astype(np.float32)
        args = dict(x=torch.from_numpy(xq).cuda(), x_scales=torch.from_numpy(xs).cuda())
    else:
        x = _x(M, n, dtype, n)
        xq, xs = block.quantize(x.float().numpy())
        args = dict(x=x.cuda())
    want = block.int8_product(codes[0], scales[0], xq, xs)
    w = _dev(codes, scales)
    for out_dtype in TYPES:
        announce(f"linear {size} {dtype} {out_dtype} {path}")
        buf = torch.full((M * out + 64,), 7.0, dtype=out_dtype, device="cuda")
        y = q.int8_linear(w, y=buf[32:-32].view(M, out), **args)
        _same(y, want)
        assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()


def test_largest_sums():
    """65536 products of -128 by -128: 2^30."""
    w = q.Int8Weights(torch.full((1, 70, 65536), -128, dtype=torch.int8, device="cuda"), torch.ones(1, 70, device="cuda"))
    x = torch.full((40, 65536), -128, dtype=torch.int8, device="cuda")
    for rows in (1, 20, 40):
        assert (q.int8_linear(w, x[:rows], torch.ones(rows, device="cuda")) == 2.0 ** 30).all()


def test_rows_with_nan_or_infinity_keep_to_themselves():
    for rows, n in ((4, 256), (6, 256), (300, 256), (300, 16)):
        x = _x(rows, n, torch.float32, 1)
        x[1, 3], x[3, 5] = float("nan"), float("inf")
        w = _dev(*_w(1, 80, n))
        y = q.int8_linear(w, x.cuda()).cpu()
        assert y.isnan().all(1).nonzero().flatten().tolist() == [1, 3]
        assert torch.isfinite(y[[0, 2] + list(range(4, rows))]).all()
    scales = torch.full((1, 80), 1e-2)
    scales[0, 7], scales[0, 8] = float("nan"), float("inf")
    w = q.Int8Weights(w.codes, scales.cuda())
    y = q.int8_linear(w, torch.ones(300, 16, device="cuda"))
    assert y[:, 7].isnan().all() and not torch.isfinite(y[:, 8]).any() and torch.isfinite(y[:, :7]).all()


def test_leading_dimensions_and_no_rows():
    w = _dev(*_w(1, 24, 64))
    x = torch.randn(3, 5, 64, device="cuda")
    y = q.int8_linear(w, x)
    assert y.shape == (3, 5, 24) and torch.equal(y.view(15, 24), q.int8_linear(w, x.view(15, 64)))
    assert q.int8_linear(w, torch.empty(0, 64, device="cuda")).shape == (0, 24)


def test_a_rows_bits_do_not_depend_on_its_place():
    for M, out, n in ((4, 100, 2048), (29, 100, 2048), (100, 100, 512), (1869, 516, 64), (2000, 1290, 272), (2382, 1743, 64), (2600, 4100, 400)):
        x, w = _x(M, n, torch.bfloat16, 5).cuda(), _dev(*_w(1, out, n))
        perm = torch.randperm(M, generator=torch.Generator().manual_seed(1)).cuda()
        for dtype in TYPES:
            assert torch.equal(q.int8_linear(w, x, out_dtype=dtype)[perm], q.int8_linear(w, x[perm], out_dtype=dtype))


def test_workspace_of_exactly_the_size_asked_for():
    w, x = _dev(*_w(1, 130, 528)), _x(100, 528, torch.bfloat16).cuda()
    need = q.int8_linear_workspace_bytes(w, 100)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    y = q.int8_linear(w, x, workspace=ws[:need])
    assert torch.equal(y, q.int8_linear(w, x)) and (ws[need:] == 0xA5).all()
    codes, scales = q.int8_quantize(x)
    assert torch.equal(q.int8_linear(w, codes, scales), y)
    assert q.int8_linear_workspace_bytes(w, 100, torch.int8) == 0
    with pytest.raises(q.IqkValueError):
        q.int8_linear(w, x, workspace=ws[:need - 1])


# ---------------------------------------------------------------------------
# grouped product
# ---------------------------------------------------------------------------

# (experts, out, in, rows of each expert, rows of none) at which each kernel of the grouped product runs
GROUPED = [((3, 33, 64, [2, 0, 1], 0), ("few",)), ((256, 40, 4096, [0] * 200 + [1] * 6 + [0] * 50, 2), ("few",)),
           ((4, 30, 2048, [30, 0, 0, 2], 0), ("few",)), ((2, 20, 65536, [1, 2], 1), ("tiles", 16, 128)),
           ((60, 141, 272, [5] * 30 + [0, 9] * 15, 3), ("tiles", 16, 128)), ((3, 257, 400, [129, 127, 128], 70), ("tiles", 16, 128)),
           ((2, 50, 16, [0, 0], 50), ("tiles", 16, 128)), ((16, 131, 64, [250, 0] * 4 + [149] * 8, 186), ("tiles", 32, 128)),
           ((16, 1024, 2048, [50] * 10 + [0, 99] * 3, 3), ("tiles", 32, 128)), ((40, 262, 64, [0, 115, 57] * 13 + [40], 19), ("tiles", 64, 128)),
           ((40, 711, 80, [61, 0, 64, 65, 100] * 8, 0), ("tiles", 128, 128)), ((8, 4100, 256, [300, 0, 250, 290, 310, 280, 340, 250], 9), ("tiles", 128, 128)),
           ((16, 1000, 512, [300, 255, 129, 0] * 4, 2000), ("tiles", 128, 256)),
           ((16, 2997, 144, [257, 130, 0, 390] * 4, 0), ("tiles", 256, 256))]


@pytest.mark.parametrize("size,path", GROUPED)
def test_grouped_paths(size, path):
    E, out, n, counts, none = size
    assert len(counts) == E and q.int8_path(E, out, n, sum(counts) + none, grouped=True) == path


@pytest.mark.parametrize("size,path", GROUPED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16, torch.int8])
def test_grouped(size, path, dtype):
    E, out, n, counts, none = size
    rows = sum(counts) + none
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    codes, scales = _w(E, out, n, rows)
    if dtype == torch.int8:
        rng = np.random.default_rng(n)
        xq, xs = rng.integers(-128, 128, (rows, n)).astype(np.int8), rng.uniform(0.5, 2, rows).astype(np.float32)
        args = dict(x=torch.from_numpy(xq).cuda(), x_scales=torch.from_numpy(xs).cuda())
    else:
        x = _x(rows, n, dtype, n)
        x[rows - none:] = float("nan")  # rows of none do not matter
        xq, xs = block.quantize(x.float().numpy())
        args = dict(x=x.cuda())
    want = block.int8_grouped(codes, scales, xq, xs, offsets)
    w, off = _dev(codes, scales), torch.from_numpy(offsets).cuda()
    for out_dtype in TYPES:
        announce(f"grouped {E} {out} {n} {rows} {dtype} {out_dtype} {path}")
        buf = torch.full((rows * out + 64,), 7.0, dtype=out_dtype, device="cuda")
        y = q.int8_grouped(w, offsets=off, y=buf[32:-32].view(rows, out), **args)
        _same(y, want)
        assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()


def test_offsets_outside_the_rows_are_cut():
    w, x = _dev(*_w(3, 40, 64)), _x(100, 64, torch.float32).cuda()
    good = q.int8_grouped(w, x, torch.tensor([0, 30, 100, 100], dtype=torch.int32, device="cuda"))
    assert torch.equal(good, q.int8_grouped(w, x, torch.tensor([-5, 30, 2 ** 31 - 1, 101], dtype=torch.int32, device="cuda")))
    few = x[:20].contiguous()
    good = q.int8_grouped(w, few, torch.tensor([0, 3, 20, 20], dtype=torch.int32, device="cuda"))
    assert torch.equal(good, q.int8_grouped(w, few, torch.tensor([-5, 3, 2 ** 31 - 1, 21], dtype=torch.int32, device="cuda")))


def test_grouped_is_the_dense_product_of_each_expert():
    E, out, n = 4, 200, 320
    w = _dev(*_w(E, out, n, 3))
    counts = [100, 0, 57, 300]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    x = _x(sum(counts), n, torch.bfloat16, 4).cuda()
    y = q.int8_grouped(w, x, off)
    at = 0
    for e, c in enumerate(counts):
        one = q.Int8Weights(w.codes[e:e + 1], w.scales[e:e + 1])
        assert torch.equal(y[at:at + c], q.int8_linear(one, x[at:at + c].contiguous()))
        at += c


def test_grouped_workspace_of_exactly_the_size_asked_for():
    w, x = _dev(*_w(9, 130, 528)), _x(200, 528, torch.bfloat16).cuda()
    off = torch.tensor([0, 20, 20, 50, 51, 90, 100, 150, 170, 190], dtype=torch.int32, device="cuda")
    need = q.int8_grouped_workspace_bytes(w, 200)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    y = q.int8_grouped(w, x, off, workspace=ws[:need])
    assert torch.equal(y, q.int8_grouped(w, x, off)) and (ws[need:] == 0xA5).all()
    codes, scales = q.int8_quantize(x)
    need = q.int8_grouped_workspace_bytes(w, 200, torch.int8)
    assert torch.equal(q.int8_grouped(w, codes, off, scales, workspace=ws[:need]), y)
    assert q.int8_grouped(w, x[:0], off).shape == (0, 130)


def test_weights_beyond_32_bits():
    """40 experts of 16384 x 8192: 5.4 GB of codes."""
    E, out, n = 40, 16384, 8192
    codes = torch.randint(-128, 128, (E, out, n), dtype=torch.int8, device="cuda")
    scales = torch.rand(E, out, device="cuda")
    w = q.Int8Weights(codes, scales)
    for counts in ([0] * 38 + [3, 2], [1] * 40, [0] * 37 + [100, 50, 70]):
        off = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device="cuda")
        x = _x(sum(counts), n, torch.bfloat16, 1).cuda()
        y = q.int8_grouped(w, x, off)
        one = q.Int8Weights(codes[39:], scales[39:])
        assert torch.equal(y[off[39]:], q.int8_linear(one, x[off[39]:].contiguous()))
