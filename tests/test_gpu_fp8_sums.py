"""What the sums of the 8-bit products keep, element by element.

float32 and float16 results are float32 sums with one rounding; a bfloat16
result of more than 32 dense rows may also be off by 7 * 2^-13 of the largest
product of each eight consecutive values of the depth.

Bars.  Where every partial sum is a float32 value (multiples of 2^-4 below
2^19, scales of one) the sum is exact and the result its rounding: equality.
Elsewhere a float32 sum of K products rounds at most K times by 2^-24 of the
sum of their magnitudes, twice more for the scales, and the result by half a
unit of its type.  Rounding to nearest of values of any size has a root mean
square of at most u / sqrt(12) of the values' (u the unit at the low end of a
binade: 2^-7 for bfloat16, 2^-10 for float16); cutting off has twice that.
5 % are left for the spread of a row's norm, 1e-4 for the eights."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from oracle import layer
from test_gpu_fp8 import DT, _activations, _dev, _device_weights, _weights

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu
EIGHT = 7 * 2.0 ** -13
# few rows, 17 to 32 rows, tiles of 64, 64 split along the depth, 128 and (bfloat16) 256
SHAPES = [(3, 130, 272), (20, 130, 272), (40, 130, 272), (64, 64, 8192), (1300, 2000, 272), (4000, 2600, 272)]


def _rounded(v, yt):
    """float64 values that float32 holds, rounded to the result's type."""
    return torch.from_numpy(v.astype(np.float32)).to(DT[yt]).double().numpy()


def _half_unit(v, yt):
    bits, least = {"f32": (24, -126), "bf16": (8, -126), "f16": (11, -14)}[yt]
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 1e-300))), least)
    return 2.0 ** (e - bits)


def _loudest_of_eight(xv, wv):
    """Sum over the eights of their largest |product|, [M, N]."""
    total = np.zeros((xv.shape[0], wv.shape[0]))
    for k in range(0, xv.shape[1], 8):
        most = np.zeros_like(total)
        for i in range(k, k + 8):
            np.maximum(most, np.abs(xv[:, i, None] * wv[None, :, i]), out=most)
        total += most
    return total


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_small_products_beside_loud_ones_that_cancel(M, N, K):
    """Two products of 448 * c cancel; what is left are the small ones beside the first."""
    announce(f"cancel M={M} N={N} K={K}")
    rng = np.random.default_rng(M + K)
    x, w = np.zeros((M, K)), np.zeros((N, K))
    eight = slice(40, 48)
    x[:, eight] = rng.integers(-8, 9, (M, 8)) / 4    # multiples of 1/4 up to 2: e4m3 values
    w[:, eight] = rng.integers(-8, 9, (N, 8)) / 4
    c = rng.choice([256.0, 320.0, 448.0], N)
    x[:, 43] = x[:, 90] = 448
    w[:, 43], w[:, 90] = c, -c
    ref = x[:, 40:43] @ w[:, 40:43].T + x[:, 44:48] @ w[:, 44:48].T
    nb = -(-K // 128)
    W = _device_weights(layer.to_e4m3(w)[None], np.ones((1, -(-N // 128), nb), np.float32))
    codes = _dev(layer.to_e4m3(x)).view(torch.float8_e4m3fn)
    ones = torch.ones(M, nb, device="cuda")
    for yt in ("f32", "f16", "bf16"):
        got = q.fp8_linear(W, codes, ones, out_dtype=DT[yt]).double().cpu().numpy()
        if yt == "bf16" and M > 32:
            room = EIGHT * (448 * c + 448 * c)[None, :] + _half_unit(np.abs(ref) + 400, yt)
            assert (np.abs(got - ref) <= room).all()
        else:
            np.testing.assert_array_equal(got, _rounded(ref, yt), err_msg=yt)


@pytest.mark.parametrize("M,N,K", SHAPES[:4] + [(300, 384, 400)])
def test_each_element_beside_loud_channels(M, N, K):
    """Normal values with a loud channel in every block: each element within its bound."""
    announce(f"loud channels M={M} N={N} K={K}")
    M, K = min(M, 300), min(K, 2048)
    rng = np.random.default_rng(M + N)
    w, s = _weights(rng, 1, N, K)
    W = _device_weights(w, s)
    x = rng.normal(size=(M, K))
    x[:, 5::128] *= 100
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    rc, rs = layer.quantize(x.astype(np.float32))
    ref = layer.linear(w[0], s[0], rc, rs)
    xv = layer.e4m3_values()[rc] * np.repeat(rs, 128, 1)[:, :K].astype(np.float64)
    wv = layer.e4m3_values()[w[0]] * np.repeat(np.repeat(s[0], 128, 0), 128, 1)[:N, :K].astype(np.float64)
    f32 = (K + 2) * 2.0 ** -24 * (np.abs(xv) @ np.abs(wv).T)
    eights = EIGHT * _loudest_of_eight(xv, wv)
    for yt in ("f32", "f16", "bf16"):
        got = q.fp8_linear(W, t, out_dtype=DT[yt]).double().cpu().numpy()
        room = f32 + (eights if yt == "bf16" and M > 32 else 0)
        assert (np.abs(got - ref) <= room + _half_unit(np.abs(ref) + room, yt)).all(), yt


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_rounding_to_nearest(M, N, K):
    """A 16-bit result is the float32 result rounded to nearest even; where the eights take part, off by no more
    than the rounding in norm."""
    announce(f"rounding M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K)
    W = _device_weights(*_weights(rng, 1, N, K))
    t, _ = _activations(rng, M, K, "bf16")
    wide = q.fp8_linear(W, t)
    assert torch.equal(q.fp8_linear(W, t, out_dtype=torch.float16), wide.to(torch.float16))
    half = q.fp8_linear(W, t, out_dtype=torch.bfloat16)
    if M <= 32:
        assert torch.equal(half, wide.to(torch.bfloat16))
    else:
        off = (half.double() - wide.double()).norm(dim=1) / wide.double().norm(dim=1)
        assert float(off.max()) <= 2.0 ** -7 / 12 ** 0.5 * 1.05 + 1e-4


@pytest.mark.parametrize("T,k,E,N,K", [(1, 6, 16, 256, 512), (70, 4, 8, 200, 400), (800, 2, 8, 1000, 528),
                                       (2048, 2, 8, 2570, 272), (2050, 2, 8, 2560, 256)])
def test_routed_float16_results_are_rounded_float32_ones(T, k, E, N, K):
    announce(f"routed rounding T={T} k={k} E={E} N={N} K={K}")
    rng = np.random.default_rng(T + E)
    W = _device_weights(*_weights(rng, E, N, K))
    t, _ = _activations(rng, T, K, "bf16")
    ids = _dev(np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32))
    assert torch.equal(q.moe_fp8(W, t, ids, out_dtype=torch.float16), q.moe_fp8(W, t, ids).to(torch.float16))
