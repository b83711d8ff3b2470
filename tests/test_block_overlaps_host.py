"""Results that lie over a call's inputs where rows would be written before another workgroup has read them are
refused on the host (no GPU needed; the pointers are never followed)."""
import ctypes

import pytest

import dequant_iqk_moe_amd as q

E_ARG, E_HIP = -1, -8
F32, F16, BF16 = 0, 1, 2
T, N = 10, 64
FAR = 0x100000  # apart from everything else


def _norm(r, h, dtype=BF16, y_dtype=BF16, x=1 * FAR, y=2 * FAR):
    b = q._Block(T=T, n=N, dtype=dtype, y_dtype=y_dtype, weight_dtype=F32, gate_dtype=F32, gate_kind=0, alpha=1.0, beta=1.0, eps=1e-6,
                 x=x, y=y, post_weight=3 * FAR, gate=None, next_weight=4 * FAR)
    return q._lib.iqk_block_norm(ctypes.byref(b), r, h, None)


X, Y, R, H = 1 * FAR, 2 * FAR, 5 * FAR, 6 * FAR
BYTES = T * N * 2


@pytest.mark.parametrize("r,h,types", [
    (Y, H, (BF16, F32)), (R, Y, (BF16, F32)), (Y, X, (F16, F32)),           # the row of another type
    (Y + BYTES, H, (BF16, F32)), (R, Y + 2 * BYTES - 16, (BF16, F32)),      # its second half, its end
    (X + 2 * N, H, (BF16, BF16)), (R, X - 2 * N, (BF16, BF16)),             # a row further on or back
    (Y + 16, H, (BF16, BF16)), (R, Y - 16, (F32, F32)),
    (R, R + 2 * N, (BF16, BF16)), (R + 16, R, (F32, F32))])                 # each other
def test_norm_refuses_overlaps(r, h, types):
    assert _norm(r, h, *types) == E_ARG
    assert b"overlap" in q._lib.iqk_last_error()


INT8 = 4
SX, IDS, XS, OFF, PLACE = 1 * FAR, 2 * FAR, 3 * FAR, 4 * FAR, 5 * FAR


@pytest.mark.parametrize("k,xs,place", [
    (1, SX, PLACE), (4, SX, PLACE), (4, SX - 4 * BYTES + 2, PLACE), (2, SX + BYTES - 2, PLACE),
    (1, XS, IDS), (4, XS, IDS + 4 * (4 * T - 1)), (4, XS, IDS - 4 * (4 * T - 1))])
def test_sort_refuses_overlaps(k, xs, place):
    """In place, or over the end or the beginning of it."""
    assert q._lib.iqk_moe_sort(SX, BF16, IDS, T, k, 8, N, None, 0, xs, OFF, place, None) == E_ARG
    assert b"overlap" in q._lib.iqk_last_error()


@pytest.mark.parametrize("codes", [X, X + T * N * 4 - 16, X - T * N + 16])
def test_quantize_refuses_overlaps(codes):
    assert q._lib.iqk_int8_quantize(X, F32, T, N, codes, R, None) == E_ARG
    assert b"overlap" in q._lib.iqk_last_error()


@pytest.mark.parametrize("rows", [1, T, 100])
@pytest.mark.parametrize("x_dtype,scales", [(F32, None), (BF16, None), (INT8, R)])
@pytest.mark.parametrize("at", ["in place", "end", "beginning"])
@pytest.mark.parametrize("grouped", [False, True])
def test_products_refuse_overlaps(rows, x_dtype, scales, at, grouped):
    size = {F32: 4, BF16: 2, INT8: 1}[x_dtype]
    y = {"in place": X, "end": X + rows * N * size - 4, "beginning": X - rows * N * 4 + 4}[at]
    w = q._Int8Weights(1, N, N, 3 * FAR, N * N, 4 * FAR, N)
    tail = (rows, 7 * FAR, 1 << 19, y, F32, None)
    if grouped:
        rc = q._lib.iqk_int8_grouped(ctypes.byref(w), X, x_dtype, scales, 8 * FAR, *tail)
    else:
        rc = q._lib.iqk_int8_linear(ctypes.byref(w), X, x_dtype, scales, *tail)
    assert rc == E_ARG and b"overlap" in q._lib.iqk_last_error()
