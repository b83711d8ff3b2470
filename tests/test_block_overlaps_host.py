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
