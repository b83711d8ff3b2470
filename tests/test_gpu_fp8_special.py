"""NaN and infinite values of x, of its scales and of the weights' scales in the
routed 8-bit product: they reach the pairs and the expert they belong to, on
every path."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from test_gpu_fp8 import DT, _activations, _dev, _device_weights, _weights

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu

# T, k, E, out, in and the path for float32 and for bfloat16 results
SIZES = [
    (2, 2, 4, 200, 400, ("few",), ("few",)),
    (40, 3, 6, 530, 400, ("tiles", 16, 128, 1), ("tiles", 16, 128, 1)),
    (150, 2, 8, 2060, 272, ("tiles", 32, 128, 1), ("tiles", 32, 128, 1)),
    (190, 2, 8, 2580, 256, ("tiles", 64, 128, 1), ("tiles", 64, 128, 1)),
    (580, 2, 8, 1030, 272, ("tiles", 128, 128, 1), ("tiles", 128, 128, 1)),
    (580, 2, 8, 4100, 256, ("tiles", 128, 256, 1), ("tiles", 128, 256, 1)),
    (1160, 2, 8, 5130, 272, ("tiles", 128, 256, 1), ("tiles", 256, 256, 1)),
]


def _setup(T, k, E, N, K, wide, bf16, slots):
    assert q.fp8_path(E, N, K, T, k) == wide and q.fp8_path(E, N, K, T, k, torch.bfloat16) == bf16
    rng = np.random.default_rng(T + N + slots)
    w, s = _weights(rng, E, N, K)
    t, _ = _activations(rng, T * slots, K, "f32")
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    return rng, w, s, t, ids


@pytest.mark.parametrize("T,k,E,N,K,wide,bf16", SIZES)
@pytest.mark.parametrize("shared", [True, False])
def test_rows_of_x(T, k, E, N, K, wide, bf16, shared):
    """A NaN in the depth's last chunk of one row, an infinity in another: those rows' pairs, and no other bit."""
    announce(f"special x {T} {k} {E} {N} {K} shared={shared}")
    slots = 1 if shared else k
    rng, w, s, t, ids = _setup(T, k, E, N, K, wide, bf16, slots)
    W, dids = _device_weights(w, s), _dev(ids)
    bad = t.clone()
    rows = [0, T * slots - 1]
    bad[rows[0], K - 1], bad[rows[1], 0] = float("nan"), float("inf")
    hit = torch.zeros(T, k, dtype=torch.bool, device="cuda")
    for r in rows:
        if shared:
            hit[r] = True
        else:
            hit.view(-1)[r] = True
    for yt in ("f32", "f16", "bf16"):
        clean = q.moe_fp8(W, t, dids, x_slots=slots, out_dtype=DT[yt])
        y = q.moe_fp8(W, bad, dids, x_slots=slots, out_dtype=DT[yt])
        assert torch.equal(y[~hit], clean[~hit])
        assert not torch.isfinite(y[hit]).any()
        codes, scales = q.fp8_quantize(t)
        scales[rows[0], -1], scales[rows[1], 0] = float("nan"), float("inf")
        y = q.moe_fp8(W, codes, dids, x_slots=slots, x_scales=scales, out_dtype=DT[yt])
        assert torch.equal(y[~hit], clean[~hit])
        assert not torch.isfinite(y[hit]).any()


@pytest.mark.parametrize("T,k,E,N,K,wide,bf16", SIZES)
def test_weights(T, k, E, N, K, wide, bf16):
    """A NaN code: its weight row of its expert.  A NaN or infinite scale: its 128 weight rows, or fewer at the edge."""
    announce(f"special weights {T} {k} {E} {N} {K}")
    rng, w, s, t, ids = _setup(T, k, E, N, K, wide, bf16, 1)
    dids = _dev(ids)
    one = int(ids[T - 1, 0])
    code = w.copy()
    code[one, N - 1, K - 1] = 0x7F
    for yt in ("f32", "f16", "bf16"):
        clean = q.moe_fp8(_device_weights(w, s), t, dids, out_dtype=DT[yt])
        at = (dids == one)[:, :, None] & (torch.arange(N, device="cuda") == N - 1)
        y = q.moe_fp8(_device_weights(code, s), t, dids, out_dtype=DT[yt])
        assert torch.isnan(y[at]).all() and torch.equal(y[~at], clean[~at])
        for value in (np.nan, np.inf):
            for block in (0, -1):
                bad = s.copy()
                bad[one, block, -1] = value
                cols = torch.arange(N, device="cuda") // 128 == (block if block == 0 else (N - 1) // 128)
                at = (dids == one)[:, :, None] & cols
                y = q.moe_fp8(_device_weights(w, bad), t, dids, out_dtype=DT[yt])
                assert not torch.isfinite(y[at]).any() and torch.equal(y[~at], clean[~at])
