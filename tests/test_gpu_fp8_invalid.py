"""Pairs whose id lies outside the experts held here, as on a device with a
share of them: NaN rows, whole, and nothing else; the others as without them."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from test_gpu_fp8 import DT, _activations, _dev, _device_weights, _weights

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,N,K", [(3, 2, 4, 33, 144), (60, 3, 6, 1, 272), (61, 3, 6, 530, 272), (700, 2, 8, 263, 144),
                                       (5000, 2, 5, 129, 144), (600, 4, 1100, 77, 144)])
@pytest.mark.parametrize("share", [0.125, 0.0])
@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
def test_most_ids_are_elsewhere(T, k, E, N, K, share, yt):
    announce(f"invalid ids T={T} k={k} E={E} N={N} share={share} {yt}")
    rng = np.random.default_rng(T + N)
    W = _device_weights(*_weights(rng, E, N, K))
    t, _ = _activations(rng, T, K, "bf16")
    all_ids = rng.integers(0, E, (T, k)).astype(np.int32)
    out = rng.random((T, k)) >= share
    ids = np.where(out, rng.choice(np.int32([-1, E, E + 7, 2 ** 31 - 1, -2 ** 31]), (T, k)), all_ids).astype(np.int32)
    want = q.moe_fp8(W, t, _dev(all_ids), out_dtype=DT[yt])
    buf = torch.full((T * k * N + 64,), 7.0, dtype=DT[yt], device="cuda")
    y = buf[1:1 + T * k * N].view(T, k, N)
    q.moe_fp8(W, t, _dev(ids), y=y)
    gone = torch.from_numpy(out).cuda()
    assert torch.isnan(y[gone]).all() and torch.equal(y[~gone], want[~gone])
    assert (buf[0] == 7) and (buf[1 + T * k * N:] == 7).all()
