"""Each kernel of the 8-bit products against the 64-bit oracle, at sizes whose
path is asserted: a change of the rules fails here instead of moving a case to
another kernel.  Bars as in test_gpu_fp8; 16-bit results are the float32
result's rounding, or (bfloat16 tiles of many rows) off by it in norm."""
import numpy as np
import pytest
import torch

from fp8_paths import DENSE, GROUPED, MANY_EXPERTS
from gpu_common import announce
from oracle import layer
from test_gpu_fp8 import BAR, _activations, _dev, _device_weights, _moe_check, _off, _weights

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu
# of a row's norm: root mean square of rounding at the low end of a binade, 5 % for its spread, 1e-4 for the sums
ROUNDED = 2.0 ** -7 / 12 ** 0.5 * 1.05 + 1e-4


def _check_rounding(call, exact_bf16):
    wide = call(torch.float32)
    assert torch.equal(call(torch.float16), wide.to(torch.float16))
    half = call(torch.bfloat16)
    if exact_bf16:
        assert torch.equal(half, wide.to(torch.bfloat16))
    elif wide.shape[-1] >= 200:
        off = (half.double() - wide.double()).norm(dim=-1) / wide.double().norm(dim=-1)
        assert float(off.max()) <= ROUNDED
    return wide


@pytest.mark.parametrize("size,wide,bf16", DENSE)
def test_dense(size, wide, bf16):
    M, N, K = size
    announce(f"dense path M={M} N={N} K={K}")
    assert q.fp8_path(1, N, K, M) == wide and q.fp8_path(1, N, K, M, out_dtype=torch.bfloat16) == bf16
    rng = np.random.default_rng(M + N + K)
    w, s = _weights(rng, 1, N, K)
    W = _device_weights(w, s)
    t, x = _activations(rng, M, K, "bf16")
    ref = layer.linear(w[0], s[0], *layer.quantize(x))
    y = _check_rounding(lambda dt: q.fp8_linear(W, t, out_dtype=dt), bf16[0] != "tiles")
    assert _off(y, ref) <= BAR["f32"]


@pytest.mark.parametrize("counts,N,wide,bf16", GROUPED)
@pytest.mark.parametrize("K", [272, 256])
def test_grouped(counts, N, wide, bf16, K):
    announce(f"grouped path {counts} N={N} K={K}")
    E, P = len(counts), sum(counts)
    assert q.fp8_path(E, N, K, P, 1) == wide and q.fp8_path(E, N, K, P, 1, torch.bfloat16) == bf16
    rng = np.random.default_rng(P + N + K)
    w, s = _weights(rng, E, N, K)
    ids = rng.permutation(np.repeat(np.arange(E), counts)).astype(np.int32)[:, None]
    for yt in ("f32", "bf16"):
        _moe_check(w, s, ids, 1, "bf16", yt, rng)
    W, t, dids = _device_weights(w, s), _activations(rng, P, K, "f32")[0], _dev(ids)
    _check_rounding(lambda dt: q.moe_fp8(W, t, dids, out_dtype=dt), bf16[1] < 128)


@pytest.mark.parametrize("E,T,k,N,K", MANY_EXPERTS)
def test_many_experts(E, T, k, N, K):
    """The last expert's offsets and tiles, where the experts fill the workgroup that counts them and one past that."""
    announce(f"many experts E={E} T={T} k={k}")
    rng = np.random.default_rng(E + T)
    w, s = _weights(rng, E, N, K)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[:40] = E - 1                     # more than a tile at the last expert
    ids[41, 0], ids[T - 1, 1] = E, -1
    for slots in (1, k):
        _moe_check(w, s, ids, slots, "bf16", "f32", rng)
