"""Workspace of the routed 8-bit product for x that comes as codes."""
import numpy as np
import pytest
import torch

from test_gpu_fp8 import _activations, _dev, _device_weights, _weights

import dequant_iqk_moe_amd as q


def _round256(n):
    return -(-n // 256) * 256


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,slots", [(300, 2, 8, 1), (5000, 2, 5, 2), (600, 4, 1100, 1), (1, 1, 1, 1)])
def test_codes_need_no_memory_for_codes(T, k, E, slots):
    """They do with the grouping's share, and leave what lies behind it alone."""
    N, K = 130, 144
    rng = np.random.default_rng(T)
    W = _device_weights(*_weights(rng, E, N, K))
    t, _ = _activations(rng, T * slots, K, "bf16")
    ids = _dev(np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32))
    full = q.moe_fp8_workspace_bytes(W, T, k, slots)
    quantized = _round256(T * slots * K) + _round256(T * slots * 2 * 4)
    need = full - quantized if full else 0
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    codes, scales = q.fp8_quantize(t)
    y = q.moe_fp8(W, codes, ids, x_slots=slots, x_scales=scales, workspace=ws[:need])
    assert (ws[need:] == 0x5A).all()
    assert torch.equal(y, q.moe_fp8(W, t, ids, x_slots=slots))
    assert torch.equal(y, q.moe_fp8(W, codes, ids, x_slots=slots, x_scales=scales))
    if need:
        with pytest.raises(q.IqkValueError, match=f"workspace needs {need} bytes"):
            q.moe_fp8(W, codes, ids, x_slots=slots, x_scales=scales, workspace=ws[:need - 1])
