"""Bad arguments of the expert-selection and 8-bit calls of the binding raise
its own error before anything is allocated (no GPU needed)."""
import pytest
import torch

import dequant_iqk_moe_amd as q
from test_binding_sizes import FakeDev


@pytest.mark.parametrize("k", [-1, 0, 65])
def test_router_refuses_k(k):
    with pytest.raises(q.IqkValueError, match="k = "):
        q.router_topk(FakeDev((3, 64), torch.float32), k)


@pytest.mark.parametrize("shape", [(0, 4, 16), (2, 0, 16), (2, 4, 0)])
def test_weights_without_values(shape):
    E, out, n = shape
    with pytest.raises(q.IqkValueError, match="codes"):
        q.Fp8Weights(torch.zeros(shape, dtype=torch.float8_e4m3fn), torch.zeros(E, -(-out // 128), -(-n // 128)))
