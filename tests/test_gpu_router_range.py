"""Values at the ends of float32 in expert selection and its gradient, against
the 64-bit oracle.  Bars as in test_gpu_router."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from oracle import layer
from test_gpu_router import DT, _check, _dev

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu
INF = np.inf
LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("least", [-85.0, -60.0, -20.0])
def test_gradient_of_small_scores(least, dtype):
    """Sigmoid scores of e^-85 with weights divided by their sum: the gradient is
    w_j (1 - s_j) (g_j - sum g w), of the size of g, whatever the scores'."""
    announce(f"router grad of logits from {least} {dtype}")
    rng = np.random.default_rng(int(-least))
    T, E, k = 9, 40, 4
    l = least + rng.integers(0, 8, (T, E)) / 2
    dw = (rng.normal(size=(T, k)) * 10.0 ** rng.integers(0, 7, (T, 1))).astype(np.float32)
    ids, _ = layer.router(l, k, "sigmoid")
    ref = layer.router_grad(l, ids, dw, "sigmoid", True, 2.5)
    got = q.router_topk_grad(_dev(l, DT[dtype]), _dev(ids), _dev(dw), scoring="sigmoid", scale=2.5).double().cpu().numpy()
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    room = 1e-5 * 2.5 * np.abs(dw).max(1)[:, None] + half * np.abs(ref)
    assert (np.abs(got - ref) <= room).all()


