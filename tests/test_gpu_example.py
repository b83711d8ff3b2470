"""The example layer against the same layer in float64 from dequantized weights.

Bar: the steps round activations to bfloat16 (h, 2^-9 of a value in the mean)
and to e4m3 (2^-5 in the mean of a value, 3 % in norm), the latter twice in a
row on the 8-bit paths; the layer's output sums them: 8 % in norm with 8-bit
experts throughout, 6 % with the shared expert alone in 8 bits."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def _silu_mul(gu):
    g, u = gu.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def test_example_layer():
    import dequant_iqk_moe_amd as q
    import moe_layer as m
    from oracle import layer as oracle_layer

    got = m.main(["--tokens", "48", "--steps", "12"])
    layer, x = m.Layer(), got["x"]
    wide = lambda w: q.dequant(w, layer.values).view(w.experts, w.out, w.in_features).double()
    wide8 = lambda w: (w.codes.float() * w.scales.repeat_interleave(128, 1).repeat_interleave(128, 2)).double()
    xd = x.double()
    logits = (x.float() @ layer.gate.t()).cpu().numpy()
    ids, weights = oracle_layer.router(logits, m.K, bias=layer.bias.cpu().numpy(), **m.ROUTING)
    got_ids = layer.route(x)[1].cpu().numpy()
    np.testing.assert_array_equal(got_ids, ids)
    gu, dn = wide(layer.gate_up), wide(layer.down)
    y = torch.zeros(48, m.HIDDEN, dtype=torch.float64, device="cuda")
    for t in range(48):
        for j in range(m.K):
            e = int(ids[t, j])
            y[t] += float(weights[t, j]) * (dn[e] @ _silu_mul(gu[e] @ xd[t]))
    shared = _silu_mul(xd @ wide8(layer.shared_gate_up)[0].t()) @ wide8(layer.shared_down)[0].t()
    want = y + shared
    for eight, bar in ((False, 0.06), (True, 0.08)):
        off = float((layer(x, eight_bits=eight).double() - want).norm() / want.norm())
        assert off <= bar, (eight, off)
    # the choice of experts jumps from step to step, and the loss with it: its best step
    assert min(got["losses"]) < 0.5 * got["losses"][0]
