"""One mixture-of-experts layer from its router's logits to its output.

    python examples/moe_layer.py [--tokens T] [--steps N]

The layer: a router (sigmoid scores, balance bias, groups of experts) chooses k
experts per token; the routed experts are IQ2_K (``moe_auto`` with the SwiGLU
and combine steps) or kept in 8 bits (``moe_fp8``); a shared expert in 8 bits
(``fp8_linear``) sees every token.  Then the router is recalibrated: with the
IQ2_K experts frozen, its weights descend on the distance to the output of the
8-bit experts they were made beside (``router_topk_grad``).

Weights and inputs are random; the sizes are small enough to run anywhere.
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import dequant_iqk_moe_amd as q
import synth

HIDDEN, INNER, EXPERTS, K = 512, 512, 16, 4
ROUTING = dict(scoring="sigmoid", n_group=4, topk_group=2, group_top=2, renorm=True, scale=2.5)


def to_fp8(w: torch.Tensor) -> q.Fp8Weights:
    """Weights [E, out, in] to 8 bits, one scale per 128 x 128 block (sizes here are multiples of 128)."""
    E, out, n = w.shape
    blocks = w.float().view(E, out // 128, 128, n // 128, 128)
    scales = blocks.abs().amax((2, 4)) / 448.0
    codes = (blocks / scales[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.Fp8Weights(codes.view(E, out, n), scales.contiguous())


class Layer:
    def __init__(self, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.gate = (torch.randn(EXPERTS, HIDDEN, generator=g) / HIDDEN**0.5).cuda()
        self.bias = (torch.randint(-20, 21, (EXPERTS,), generator=g) * 0.001).cuda()
        self.values = synth.values_table(seed + 1)
        # gate/up rows [0, I) gate and [I, 2I) up; down [hidden, I]
        self.gate_up = q.Weights.from_wire(q.IQ2_K, EXPERTS, 2 * INNER, HIDDEN,
                                           synth.wire(q.IQ2_K, EXPERTS * 2 * INNER, HIDDEN, seed + 2, sigma=5e-4))
        self.down = q.Weights.from_wire(q.IQ2_K, EXPERTS, HIDDEN, INNER,
                                        synth.wire(q.IQ2_K, EXPERTS * HIDDEN, INNER, seed + 3, sigma=5e-4))
        # the same experts in 8 bits, and a shared one
        wide = lambda w: q.dequant(w, self.values, out_dtype=torch.float32).view(w.experts, w.out, w.in_features)
        self.gate_up8, self.down8 = to_fp8(wide(self.gate_up)), to_fp8(wide(self.down))
        self.shared_gate_up = to_fp8((torch.randn(1, 2 * INNER, HIDDEN, generator=g) / HIDDEN**0.5).cuda())
        self.shared_down = to_fp8((torch.randn(1, HIDDEN, INNER, generator=g) / INNER**0.5).cuda())

    def route(self, x: torch.Tensor):
        logits = x.float() @ self.gate.t()
        ids, weights = q.router_topk(logits, K, bias=self.bias, **ROUTING)
        return logits, ids, weights

    def routed(self, x: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
        """Outputs of the chosen IQ2_K experts, [T, k, hidden]."""
        gu, _ = q.moe_auto(self.gate_up, x, ids, self.values)
        return q.moe_auto(self.down, q.swiglu(gu), ids, self.values, x_slots=K)[0]

    def routed8(self, x: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
        """The same from the 8-bit experts."""
        h = q.swiglu(q.moe_fp8(self.gate_up8, x, ids))
        return q.moe_fp8(self.down8, h.view(-1, INNER), ids, x_slots=K)

    def shared(self, x: torch.Tensor) -> torch.Tensor:
        return q.fp8_linear(self.shared_down, q.swiglu(q.fp8_linear(self.shared_gate_up, x)))

    def __call__(self, x: torch.Tensor, eight_bits: bool = False) -> torch.Tensor:
        _, ids, weights = self.route(x)
        y = self.routed8(x, ids) if eight_bits else self.routed(x, ids)
        return q.combine(y, weights) + self.shared(x)


def recalibrate(layer: Layer, x: torch.Tensor, steps: int, rate: float = 0.2) -> list[float]:
    """Descends the router's weights, from half of what they should be, on the
    distance between the layer with its IQ2_K experts and the output it had with
    its 8-bit ones.  (The gradient holds the choice of experts fixed, so the loss
    jumps where a step changes a choice.)"""
    target = layer(x, eight_bits=True)
    layer.gate *= 0.5
    losses = []
    for _ in range(steps):
        logits, ids, weights = layer.route(x)
        y = layer.routed(x, ids)
        off = q.combine(y, weights) + layer.shared(x) - target
        losses.append(float(off.square().mean()))
        d_weights = (y * (2.0 / off.numel() * off)[:, None, :]).sum(-1)
        d_logits = q.router_topk_grad(logits, ids, d_weights, scoring=ROUTING["scoring"], renorm=ROUTING["renorm"],
                                      scale=ROUTING["scale"])
        layer.gate -= rate * (d_logits.t() @ x.float())
    return losses


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    layer = Layer()
    x = torch.randn(a.tokens, HIDDEN, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).cuda()
    y, y8 = layer(x), layer(x, eight_bits=True)
    off = float((y - y8).norm() / y.norm())
    losses = recalibrate(layer, x, a.steps)
    print(f"{a.tokens} tokens, top-{K} of {EXPERTS} experts: output {tuple(y.shape)}, "
          f"8-bit experts differ from IQ2_K ones by {off:.2e}")
    print(f"recalibration: loss {losses[0]:.3e} -> {losses[-1]:.3e} in {a.steps} steps")
    return {"off": off, "losses": losses, "layer": layer, "x": x}


if __name__ == "__main__":
    main()
