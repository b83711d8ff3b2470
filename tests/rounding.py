"""Values with a bound on how far a float32 computation of them may be off.

Each step of a formula carries the first-order error of its inputs on and adds
its own rounding, at most half a unit: 2^-24 of its result.  ``sum`` takes the
longest chain of additions a value goes through.  Second-order terms are covered
by a factor of 1.01 where the bound is used (errors here are below 1e-4)."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


class Ev:
    def __init__(self, value, bound=0.0):
        self.v = np.asarray(value, np.float64)
        self.e = np.broadcast_to(np.asarray(bound, np.float64), self.v.shape)

    def __add__(self, o):
        o = o if isinstance(o, Ev) else Ev(o)
        v = self.v + o.v
        return Ev(v, self.e + o.e + U * np.abs(v))

    def __neg__(self):
        return Ev(-self.v, self.e)

    def __sub__(self, o):
        return self + (-(o if isinstance(o, Ev) else Ev(o)))

    def __mul__(self, o):
        o = o if isinstance(o, Ev) else Ev(o)
        v = self.v * o.v
        return Ev(v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + U * np.abs(v))

    __rmul__ = __mul__

    def sum(self, axis, chain):
        return Ev(self.v.sum(axis, keepdims=True), (self.e + chain * U * np.abs(self.v)).sum(axis, keepdims=True))

    def inv_sqrt(self):
        """1 / sqrt: a root and a quotient"""
        v = 1.0 / np.sqrt(self.v)
        return Ev(v, v * (0.5 * self.e / self.v + 2 * U))

    def check(self, got: torch.Tensor):
        """got, of its own type, is within the bound and one rounding to that type."""
        half = torch.finfo(got.dtype).eps / 2
        tiny = torch.finfo(got.dtype).smallest_normal * half  # half the spacing of the subnormals
        g = got.detach().cpu().double().numpy()
        assert g.shape == self.v.shape, (g.shape, self.v.shape)
        off, allowed = np.abs(g - self.v), 1.01 * self.e + half * (np.abs(self.v) + 1.01 * self.e) + tiny
        bad = ~(off <= allowed)
        assert not bad.any(), (int(bad.sum()), float((off / np.maximum(allowed, 1e-300)).max()))
