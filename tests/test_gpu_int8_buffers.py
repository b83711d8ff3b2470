"""Caller's buffers of the 8-bit integer calls: written, and known to autograd as changed."""
import pytest
import torch

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu


def test_given_buffers_count_as_changed():
    x = torch.randn(6, 64, device="cuda")
    want = q.int8_quantize(x)
    for given in (dict(codes=torch.empty(6, 64, dtype=torch.int8, device="cuda")), dict(scales=torch.empty(6, device="cuda")),
                  dict(codes=torch.empty(6, 64, dtype=torch.int8, device="cuda"), scales=torch.empty(6, device="cuda"))):
        before = {m: t._version for m, t in given.items()}
        codes, scales = q.int8_quantize(x, **given)
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
        assert all(t._version > before[m] for m, t in given.items())
    w = q.Int8Weights(torch.randint(-9, 9, (1, 32, 64), dtype=torch.int8, device="cuda"), torch.rand(1, 32, device="cuda"))
    offsets = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    for call in (lambda **y: q.int8_linear(w, x, **y), lambda **y: q.int8_grouped(w, x, offsets, **y)):
        y = torch.empty(6, 32, device="cuda")
        before = y._version
        assert call(y=y) is y and torch.equal(y, call()) and y._version > before
