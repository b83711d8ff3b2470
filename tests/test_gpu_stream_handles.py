"""The default stream's handle as the stream argument, from within another stream: calls, results' memory and
gradients belong to the default stream."""
import pytest
import torch

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu


def test_default_streams_handle():
    x = torch.randn(300, 256, device="cuda")
    w, dh = torch.ones(256, device="cuda"), torch.randn(300, 256, device="cuda")
    want, want_grad = q.block_norm(x, next_weight=w)[1], q.block_norm_grad(x, None, None, dh, next_weight=w)[0]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        for given in (0, torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream):
            with q._on(given):
                assert torch.cuda.current_stream() == torch.cuda.default_stream()
            assert torch.cuda.current_stream() == other
            leaf, place = x.clone().requires_grad_(), torch.arange(300, dtype=torch.int32, device="cuda").view(300, 1)
            torch.cuda.synchronize()
            _, h = q.block_norm(leaf, next_weight=w, stream=given)
            y = q.moe_unsort(x, place, stream=given)
            torch.cuda.synchronize()
            assert torch.equal(h, want) and torch.equal(y, x)
            h.backward(dh)
            torch.cuda.synchronize()
            assert torch.equal(leaf.grad, want_grad)
