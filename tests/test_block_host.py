"""Refusals of the operators around the routed experts: every bad argument fails
before any HIP call (no GPU needed; the pointers are never followed)."""
import ctypes

import pytest
import torch

import dequant_iqk_moe_amd as q
from test_binding_sizes import FakeDev

P = 0x1000
E_ARG, E_SHAPE, E_SIZE = -1, -3, -6
F32, F16, BF16, E4M3, INT8 = 0, 1, 2, 3, 4


@pytest.mark.parametrize("change,code", [
    (dict(x=None), E_ARG), (dict(x=P + 1), E_ARG), (dict(dtype=E4M3), E_ARG), (dict(dtype=INT8), E_ARG), (dict(ids=None), E_ARG),
    (dict(ids=P + 2), E_ARG), (dict(T=-1), E_ARG), (dict(T=1 << 23), E_ARG), (dict(k=0), E_ARG), (dict(k=65), E_ARG),
    (dict(E=0), E_ARG), (dict(E=2049), E_ARG), (dict(n=0), E_ARG), (dict(n=(1 << 20) + 1), E_ARG), (dict(xs=None), E_ARG),
    (dict(xs=P + 1), E_ARG), (dict(offsets=None), E_ARG), (dict(offsets=P + 1), E_ARG), (dict(place=None), E_ARG),
    (dict(place=P + 2), E_ARG), (dict(T=3000), E_SIZE), (dict(T=3000, ws=P), E_SIZE), (dict(T=3000, nbytes=1 << 20), E_SIZE),
    (dict(T=3000, ws=P + 2, nbytes=1 << 20), E_ARG)])
def test_sort_refuses(change, code):
    a = dict(x=P, dtype=BF16, ids=P, T=100, k=4, E=64, n=33, ws=None, nbytes=0, xs=P, offsets=P, place=P, stream=None)
    a.update(change)
    assert q._lib.iqk_moe_sort(*a.values()) == code
    assert q._lib.iqk_last_error()


def test_sort_workspace():
    for T, k in ((0, 1), (1, 64), (1024, 8), (2048, 2), (2896, 1), (128, 64)):
        assert q.moe_sort_workspace_bytes(T, k, 64) == 0
    for T, k, slices in ((1025, 8, 9), (2049, 2, 5), (2897, 1, 3), (129, 64, 9), (2049, 4, 9)):
        assert q.moe_sort_workspace_bytes(T, k, 64) == slices * 65 * 4  # a slice per 1024 pairs
    assert q.moe_sort_workspace_bytes(1 << 22, 4, 2048) == 128 * 2049 * 4
    for bad in ((-1, 4, 64), (4, 0, 64), (4, 4, 0), (1 << 24, 2, 64)):
        with pytest.raises(q.IqkValueError):
            q.moe_sort_workspace_bytes(*bad)


@pytest.mark.parametrize("change", [
    dict(ys=None), dict(ys=P + 2), dict(dt=E4M3), dict(place=None), dict(place=P + 1), dict(w=P + 1), dict(T=-1), dict(k=0),
    dict(k=65), dict(T=1 << 23), dict(n=0), dict(y=None), dict(y=P + 1), dict(ydt=INT8)])
def test_unsort_refuses(change):
    a = dict(ys=P, dt=F32, place=P, w=P, T=10, k=4, n=33, y=P, ydt=BF16, stream=None)
    a.update(change)
    assert q._lib.iqk_moe_unsort(*a.values()) == E_ARG


@pytest.mark.parametrize("change", [
    dict(dy=None), dict(dy=P + 1), dict(ddt=E4M3), dict(ys=None), dict(ys=P + 2), dict(dt=7), dict(place=None), dict(w=P + 2),
    dict(T=-1), dict(k=0), dict(n=0), dict(d_ys=P + 2), dict(d_w=P + 2), dict(d_ys=None, d_w=None)])
def test_unsort_grad_refuses(change):
    a = dict(dy=P, ddt=BF16, ys=P, dt=F32, place=P, w=P, T=10, k=4, n=33, d_ys=P, d_w=P, stream=None)
    a.update(change)
    assert q._lib.iqk_moe_unsort_grad(*a.values()) == E_ARG


def test_unsort_of_no_tokens():
    assert q._lib.iqk_moe_unsort(None, F32, None, None, 0, 4, 33, None, F32, None) == 0
    assert q._lib.iqk_moe_unsort_grad(None, F32, None, F32, None, None, 0, 4, 33, None, None, None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(x=None), E_ARG), (dict(x=P + 8), E_ARG), (dict(dtype=INT8), E_ARG), (dict(rows=-1), E_ARG),
    (dict(rows=(1 << 24) + 1), E_ARG), (dict(n=0), E_ARG), (dict(n=24), E_SHAPE), (dict(n=(1 << 16) + 16), E_ARG),
    (dict(codes=None), E_ARG), (dict(codes=P + 8), E_ARG), (dict(scales=None), E_ARG), (dict(scales=P + 2), E_ARG)])
def test_quantize_refuses(change, code):
    a = dict(x=P, dtype=F32, rows=3, n=256, codes=P, scales=P, stream=None)
    a.update(change)
    assert q._lib.iqk_int8_quantize(*a.values()) == code


def _w(experts=1, out=256, in_=512, codes=P, nbytes=None, scales=P, count=None):
    nb = experts * out * in_ if nbytes is None else nbytes
    ns = experts * out if count is None else count
    return q._Int8Weights(experts, out, in_, codes, max(nb, 0), scales, max(ns, 0))


@pytest.mark.parametrize("weights,code", [
    (dict(experts=0), E_ARG), (dict(out=0), E_ARG), (dict(in_=0), E_ARG), (dict(in_=520), E_SHAPE),
    (dict(in_=(1 << 16) + 16), E_ARG), (dict(out=1 << 20, in_=1 << 12), E_ARG), (dict(codes=None), E_ARG),
    (dict(codes=P + 8), E_ARG), (dict(scales=None), E_ARG), (dict(scales=P + 1), E_ARG), (dict(nbytes=256 * 512 - 1), E_SIZE),
    (dict(count=255), E_SIZE)])
@pytest.mark.parametrize("grouped", [False, True])
def test_products_refuse_weights(weights, code, grouped):
    assert _product(_w(**weights), grouped) == code


def _product(w, grouped, **change):
    a = dict(x=P, dtype=BF16, xs=None, offsets=P, M=100, ws=P, nbytes=1 << 20, y=P, ydt=F32, stream=None)
    a.update(change)
    if not grouped:
        del a["offsets"]
    return (q._lib.iqk_int8_grouped if grouped else q._lib.iqk_int8_linear)(ctypes.byref(w), *a.values())


@pytest.mark.parametrize("change,code", [
    (dict(x=None), E_ARG), (dict(x=P + 8), E_ARG), (dict(dtype=E4M3), E_ARG), (dict(dtype=5), E_ARG), (dict(xs=P), E_ARG),
    (dict(dtype=INT8), E_ARG), (dict(dtype=INT8, xs=P + 1), E_ARG), (dict(M=-1), E_ARG), (dict(M=(1 << 24) + 1), E_ARG),
    (dict(ws=None), E_SIZE), (dict(nbytes=16), E_SIZE), (dict(ws=P + 8), E_ARG), (dict(y=None), E_ARG), (dict(ydt=INT8), E_ARG),
    (dict(y=P + 2), E_ARG)])
@pytest.mark.parametrize("grouped", [False, True])
def test_products_refuse(change, code, grouped):
    assert _product(_w(), grouped, **change) == code


def test_products_refuse_what_is_their_own():
    assert _product(_w(experts=2), False) == E_ARG
    assert _product(_w(experts=2049), True) == E_ARG
    assert _product(_w(experts=2), True, offsets=None) == E_ARG
    assert _product(_w(experts=2), True, offsets=P + 2) == E_ARG
    for grouped in (False, True):
        assert _product(_w(), grouped, M=0, x=None, y=None, ws=None, nbytes=0, **({"offsets": None} if grouped else {})) == 0


def test_product_workspaces():
    need = ctypes.c_size_t()
    L, w = q._lib, _w(experts=1)
    for dtype, want in ((BF16, 100 * 512 + 512), (INT8, 0)):
        assert L.iqk_int8_linear_workspace(ctypes.byref(w), 100, dtype, ctypes.byref(need)) == 0 and need.value == want
        assert L.iqk_int8_grouped_workspace(ctypes.byref(w), 100, dtype, ctypes.byref(need)) == 0 and need.value == want + 256
    assert L.iqk_int8_linear_workspace(ctypes.byref(w), 4, BF16, ctypes.byref(need)) == 0 and need.value == 0
    assert L.iqk_int8_linear_workspace(ctypes.byref(w), 16, E4M3, ctypes.byref(need)) == E_ARG
    assert L.iqk_int8_linear_workspace(ctypes.byref(w), 16, BF16, None) == E_ARG


def _block(**change):
    a = dict(T=10, n=33, dtype=BF16, y_dtype=F32, weight_dtype=F32, gate_dtype=F32, gate_kind=1, alpha=1.0, beta=1.0, eps=1e-6,
             x=P, y=P, post_weight=P, gate=P, next_weight=P)
    a.update(change)
    return q._Block(**a)


BAD_BLOCKS = [
    dict(T=-1), dict(T=(1 << 24) + 1), dict(n=0), dict(n=8193), dict(dtype=E4M3), dict(y_dtype=F16), dict(weight_dtype=9),
    dict(gate_dtype=INT8), dict(gate_kind=4), dict(gate_kind=-1), dict(gate_kind=0), dict(gate=None), dict(alpha=float("inf")),
    dict(beta=float("nan")), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None),
    dict(x=P + 1), dict(y=P + 2), dict(post_weight=P + 2), dict(gate=P + 1), dict(next_weight=P + 1), dict(y=None),
    dict(y=None, gate=None, gate_kind=0), dict(y=None, post_weight=None),
    dict(y=None, post_weight=None, gate=None, gate_kind=0, next_weight=None),
    dict(y=None, post_weight=None, gate=None, gate_kind=0, alpha=0.5)]


@pytest.mark.parametrize("change", BAD_BLOCKS)
def test_norm_refuses_blocks(change):
    b = _block(**change)
    r = None if "y" in change and change["y"] is None else P
    h = None if change.get("next_weight", 1) is None else P * 2
    assert q._lib.iqk_block_norm(ctypes.byref(b), r, h, None) == E_ARG
    assert q._lib.iqk_block_norm_grad(ctypes.byref(b), P, None, P, None, None, None, None, None, 0, None) == E_ARG


@pytest.mark.parametrize("block,r,h", [
    ({}, None, P), ({}, P, None), ({}, P, P), ({}, P + 1, 2 * P), ({}, P, 2 * P + 1), (dict(next_weight=None), P, 2 * P),
    (dict(y=None, post_weight=None, gate=None, gate_kind=0), P, 2 * P)])
def test_norm_refuses_results(block, r, h):
    b = _block(**block)
    assert q._lib.iqk_block_norm(ctypes.byref(b), r, h, None) == E_ARG


@pytest.mark.parametrize("block,change,code", [
    ({}, dict(dr=None, dh=None), E_ARG), (dict(next_weight=None), {}, E_ARG), (dict(next_weight=None), dict(dh=None), E_ARG),
    (dict(post_weight=None), {}, E_ARG), (dict(gate=None, gate_kind=0), {}, E_ARG),
    (dict(y=None, post_weight=None, gate=None, gate_kind=0), dict(d_post=None, d_gate=None), E_ARG),
    ({}, dict(dr=P + 1), E_ARG), ({}, dict(dh=P + 1), E_ARG), ({}, dict(dx=P + 1), E_ARG), ({}, dict(dy=P + 2), E_ARG),
    ({}, dict(d_post=P + 2), E_ARG), ({}, dict(d_gate=P + 2), E_ARG), ({}, dict(d_next=P + 2), E_ARG), ({}, dict(ws=None), E_SIZE),
    ({}, dict(nbytes=64), E_SIZE), ({}, dict(ws=P + 8), E_ARG)])
def test_norm_grad_refuses(block, change, code):
    a = dict(dr=P, dh=P, dx=P, dy=P, d_post=P, d_gate=P, d_next=P, ws=P, nbytes=1 << 20, stream=None)
    a.update(change)
    b = _block(**block)
    assert q._lib.iqk_block_norm_grad(ctypes.byref(b), *a.values()) == code


def test_norm_of_no_tokens():
    b = _block(T=0, x=None, y=None, post_weight=None, gate=None, next_weight=None, gate_kind=0)
    assert q._lib.iqk_block_norm(ctypes.byref(b), None, None, None) == 0
    assert q._lib.iqk_block_norm_grad(ctypes.byref(b), None, None, None, None, None, None, None, None, 0, None) == 0


def test_binding_refuses_wrong_sizes():
    V = q.IqkValueError
    f = lambda *shape, dtype=torch.float32: Fake(shape, dtype)
    i32 = torch.int32
    for call in (
            lambda: q.moe_sort(f(3, 8), f(2, 4, dtype=i32), 8), lambda: q.moe_sort(f(24), f(3, 4, dtype=i32), 8),
            lambda: q.moe_sort(f(3, 8, dtype=torch.float64), f(3, 4, dtype=i32), 8, xs=f(12, 8), offsets=f(9, dtype=i32), place=f(3, 4, dtype=i32)),
            lambda: q.moe_sort(f(3, 8), f(3, 4, dtype=i32), 8, xs=f(11, 8), offsets=f(9, dtype=i32), place=f(3, 4, dtype=i32)),
            lambda: q.moe_sort(f(3, 8), f(3, 4, dtype=i32), 8, xs=f(12, 8), offsets=f(8, dtype=i32), place=f(3, 4, dtype=i32)),
            lambda: q.moe_sort(f(3, 8), f(3, 4, dtype=torch.int64), 8, xs=f(12, 8), offsets=f(9, dtype=i32), place=f(3, 4, dtype=i32)),
            lambda: q.moe_unsort(f(11, 8), f(3, 4, dtype=i32)),
            lambda: q.moe_unsort(f(12, 8), f(3, 4, dtype=i32), f(3, 3)),
            lambda: q.moe_unsort(f(12, 8), f(3, 4, dtype=i32), f(3, 4, dtype=torch.float16)),
            lambda: q.moe_unsort(f(12, 8), f(3, 4, dtype=i32), y=f(3, 7)),
            lambda: q.moe_unsort(f(12, 8), f(3, 4, dtype=i32), y=f(3, 8, dtype=torch.int32)),
            lambda: q.moe_unsort_grad(f(2, 8), f(12, 8), f(3, 4, dtype=i32), f(3, 4), d_ys=f(12, 8), d_weights=f(3, 4)),
            lambda: q.moe_unsort_grad(f(3, 8), f(12, 8), f(3, 4, dtype=i32), f(3, 4), d_ys=f(12, 7), d_weights=f(3, 4)),
            lambda: q.moe_unsort_grad(f(3, 8), f(12, 8), f(3, 4, dtype=i32), None, want_ys=False),
            lambda: q.int8_quantize(f(3, 64, dtype=torch.int8)), lambda: q.int8_quantize(f()),
            lambda: q.int8_quantize(f(3, 64), codes=f(3, 63, dtype=torch.int8), scales=f(3)),
            lambda: q.Int8Weights(torch.zeros(2, 4, 16), torch.zeros(2, 4)),
            lambda: q.Int8Weights(torch.zeros(2, 4, 16, dtype=torch.int8), torch.zeros(2, 3)),
            lambda: q.Int8Weights(torch.zeros(2, 0, 16, dtype=torch.int8), torch.zeros(2, 0)),
            lambda: q.int8_linear(_weights(), f(3, 15)), lambda: q.int8_linear(_weights(), f(3, 16, dtype=torch.float64)),
            lambda: q.int8_linear(_weights(), f(3, 16), x_scales=f(2)), lambda: q.int8_linear(_weights(), f(3, 16), y=f(3, 5)),
            lambda: q.int8_grouped(_weights(), f(3, 16), f(4, dtype=i32)), lambda: q.int8_grouped(_weights(), f(3, 16), f(3)),
            lambda: q.int8_grouped(_weights(), f(16), f(3, dtype=i32)),
            lambda: q.block_norm(f(3, 8), f(8, 3), r=f(3, 8)), lambda: q.block_norm(f(3, 8), f(24), r=f(3, 8)),
            lambda: q.block_norm(f(3, 8), f(3, 7), r=f(3, 8)), lambda: q.block_norm(f(3, 8), f(3, 8), r=f(3, 7)),
            lambda: q.block_norm(f(3, 8), f(3, 8), post_weight=f(7)), lambda: q.block_norm(f(3, 8), f(3, 8), gate=f(3)),
            lambda: q.block_norm(f(3, 8), f(3, 8), gate=f(8, 3)),
            lambda: q.block_norm(f(3, 8), f(3, 8), post_weight=f(8), next_weight=f(8, dtype=torch.float16)),
            lambda: q.block_norm_grad(f(3, 8), f(3, 8), f(3, 7)), lambda: q.block_norm(f(3, 8, dtype=torch.int8), f(3, 8))):
        with pytest.raises(V):
            call()


class Fake(FakeDev):
    requires_grad = False
    at = -1

    def get_device(self):
        return self.at


def _weights():
    w = q.Int8Weights(torch.zeros(2, 4, 16, dtype=torch.int8), torch.zeros(2, 4))
    w.codes, w.scales = Fake((2, 4, 16), torch.int8), Fake((2, 4), torch.float32)
    return w


def test_binding_refuses_host_and_strided_tensors():
    V = q.IqkValueError
    x = torch.zeros(4, 64)
    with pytest.raises(V, match="device tensor"):
        q.int8_quantize(x, codes=torch.zeros(4, 64, dtype=torch.int8), scales=torch.zeros(4))
    with pytest.raises(V, match="device tensor"):
        q.block_norm(x, x)
    with pytest.raises(V):
        q.moe_unsort(x, torch.zeros(2, 2, dtype=torch.int32))


def test_binding_refuses_another_device(monkeypatch):
    """Kernels run on the current device: a tensor on another one is refused, not read from there."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = Fake((4, 64), torch.float32)
    x.at = 1
    for call in (lambda: q.int8_quantize(x), lambda: q.block_norm(x, x), lambda: q.moe_unsort(x, Fake((2, 2), torch.int32)),
                 lambda: q.moe_sort(x, Fake((4, 2), torch.int32), 4)):
        with pytest.raises(q.IqkValueError, match="cuda:1"):
            call()
