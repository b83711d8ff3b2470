"""Refusals of the expert-selection and 8-bit calls: every bad argument fails
before any HIP call (no GPU needed; the pointers are never followed)."""
import ctypes

import pytest
import torch

import dequant_iqk_moe_amd as q
from test_binding_sizes import FakeDev

P = 0x1000
E_ARG, E_SHAPE, E_SIZE = -1, -3, -6
F32, F16, BF16, E4M3 = 0, 1, 2, 3


def _router(**change):
    a = dict(logits=P, dtype=F32, T=2, E=64, k=4, scoring=0, bias=None, n_group=1, topk_group=1, group_top=1,
             renorm=1, scale=1.0, ids=P, weights=P, stream=None)
    a.update(change)
    return q._lib.iqk_router_topk(*a.values())


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(logits=P + 2), dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(E=0), dict(E=1025),
    dict(k=0), dict(k=65, E=128), dict(k=5, E=4), dict(scoring=2), dict(n_group=0), dict(n_group=3), dict(n_group=65, E=65),
    dict(n_group=4, topk_group=5), dict(topk_group=0), dict(group_top=0), dict(group_top=3), dict(renorm=2),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(ids=None), dict(weights=None), dict(bias=P + 1)])
def test_router_refuses(change):
    assert _router(**change) == E_ARG
    assert q._lib.iqk_last_error()


def test_router_of_no_tokens():
    assert _router(T=0, logits=None, ids=None, weights=None) == 0


@pytest.mark.parametrize("change", [dict(logits=None), dict(ids=None), dict(dw=None), dict(out=None), dict(out=P + 1),
                                    dict(E=2000), dict(k=0), dict(scoring=-1), dict(renorm=3), dict(T=-2)])
def test_router_grad_refuses(change):
    a = dict(logits=P, dtype=BF16, ids=P, dw=P, T=2, E=64, k=4, scoring=1, renorm=1, scale=1.0, out=P, stream=None)
    a.update(change)
    assert q._lib.iqk_router_topk_grad(*a.values()) == E_ARG


@pytest.mark.parametrize("change,code", [
    (dict(x=None), E_ARG), (dict(x=P + 8), E_ARG), (dict(dtype=E4M3), E_ARG), (dict(rows=-1), E_ARG),
    (dict(rows=(1 << 24) + 1), E_ARG), (dict(n=0), E_ARG), (dict(n=24), E_SHAPE), (dict(n=(1 << 20) + 16), E_ARG),
    (dict(codes=None), E_ARG), (dict(codes=P + 4), E_ARG), (dict(scales=None), E_ARG), (dict(scales=P + 2), E_ARG)])
def test_quantize_refuses(change, code):
    a = dict(x=P, dtype=F32, rows=3, n=256, codes=P, scales=P, stream=None)
    a.update(change)
    assert q._lib.iqk_fp8_quantize(*a.values()) == code


def _w(experts=1, out=256, in_=512, codes=P, nbytes=None, scales=P, count=None):
    nb = experts * out * in_ if nbytes is None else nbytes
    ns = experts * (-(-out // 128)) * (-(-in_ // 128)) if count is None else count
    return q._Fp8Weights(experts, out, in_, codes, max(nb, 0), scales, max(ns, 0))


BAD_WEIGHTS = [(dict(experts=0), E_ARG), (dict(out=0), E_ARG), (dict(in_=0), E_ARG), (dict(in_=520), E_SHAPE),
               (dict(out=1 << 20, in_=1 << 12), E_ARG), (dict(codes=None), E_ARG), (dict(codes=P + 8), E_ARG),
               (dict(scales=None), E_ARG), (dict(nbytes=256 * 512 - 1), E_SIZE), (dict(count=7), E_SIZE)]


def _linear(w, **change):
    a = dict(x=P, dtype=BF16, xs=None, M=100, ws=P, nbytes=1 << 20, y=P, ydt=F32, stream=None)
    a.update(change)
    return q._lib.iqk_fp8_linear(ctypes.byref(w), *a.values())


@pytest.mark.parametrize("weights,code", BAD_WEIGHTS)
def test_linear_refuses_weights(weights, code):
    assert _linear(_w(**weights)) == code


@pytest.mark.parametrize("change,code", [
    (dict(x=None), E_ARG), (dict(x=P + 8), E_ARG), (dict(dtype=4), E_ARG), (dict(xs=P), E_ARG),
    (dict(dtype=E4M3), E_ARG), (dict(M=-1), E_ARG), (dict(ws=None), E_SIZE), (dict(nbytes=16), E_SIZE),
    (dict(ws=P + 8), E_ARG), (dict(y=None), E_ARG), (dict(ydt=E4M3), E_ARG), (dict(y=P + 2), E_ARG)])
def test_linear_refuses(change, code):
    assert _linear(_w(), **change) == code


def test_linear_of_a_long_depth_wants_its_sums():
    """Codes need no memory for codes, but that of the sums of the depth's parts."""
    w = _w(in_=1 << 14)
    assert _linear(w, dtype=E4M3, xs=P, ws=None, nbytes=0) == E_SIZE
    need = ctypes.c_size_t()
    assert q._lib.iqk_fp8_linear_workspace(ctypes.byref(w), 100, ctypes.byref(need)) == 0
    codes = 100 * (1 << 14) + 100 * 128 * 4
    assert need.value > codes and (need.value - codes) % (100 * 256 * 4) == 0
    assert _linear(w, nbytes=need.value - 1) == E_SIZE


def test_linear_takes_one_expert_and_no_rows():
    assert _linear(_w(experts=2)) == E_ARG
    assert _linear(_w(), M=0, x=None, y=None, ws=None, nbytes=0) == 0


@pytest.mark.parametrize("change,code", [
    (dict(x=None), E_ARG), (dict(ids=None), E_ARG), (dict(y=None), E_ARG), (dict(x_slots=2), E_ARG), (dict(k=0), E_ARG),
    (dict(T=-1), E_ARG), (dict(T=1 << 24), E_ARG), (dict(sorted=2), E_ARG), (dict(nbytes=64), E_SIZE),
    (dict(ws=None), E_SIZE), (dict(xs=P), E_ARG)])
def test_moe_refuses(change, code):
    a = dict(x=P, dtype=BF16, xs=None, x_slots=1, ids=P, T=300, k=4, sorted=0, ws=P, nbytes=1 << 20, y=P, ydt=F32,
             stream=None)
    a.update(change)
    w = _w(experts=8)
    assert q._lib.iqk_moe_fp8(ctypes.byref(w), *a.values()) == code


def test_binding_refuses_wrong_sizes():
    V = q.IqkValueError
    logits = FakeDev((3, 64), torch.float32)
    with pytest.raises(V):
        q.router_topk(logits, 4, scoring="relu", ids=FakeDev((3, 4), torch.int32), weights=FakeDev((3, 4), torch.float32))
    with pytest.raises(V):
        q.router_topk(logits, 4, bias=FakeDev((63,), torch.float32), ids=FakeDev((3, 4), torch.int32),
                      weights=FakeDev((3, 4), torch.float32))
    with pytest.raises(V):
        q.router_topk(logits, 4, ids=FakeDev((3, 3), torch.int32), weights=FakeDev((3, 4), torch.float32))
    with pytest.raises(V):
        q.router_topk(FakeDev((3, 64), torch.int32), 4)
    with pytest.raises(V):
        q.router_topk_grad(logits, FakeDev((2, 4), torch.int32), FakeDev((3, 4), torch.float32))
    with pytest.raises(V):
        q.fp8_quantize(FakeDev((3, 64), torch.float64))
    with pytest.raises(V):
        q.Fp8Weights(torch.zeros(2, 4, 16, dtype=torch.uint8), torch.zeros(2, 1, 1))
    with pytest.raises(V):
        q.Fp8Weights(torch.zeros(2, 4, 16, dtype=torch.float8_e4m3fn), torch.zeros(2, 1, 2))
    with pytest.raises(V):  # host weights
        q.fp8_linear(q.Fp8Weights(torch.zeros(1, 4, 16, dtype=torch.float8_e4m3fn), torch.zeros(1, 1, 1)),
                     FakeDev((2, 32), torch.bfloat16))
    with pytest.raises(V):  # a strided tensor
        q.fp8_quantize(torch.zeros(4, 64, dtype=torch.bfloat16)[:, ::2])
