"""The 8-bit products take the kernels that the GPU tests are written for (host only)."""
import ctypes

import pytest
import torch

import dequant_iqk_moe_amd as q
from fp8_paths import DENSE, GROUPED, MANY_EXPERTS


@pytest.mark.parametrize("size,wide,bf16", DENSE)
def test_dense(size, wide, bf16):
    M, N, K = size
    assert q.fp8_path(1, N, K, M) == wide
    assert q.fp8_path(1, N, K, M, out_dtype=torch.float16) == wide
    assert q.fp8_path(1, N, K, M, out_dtype=torch.bfloat16) == bf16


@pytest.mark.parametrize("counts,N,wide,bf16", GROUPED)
@pytest.mark.parametrize("K", [272, 256])
def test_grouped(counts, N, wide, bf16, K):
    E, P = len(counts), sum(counts)
    assert q.fp8_path(E, N, K, P, 1) == wide
    assert q.fp8_path(E, N, K, P, 1, torch.float16) == wide
    assert q.fp8_path(E, N, K, P, 1, torch.bfloat16) == bf16


def test_every_kernel_has_a_case():
    assert {p[1] for _, *paths in DENSE for p in paths if p[0] == "tiles"} == {64, 128, 256}
    assert {p[1:3] for *_, a, b in GROUPED for p in (a, b)} == {
        (16, 128), (32, 128), (64, 128), (128, 128), (128, 256), (256, 256)}
    for kind in ("few", "rows", "tiles"):
        assert {size[2] % 128 == 0 for size, a, _ in DENSE if a[0] == kind} == {True, False}


@pytest.mark.parametrize("E,T,k,N,K", MANY_EXPERTS)
def test_many_experts_are_grouped(E, T, k, N, K):
    assert q.fp8_path(E, N, K, T, k)[0] == "tiles"


def test_few_pairs():
    assert q.fp8_path(256, 4096, 4096, 1, 6) == ("few",)


def test_refusals():
    w = q._Fp8Weights(2, 128, 256)
    path = (ctypes.c_int32 * 4)()
    call = lambda T, k, dt, p=path: q._lib.iqk_fp8_path(ctypes.byref(w), T, k, dt, p)
    assert call(4, 2, 0) == 0
    for bad in ((0, 2, 0), (4, -1, 0), (1 << 24, 2, 0), (4, 2, 3), (4, 0, 0), (4, 2, 0, None)):
        assert call(*bad) == -1
    with pytest.raises(q.IqkValueError):
        q.fp8_path(2, 128, 256, 4, 2, torch.int8)
