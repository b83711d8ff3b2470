"""Quantization and 8-bit products on the GPU against the 64-bit oracle.

Tolerances.  Codes and scales: equal (the definition fixes every rounding).
Products, per output row in norm, against the product of the same codes and
scales: a float32 result sums at most 64 blocks here, each product of scales
and each addition rounded to 2^-24 of what is summed so far: 2e-6.  A 16-bit
result adds half a unit of its type (2^-8, 2^-11) and, where the sums run on
the 8-bit matrix instructions, at most 1.2e-4 of the sum of the products'
magnitudes per block (measured on operands over e4m3's whole range), whose
norm against the result's is below 8 for these inputs and whose signs differ
from block to block: 1.2e-4 * 2 is left for it."""
import numpy as np
import pytest
import torch

from gpu_common import announce
from oracle import layer

import dequant_iqk_moe_amd as q

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BAR = {"f32": 2e-6, "bf16": 2.0 ** -8 + 2.4e-4, "f16": 2.0 ** -11 + 2.4e-4}
INF = np.inf


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(dtype) if dtype is not None else t).cuda()


def _weights(rng, E, N, K):
    """Codes of a normal spread over e4m3's range, scales within a factor of four."""
    w = layer.to_e4m3(np.clip(rng.normal(size=(E, N, K)) * 100, -448, 448))
    s = (rng.uniform(0.5, 2, (E, -(-N // 128), -(-K // 128))) / 3000).astype(np.float32)
    return w, s


def _device_weights(w, s):
    return q.Fp8Weights(_dev(w).view(torch.float8_e4m3fn), _dev(s))


def _activations(rng, rows, K, dtype):
    """(tensor, its float32 values): unit spread, one loud channel in a hundred."""
    x = rng.normal(size=(rows, K)) * np.where(rng.random(K) < 0.01, 20, 1)
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    return t.cuda(), t.float().numpy()


def _off(y, ref):
    y = y.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(y).all()
    return np.linalg.norm(y - ref, axis=-1).max() if not ref.any() else (
        np.linalg.norm(y - ref, axis=-1) / np.linalg.norm(ref, axis=-1)).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (5, 1040), (64, 2048), (129, 4096)])
def test_quantize(M, K, dtype):
    announce(f"quantize M={M} K={K} {dtype}")
    t, x = _activations(np.random.default_rng(M + K), M, K, dtype)
    codes, scales = q.fp8_quantize(t)
    rc, rs = layer.quantize(x)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.view(torch.uint8).cpu().numpy(), rc)


def test_quantize_special_values():
    x = np.zeros((6, 256), np.float32)
    x[1, 3] = 1e-38                      # below the floor: no infinite reciprocal
    x[2, 200] = 3e38
    x[3, :128] = np.linspace(-448, 448, 128)   # scale 1: the codes' own grid
    x[4, 0] = np.nan
    x[4, 1] = 1.0
    x[5, 130] = INF
    codes, scales = q.fp8_quantize(_dev(x))
    codes, scales = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    rc, rs = layer.quantize(x[:4])
    np.testing.assert_array_equal(codes[:4], rc)
    np.testing.assert_array_equal(scales[:4], rs)
    assert (codes[0] == 0).all() and codes[1, 3] == 0
    assert codes[4, 0] & 0x7F == 0x7F and codes[4, 1] == 0x7E and (codes[4, 2:] == 0).all()
    assert codes[5, 130] & 0x7F == 0x7F and scales[5, 1] == INF and (codes[5, :128] == 0).all()


SHAPES = [(1, 16, 16), (1, 1, 16), (1, 4096, 4096), (2, 17, 144), (3, 5, 48), (7, 250, 1040), (15, 128, 2048),
          (16, 16, 128), (17, 130, 144), (31, 64, 400), (33, 257, 272), (64, 64, 2064), (65, 513, 512),
          (130, 300, 1040), (257, 129, 4096), (400, 384, 512), (513, 1000, 272)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K):
    announce(f"linear M={M} N={N} K={K}")
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    w, s = _weights(rng, 1, N, K)
    W = _device_weights(w, s)
    for xt, yt in (("bf16", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")):
        t, x = _activations(rng, M, K, xt)
        rc, rs = layer.quantize(x)
        ref = layer.linear(w[0], s[0], rc, rs)
        y = q.fp8_linear(W, t, out_dtype=DT[yt])
        assert y.dtype == DT[yt] and y.shape == (M, N)
        # a row of few outputs can be small against its terms: measured against at least the rows' mean
        norms = np.linalg.norm(ref, axis=-1)
        off = np.linalg.norm(y.double().cpu().numpy() - ref, axis=-1) / np.maximum(norms, norms.mean())
        assert off.max() <= BAR[yt], (xt, yt, off.max())
        # the same product from codes and scales: the same bits
        again = q.fp8_linear(W, *q.fp8_quantize(t), out_dtype=DT[yt])
        assert torch.equal(again, y)


@pytest.mark.parametrize("M,N,K", [(34, 66, 256), (200, 1000, 656), (1300, 2000, 272), (1290, 1990, 384), (4000, 2600, 272),
                                   (3990, 2570, 256)])
def test_linear_tiles(M, N, K):
    """Enough tiles for each tile size, in whole and in partial blocks of the depth."""
    announce(f"linear tiles M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K)
    w, s = _weights(rng, 1, N, K)
    W = _device_weights(w, s)
    t, x = _activations(rng, M, K, "bf16")
    rc, rs = layer.quantize(x)
    ref = layer.linear(w[0], s[0], rc, rs)
    for yt in ("f32", "bf16", "f16"):
        assert _off(q.fp8_linear(W, t, out_dtype=DT[yt]), ref) <= BAR[yt], yt


def test_linear_is_the_transposed_products_gradient():
    """sum(y * dy) differentiated by x is the product of dy with the
    transposed codes and scales (square blocks transpose): checked against
    differences of the dequantized product."""
    rng = np.random.default_rng(3)
    M, N, K = 4, 256, 384
    w, s = _weights(rng, 1, N, K)
    back = _device_weights(w.transpose(0, 2, 1), s.transpose(0, 2, 1))
    t, dy = _activations(rng, M, N, "f32")
    dx = q.fp8_linear(back, t).double().cpu().numpy()
    rc, rs = layer.quantize(dy)
    dq = layer.e4m3_values()[rc] * np.repeat(rs, 128, 1).astype(np.float64)
    wide = layer.e4m3_values()[w[0]] * np.repeat(np.repeat(s[0].astype(np.float64), 128, 0), 128, 1)
    x = rng.normal(size=(M, K))
    for m, i in ((0, 0), (1, 200), (3, 383)):
        up, down = x.copy(), x.copy()
        up[m, i] += 0.5
        down[m, i] -= 0.5
        diff = ((up @ wide.T - down @ wide.T) * dq).sum()
        assert abs(dx[m, i] - diff) <= 2e-6 * np.linalg.norm(dx[m])


def test_linear_special_values():
    rng = np.random.default_rng(4)
    for M in (2, 40, 300):
        N, K = 200, 400
        w, s = _weights(rng, 1, N, K)
        w[0, 7, 300] = 0x7F                   # a NaN weight: its output column only
        t, x = _activations(rng, M, K, "f32")
        t[0, 390] = float("nan")              # (in the partial last block)
        t[1, :] = 0.0
        if M > 2:
            t[5, 17] = float("inf")
        for yt in ("f32", "bf16"):
            y = q.fp8_linear(_device_weights(w, s), t, out_dtype=DT[yt]).float().cpu().numpy()
            assert np.isnan(y[0]).all()
            bad = np.zeros((M, N), bool)
            bad[:, 7] = True
            bad[0] = True
            if M > 2:
                assert not np.isfinite(y[5]).any()
                bad[5] = True
            assert np.isnan(y[:, 7]).all()
            assert np.isfinite(y[~bad]).all()
            assert (y[1][~bad[1]] == 0).all()


def test_linear_leaves_its_surroundings():
    """Nothing past the end of y is written, in either alignment of its rows."""
    rng = np.random.default_rng(5)
    for M, N in ((3, 33), (40, 128), (300, 260), (129, 131)):
        w, s = _weights(rng, 1, N, 256)
        t, _ = _activations(rng, M, 256, "bf16")
        for yt in ("f32", "bf16"):
            buf = torch.full((M * N + 64,), 7.0, dtype=DT[yt], device="cuda")
            q.fp8_linear(_device_weights(w, s), t, y=buf[1:1 + M * N].view(M, N))
            ref = q.fp8_linear(_device_weights(w, s), t, out_dtype=DT[yt])
            assert torch.equal(buf[1:1 + M * N].view(M, N), ref)
            assert (buf[0] == 7) and (buf[1 + M * N:] == 7).all()


def test_linear_rows_past_32_bit_offsets():
    announce("linear, 8.6 GB of results")
    M, N, K = (1 << 22) + 5, 512, 16
    rng = np.random.default_rng(6)
    w, s = _weights(rng, 1, N, K)
    x = torch.randn(M, K, device="cuda", dtype=torch.float32)
    y = q.fp8_linear(_device_weights(w, s), x)
    for rows in (slice(0, 40), slice(M - 40, M), slice((1 << 21) - 20, (1 << 21) + 20)):
        rc, rs = layer.quantize(x[rows].cpu().numpy())
        assert _off(y[rows], layer.linear(w[0], s[0], rc, rs)) <= BAR["f32"]


def _moe_ref(w, s, x, ids, slots):
    T, k = ids.shape
    rc, rs = layer.quantize(x)
    ref = np.full((T * k, w.shape[1]), np.nan)
    flat = ids.reshape(-1)
    for e in range(w.shape[0]):
        pairs = np.nonzero(flat == e)[0]
        if pairs.size:
            rows = pairs // k if slots == 1 else pairs
            ref[pairs] = layer.linear(w[e], s[e], rc[rows], rs[rows])
    return ref.reshape(T, k, -1)


def _moe_check(w, s, ids, slots, xt, yt, rng, **kw):
    T, k = ids.shape
    t, x = _activations(rng, T * slots, w.shape[2], xt)
    y = q.moe_fp8(_device_weights(w, s), t, _dev(ids), x_slots=slots, out_dtype=DT[yt], **kw)
    assert y.shape == (T, k, w.shape[1]) and y.dtype == DT[yt]
    ref = _moe_ref(w, s, x, ids, slots)
    got = y.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got).all(-1), np.isnan(ref).all(-1))
    ok = ~np.isnan(ref).any(-1)
    if ok.any():
        norms = np.linalg.norm(ref[ok], axis=-1)
        off = np.linalg.norm(got[ok] - ref[ok], axis=-1) / np.maximum(norms, norms.mean())
        assert off.max() <= BAR[yt], (xt, yt, off.max())
    # codes with their scales: the same bits
    codes, scales = q.fp8_quantize(t)
    again = q.moe_fp8(_device_weights(w, s), codes, _dev(ids), x_slots=slots, x_scales=scales, out_dtype=DT[yt], **kw)
    same = again == y
    assert bool((same | (torch.isnan(again) & torch.isnan(y))).all())


@pytest.mark.parametrize("T,k,E,N,K", [(1, 6, 16, 256, 512), (1, 1, 1, 16, 16), (2, 3, 8, 33, 144), (5, 2, 4, 130, 272),
                                       (16, 8, 64, 64, 128), (40, 6, 256, 48, 256), (70, 4, 8, 200, 400),
                                       (300, 2, 3, 257, 272), (513, 3, 4, 384, 528)])
def test_moe(T, k, E, N, K):
    announce(f"moe T={T} k={k} E={E} N={N} K={K}")
    rng = np.random.default_rng(T + E + N)
    w, s = _weights(rng, E, N, K)
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).astype(np.int32)
    for slots, xt, yt in ((1, "bf16", "f32"), (k, "f32", "bf16"), (1, "f16", "f16")):
        _moe_check(w, s, ids, slots, xt, yt, rng)


@pytest.mark.parametrize("T,k,E,N,K", [(128, 4, 64, 512, 528),      # about 8 rows per expert
                                       (160, 2, 16, 512, 512),      # 20
                                       (180, 2, 8, 300, 656),       # 45
                                       (400, 2, 8, 520, 384),       # 100
                                       (2048, 2, 8, 2570, 272),     # 512
                                       (2050, 2, 8, 2560, 256),
                                       (600, 4, 1100, 256, 256),    # more experts than one workgroup counts
                                       (5000, 2, 5, 130, 144)])     # more pairs than one workgroup places
def test_moe_grouped(T, k, E, N, K):
    """Each size of group, and of the grouping before it."""
    announce(f"moe grouped T={T} k={k} E={E} N={N} K={K}")
    rng = np.random.default_rng(T + E + N)
    w, s = _weights(rng, E, N, K)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    ids[1, 0], ids[T - 1, 1] = E, -5
    for slots, xt, yt in ((1, "bf16", "f32"), (k, "f32", "bf16"), (1, "f16", "f16")):
        _moe_check(w, s, ids, slots, xt, yt, rng)


@pytest.mark.parametrize("counts", [[16, 17, 0, 1, 15, 33, 32, 64], [0, 0, 500, 0, 0, 0, 0, 1], [63, 65, 48, 49, 31, 47, 50, 40],
                                    [255, 257, 1, 128, 129, 0, 300, 127], [700, 200, 192, 256, 64, 320, 449, 512]])
def test_moe_group_sizes(counts):
    """Groups at and around the edges of the tiles; some empty."""
    announce(f"moe group sizes {counts}")
    rng = np.random.default_rng(sum(counts))
    E, N, K = len(counts), 2580 if sum(counts) > 2000 else 530, 272
    w, s = _weights(rng, E, N, K)
    ids = rng.permutation(np.repeat(np.arange(E), counts)).astype(np.int32)[:, None]
    for yt in ("f32", "bf16"):
        _moe_check(w, s, ids, 1, "bf16", yt, rng)


@pytest.mark.parametrize("T", [1, 9, 200])
def test_moe_ids(T):
    """Invalid, repeated, one-sided and sorted ids."""
    announce(f"moe ids T={T}")
    rng = np.random.default_rng(T)
    E, k, N, K = 6, 4, 472, 1040
    w, s = _weights(rng, E, N, K)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    for yt in ("f32", "bf16"):
        _moe_check(w, s, np.sort(ids.reshape(-1)).reshape(T, k), 1, "bf16", yt, rng, sorted=True)
        _moe_check(w, s, np.full((T, k), 4, np.int32), k, "bf16", yt, rng)        # all at one expert
        bad = ids.copy()
        bad[0, 0], bad[T // 2, 1], bad[T - 1, 3] = -1, E, 2 ** 31 - 1
        _moe_check(w, s, bad, 1, "bf16", yt, rng)
        _moe_check(w, s, np.full((T, k), -1, np.int32), 1, "bf16", yt, rng)       # nothing valid


def test_moe_weights_past_32_bit_offsets():
    announce("moe, 5 GB of weights")
    E, N, K, T, k = 300, 4096, 4096, 40, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 127, (E, N, K), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(E, N // 128, K // 128, generator=g, device="cuda")
    W = q.Fp8Weights(codes.view(torch.float8_e4m3fn), scales)
    x = torch.randn(T, K, generator=g, device="cuda")
    rc, rs = layer.quantize(x.cpu().numpy())
    for ids in (torch.tensor([[299, 298]] * T), torch.tensor([[299, 0]])):
        T1 = ids.shape[0]
        y = q.moe_fp8(W, x[:T1], ids.to(torch.int32).cuda())
        for j in range(2):
            e = int(ids[0, j])
            ref = layer.linear(codes[e].cpu().numpy()[:64], scales[e].cpu().numpy(), rc[:T1], rs[:T1])
            assert _off(y[:, j, :64], ref) <= BAR["f32"]


def test_same_result_every_time_and_on_another_stream():
    rng = np.random.default_rng(9)
    E, k, N, K, T = 8, 2, 256, 512, 100
    w, s = _weights(rng, E, N, K)
    W = _device_weights(w, s)
    t, _ = _activations(rng, T, K, "bf16")
    ids = _dev(rng.integers(0, E, (T, k)).astype(np.int32))
    first = q.moe_fp8(W, t, ids)
    ws = torch.empty(q.moe_fp8_workspace_bytes(W, T, k), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                        # whatever the workspace holds
    y = torch.empty_like(first)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    q.moe_fp8(W, t, ids, workspace=ws, y=y, stream=st)
    st.synchronize()
    assert torch.equal(first, y)


def test_new_results_belong_to_the_calls_stream():
    """Results and workspaces made by a call on another stream come from that
    stream's memory: freed, they are not given to the current stream's next
    tensors while the call still runs."""
    rng = np.random.default_rng(12)
    E, k, N, K, T = 8, 2, 512, 1024, 300
    W = _device_weights(*_weights(rng, E, N, K))
    S = _device_weights(*_weights(rng, 1, N, K))
    t, _ = _activations(rng, T, K, "bf16")
    logits = torch.randn(T, E, device="cuda")
    ids, wt = q.router_topk(logits, k)
    want = (q.moe_fp8(W, t, ids), q.fp8_linear(S, t), *q.fp8_quantize(t), wt)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        for _ in range(20):
            i2, w2 = q.router_topk(logits, k, stream=stream)
            got = (q.moe_fp8(W, t, i2, stream=stream), q.fp8_linear(S, t, stream=stream), *q.fp8_quantize(t, stream=stream), w2)
            junk = [torch.full((T * N,), float("nan"), device="cuda") for _ in range(3)]
            del junk
        st.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.float(), b.float())


def test_graph_replays():
    """A captured layer step (selection, routed and dense product) replayed on
    new inputs, with eager work in between."""
    announce("graph of router_topk + moe_fp8 + fp8_linear")
    rng = np.random.default_rng(10)
    E, k, N, K, T = 16, 3, 128, 256, 4
    W = _device_weights(*_weights(rng, E, N, K))
    S = _device_weights(*_weights(rng, 1, N, K))
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(T, E, device="cuda")

    def step():
        ids, wt = q.router_topk(logits, k)
        return q.combine(q.moe_fp8(W, x, ids), wt), q.fp8_linear(S, x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.from_numpy(rng.normal(size=(T, K)).astype(np.float32)))
        logits.copy_(torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)))
        graph.replay()
        got = [o.clone() for o in out]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_no_rows():
    W = q.Fp8Weights(torch.zeros(1, 32, 64, device="cuda").to(torch.float8_e4m3fn), torch.ones(1, 1, 1, device="cuda"))
    assert q.fp8_linear(W, torch.empty(0, 64, device="cuda")).shape == (0, 32)
    assert q.moe_fp8(W, torch.empty(0, 64, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 2, 32)
    codes, scales = q.fp8_quantize(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0, 1)


def test_quantize_more_blocks_than_one_grid_row():
    announce("quantize, 69 GB of values")
    M, K = 1 << 24, 2064  # 2^24 rows of 17 blocks: 2^32 threads and more at 16 a block
    if torch.cuda.mem_get_info()[0] < 120e9:
        pytest.skip("needs 106 GB")
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, M // 2, M - 1], device="cuda")
    some = torch.randn(4, K, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    x[rows] = some
    codes, scales = q.fp8_quantize(x)
    few, few_scales = q.fp8_quantize(some)
    assert torch.equal(codes[rows], few) and torch.equal(scales[rows], few_scales)
    assert torch.equal(codes[M - 1000:M - 1], torch.zeros_like(codes[M - 1000:M - 1]))
    del x, codes, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 272), (70, 528), (300, 400), (1100, 528)])
def test_a_rows_bits_do_not_depend_on_its_place(T, K, yt):
    """Rows in another order, and the same rows again, give the same bits."""
    rng = np.random.default_rng(T + K)
    k, E, N = 3, 4, 384
    w, s = _weights(rng, E, N, K)
    W, one = _device_weights(w, s), _device_weights(w[:1], s[:1])
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().to(torch.bfloat16)
    ids = _dev(rng.integers(0, E, (T, k)).astype(np.int32))
    y, d = q.moe_fp8(W, x, ids, out_dtype=DT[yt]), q.fp8_linear(one, x, out_dtype=DT[yt])
    for _ in range(8):
        order = torch.from_numpy(rng.permutation(T)).cuda()
        again = q.moe_fp8(W, x[order].contiguous(), ids[order].contiguous(), out_dtype=DT[yt])
        assert torch.equal(again, y[order]), (T, K, yt)
        again = q.fp8_linear(one, x[order].contiguous(), out_dtype=DT[yt])
        assert torch.equal(again, d[order]), (T, K, yt)


@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(3, 300, 272), (20, 300, 272), (40, 1000, 272), (300, 5000, 400), (4096, 8192, 256)])
def test_a_weight_scale_reaches_its_rows_only(M, N, K, yt):
    """A NaN and an infinite weight scale in the depth's last block, at the first weight rows."""
    rng = np.random.default_rng(M)
    w, s = _weights(rng, 1, N, K)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda().to(torch.bfloat16)
    clean = q.fp8_linear(_device_weights(w, s), x, out_dtype=DT[yt])
    for value in (np.nan, np.inf):
        bad = s.copy()
        bad[0, 0, -1] = value
        y = q.fp8_linear(_device_weights(w, bad), x, out_dtype=DT[yt])
        assert torch.equal(y[:, 128:], clean[:, 128:])
        assert not torch.isfinite(y[:, :128]).any()


@pytest.mark.parametrize("M,N,K", [(33, 16, 4096), (40, 33, 2832), (60, 173, 7552), (141, 261, 7920), (700, 1052, 3696),
                                   (64, 64, 1 << 16), (1030, 70, 2064)])
def test_linear_of_a_long_depth(M, N, K):
    """Few tiles of a long depth: sums of its parts, joined."""
    rng = np.random.default_rng(M + N + K)
    w, s = _weights(rng, 1, N, K)
    W = _device_weights(w, s)
    for xt, yt in (("bf16", "f32"), ("f32", "bf16"), ("bf16", "f16")):
        t, x = _activations(rng, M, K, xt)
        rc, rs = layer.quantize(x)
        buf = torch.full((M * N + 64,), 7.0, dtype=DT[yt], device="cuda")
        y = q.fp8_linear(W, t, y=buf[1:1 + M * N].view(M, N))
        assert _off(y, layer.linear(w[0], s[0], rc, rs)) <= BAR[yt], (xt, yt)
        assert (buf[0] == 7) and (buf[1 + M * N:] == 7).all()
        ws = torch.full((q.fp8_linear_workspace_bytes(W, M),), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(q.fp8_linear(W, t, out_dtype=DT[yt], workspace=ws), y)
        codes, scales = q.fp8_quantize(t)
        assert torch.equal(q.fp8_linear(W, codes, scales, out_dtype=DT[yt]), y)
        t[M // 2, K - 1] = float("nan")
        bad = torch.isnan(q.fp8_linear(W, t, out_dtype=DT[yt]))
        assert bad[M // 2].all() and int(bad.sum()) == N


@pytest.mark.parametrize("T,k,E,N,K", [(32, 2, 8, 5000, 272), (80, 2, 8, 5000, 144), (160, 2, 8, 5000, 272),
                                       (400, 2, 8, 5000, 272), (800, 2, 8, 1000, 528), (1200, 2, 8, 5000, 144)])
def test_moe_tile_sizes(T, k, E, N, K):
    """Enough workgroups that the tile follows the rows per expert: 16, 32, 64, 128 (both widths) and 256."""
    rng = np.random.default_rng(T + N)
    w, s = _weights(rng, E, N, K)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[0, 0], ids[-1, -1] = -1, E
    for xt, yt in (("bf16", "f32"), ("f32", "bf16"), ("bf16", "f16")):
        _moe_check(w, s, ids, 1, xt, yt, rng)
