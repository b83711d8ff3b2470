"""Pins of the 64-bit oracle of expert selection and the 8-bit products (CPU)."""
import numpy as np
import pytest
import torch

from oracle import layer

INF = np.inf


def test_softmax_choice_by_hand():
    l = np.log(np.array([[1.0, 4.0, 2.0, 4.0, 5.0]]))
    ids, w = layer.router(l, 3, "softmax")
    assert ids.tolist() == [[4, 1, 3]]  # the two equal scores by index
    np.testing.assert_allclose(w, [[5 / 13, 4 / 13, 4 / 13]])
    _, w = layer.router(l, 3, "softmax", renorm=False, scale=2.0)
    np.testing.assert_allclose(w, [[10 / 16, 8 / 16, 8 / 16]])


def test_bias_moves_the_choice_and_not_the_weights():
    l = np.zeros((1, 4))
    ids, w = layer.router(l, 2, "sigmoid", bias=np.array([0.0, 0.3, 0.1, -1.0]), renorm=False)
    assert ids.tolist() == [[1, 2]]
    np.testing.assert_allclose(w, [[0.5, 0.5]])


def test_groups_by_hand():
    # worth by the best two: 1.1, 1.0, 1.2; by the best one: 0.9, 0.5, 0.6
    c = np.array([0.9, 0.2, 0.5, 0.5, 0.6, 0.6])
    l = np.log(c / (1 - c))[None]
    assert layer.router(l, 2, "sigmoid", n_group=3, topk_group=1, group_top=2)[0].tolist() == [[4, 5]]
    assert layer.router(l, 2, "sigmoid", n_group=3, topk_group=1, group_top=1)[0].tolist() == [[0, 1]]


def test_masks():
    l = np.array([[-INF, 1.0, -INF, -INF], [-INF] * 4, [0.0, np.nan, 0.0, 0.0], [0.0, INF, 0.0, 0.0]])
    ids, w = layer.router(l, 2, "softmax")
    assert ids.tolist() == [[1, 1], [-1, -1], [-1, -1], [-1, -1]]
    assert w[0].tolist() == [1.0, 0.0] and w[1].tolist() == [0.0, 0.0]
    assert np.isnan(w[2]).all() and np.isnan(w[3]).all()
    assert layer.router(l, 1, "sigmoid")[0][3].tolist() == [1]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(scoring, renorm):
    rng = np.random.default_rng(5)
    T, E, k, scale = 4, 9, 3, 2.5
    l = rng.normal(size=(T, E))
    dw = rng.normal(size=(T, k))
    ids, _ = layer.router(l, k, scoring, renorm=renorm, scale=scale)

    def weights(l):
        w = np.stack([layer.scores(l[t], scoring)[ids[t]] for t in range(T)])
        return scale * (w / w.sum(1, keepdims=True) if renorm else w)

    got = layer.router_grad(l, ids, dw, scoring, renorm, scale)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            diff = ((weights(up) - weights(down)) * dw).sum() / (2 * h)
            assert abs(got[t, e] - diff) < 1e-8  # truncation h^2, rounding 1e-16 / h


def test_e4m3_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(layer.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(6)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 7, 4000),
                        # every tie between neighbours
                        (layer.e4m3_values()[:126] + layer.e4m3_values()[1:127]) / 2]).astype(np.float32)
    x = np.concatenate([x, -x])
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(layer.to_e4m3(x), ref)


def test_quantize_restores_within_half_a_step():
    rng = np.random.default_rng(7)
    x = rng.normal(size=(5, 272)).astype(np.float32)
    x[2, 128:256] = 0.0
    q, s = layer.quantize(x)
    v = layer.e4m3_values()[q] * np.repeat(s, 128, 1)[:, :272]
    # half of 2^-3 of the value, or of the smallest step (2^-9 of a scale)
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(s, 128, 1)[:, :272] * 2.0 ** -10) * 1.001).all()
    assert (q[2, 128:256] == 0).all()


def test_linear_against_widened_matrices():
    rng = np.random.default_rng(8)
    M, N, K = 3, 130, 272
    w = rng.integers(0, 256, (N, K)).astype(np.uint8)
    w[(w & 0x7F) == 0x7F] = 0
    sw = rng.uniform(0.5, 2, (2, 3)).astype(np.float32)
    q, s = layer.quantize(rng.normal(size=(M, K)))
    wide = layer.e4m3_values()[w] * np.repeat(np.repeat(sw, 128, 0), 128, 1)[:N, :K].astype(np.float64)
    x = layer.e4m3_values()[q] * np.repeat(s, 128, 1)[:, :K].astype(np.float64)
    np.testing.assert_allclose(layer.linear(w, sw, q, s), x @ wide.T, rtol=1e-12, atol=1e-9)
