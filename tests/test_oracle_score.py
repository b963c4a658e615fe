"""Pins of the oracle's routing by scores and blockwise 8-bit pieces: brute force, closed forms, central
differences and the layer's own oracle (CPU only)."""
import itertools

import numpy as np
import pytest
import torch

import oracle
from oracle import score_ref as S


def rows(T, E, seed, scale=1.0):
    return (np.random.default_rng(seed).standard_normal((T, E)) * scale).astype(np.float32)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_scores_agree_with_torch_in_64_bits(sigmoid):
    x = rows(20, 33, 1, 6.0)
    t = torch.from_numpy(x).double()
    ref = torch.sigmoid(t) if sigmoid else torch.softmax(t, 1)
    got = np.stack([S.scores(r, sigmoid) for r in x])
    assert np.allclose(got, ref.numpy(), rtol=1e-14, atol=0)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_without_bias_and_groups_the_choice_is_the_layers_own(sigmoid):
    x = rows(50, 16, 2)
    ids, w = S.route(x, 5, sigmoid, True)
    ref_ids, ref_w = oracle.route(x, 5)
    assert np.array_equal(ids, ref_ids)
    if not sigmoid:   # softmax over all, renormalised over the chosen: softmax over the chosen
        assert np.allclose(w, ref_w, rtol=1e-6)


def test_choice_is_the_best_of_all_subsets():
    """With one group the k best c have the largest sum of c of all k-subsets; with groups the same holds
    among the subsets of the experts of the best pairs of groups."""
    rng = np.random.default_rng(3)
    for _ in range(30):
        x, b = rng.standard_normal(8).astype(np.float32), rng.standard_normal(8) * 0.2
        c = S.scores(x, True) + b
        best = max(itertools.combinations(range(8), 3), key=lambda z: c[list(z)].sum())
        assert set(best) == set(S.choose(x, 3, True, b))
        pairs = max(itertools.combinations(range(4), 2), key=lambda z: sum(c[2 * g:2 * g + 2].sum() for g in z))
        inside = [e for g in pairs for e in (2 * g, 2 * g + 1)]
        best = max(itertools.combinations(inside, 3), key=lambda z: c[list(z)].sum())
        assert set(best) == set(S.choose(x, 3, True, b, 4, 2, 2))


def test_ties_bars_and_bad_values():
    x = np.zeros(8, np.float32)
    assert S.choose(x, 4, True) == [0, 1, 2, 3]
    assert S.choose(x, 4, True, groups=4, group_topk=2, group_best=2) == [0, 1, 2, 3]
    x[0] = -np.inf   # the first group has one expert left: half the others' value
    assert S.choose(x, 4, True, groups=4, group_topk=2, group_best=2) == [2, 3, 4, 5]
    assert S.choose(x, 4, True, groups=4, group_topk=2, group_best=1) == [1, 2, 3]
    bias = np.zeros(8)
    bias[1] = -np.inf
    assert S.choose(x, 4, True, bias, groups=4, group_topk=4) == [2, 3, 4, 5]
    assert S.choose(np.full(8, -np.inf, np.float32), 4, False) == []
    x[3] = np.nan
    assert S.choose(x, 4, True) is None and S.choose(x, 4, False) is None
    x[3] = np.inf
    assert S.choose(x, 1, True) == [3] and S.choose(x, 1, False) is None
    ids, w = S.route(np.stack([x, np.ones_like(x)]), 2, True, True, mask=[0, 1])
    assert (ids[0] == -1).all() and (w[0] == 0).all()


def test_weights_far_from_zero():
    """Every chosen score underflows in 64 bits; their quotients do not."""
    x = np.array([-2000.0, -2000.0 + np.log(3.0), 5.0])
    assert np.allclose(S.weights(x, [1, 0], True, True), [0.75, 0.25], rtol=1e-12)
    assert np.allclose(S.weights(x, [1, 0], False, True, 2.0), [1.5, 0.5], rtol=1e-12)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_by_differences(sigmoid, renormalise):
    x = rows(3, 7, 5).astype(np.float64)
    ids = np.array([[4, 1, 2], [0, -1, 6], [-1, -1, -1]])
    g = np.random.default_rng(6).standard_normal((3, 3))
    d, _ = S.backward(x, ids, g, sigmoid, renormalise, 1.7)

    def value(x):
        total = 0.0
        for t in range(3):
            at = [j for j in range(3) if ids[t, j] >= 0]
            total += (S.weights(x[t], ids[t, at], sigmoid, renormalise, 1.7) * g[t, at]).sum()
        return total

    for t in range(3):
        for e in range(7):
            h = np.zeros_like(x)
            h[t, e] = 1e-6
            assert abs((value(x + h) - value(x - h)) / 2e-6 - d[t, e]) < 1e-8


def test_gradient_of_the_renormalised_softmax_is_the_layers_own():
    x = rows(10, 9, 7)
    ids, w = S.route(x, 4, False, True)
    g = np.random.default_rng(8).standard_normal((10, 4))
    ref = oracle.d_logits_from_dw(w, g, ids, 9)
    assert np.allclose(S.backward(x, ids, g, False, True)[0], ref, atol=1e-12)


def test_bias_update():
    assert np.allclose(S.bias_update([4, 0, 2, 2], 0.5, [1, 1, 1, 1]), [0.5, 1.5, 1, 1])
    big = [2 ** 31 - 1] * 4
    assert np.allclose(S.bias_update(big, 0.5, np.zeros(4)), 0)


def test_quantize_forms():
    rng = np.random.default_rng(9)
    x = rng.standard_normal((200, 144)).astype(np.float32) * np.exp2(rng.integers(-6, 6, (200, 1))).astype(np.float32)
    codes, scales = S.quantize(x, "rows")
    assert codes.shape == (200, 144) and scales.shape == (200, 2)
    v = S.values(codes, scales)
    m = np.abs(x[:, :128]).max(1)
    assert np.allclose(np.abs(v[:, :128]).max(1), m, rtol=1e-6)          # the largest value is the last code
    # half a step of a normal code (2^-4), or of a subnormal one (2^-10 of the scale), and a rounding
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(scales, 128, 1)[:, :144] * 2.0 ** -10) * 1.0001).all()
    t, ts = S.quantize(x, "tokens")
    assert t.shape == (144, 208) and ts.shape == (144, 2) and (t[:, 200:] == 0).all()
    r, rs = S.quantize(np.ascontiguousarray(np.pad(x, ((0, 8), (0, 0))).T), "rows")
    assert np.array_equal(t, r) and np.array_equal(ts, rs)
    q, qs = S.quantize(x, "tiles")
    assert qs.shape == (2, 2) and qs[1, 1] == np.abs(x[128:, 128:]).max() / np.float32(448)
    zero, ones = S.quantize(np.zeros((2, 16), np.float32), "rows")
    assert (zero == 0).all() and (ones == 1).all()
    tiny, ts = S.quantize(np.full((1, 16), 1e-40, np.float32), "rows")
    assert ts[0, 0] == np.float32(2.0 ** -126) and np.allclose(S.values(tiny, ts), 1e-40, atol=2.0 ** -136)


def test_values_agree_with_the_layers_decoders():
    rng = np.random.default_rng(10)
    codes = rng.integers(0, 0x7F, (256, 256)).astype(np.uint8)
    s, b = rng.random((256, 2)).astype(np.float32), rng.random((2, 2)).astype(np.float32)
    assert np.array_equal(S.values(codes, s), oracle.dequant_rows_1x128(codes, s))
    assert np.array_equal(S.values(codes, b), oracle.dequant_blocks_128x128(codes, b))
