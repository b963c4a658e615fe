"""Routing by scores where fp32 cannot tell a value from an empty place.  Against the fp64 oracle; the bounds are those
of test_gpu_score."""
import numpy as np
import pytest
import torch

from oracle import score_ref as S
from block_testlib import assert_close, dev
from test_gpu_score import check_route, desc, draw, run_backward, run_route

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)


def test_a_group_whose_second_best_is_finite_and_far_down():
    """The group's value is the sum of both, below every ordinary group's, however good its best expert is."""
    x = np.zeros((3, 16), np.float32)
    x[:, 0] = 8
    for g in (1, 2, 3):
        x[:, 4 * g:4 * g + 4] = -g
    x[:, 13:] = 0
    x -= np.arange(16, dtype=np.float32) / 16   # no two alike: a tie is settled in 64 bits by itself
    for low in (LOWEST, -2e38, -9e37, -1e31):
        bias = np.zeros(16, np.float32)
        bias[1:4] = low
        for sigmoid in (True, False):
            got = check_route(x, 2, sigmoid, True, bias=bias, groups=4, keep=2, best=2)
            assert (got["ids"] >= 4).all()
            got = check_route(x, 2, sigmoid, True, bias=bias, groups=4, keep=2, best=1)
            assert (got["ids"][:, 0] == 0).all()


# four tokens a wave, one token a wave, and 64 bits throughout (17 experts of one token; three groups)
@pytest.mark.parametrize("E,k,groups", [(16, 2, 4), (16, 4, 1), (96, 6, 2), (256, 8, 8), (512, 8, 4), (96, 17, 4), (96, 6, 3)])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_biases_of_any_finite_size(E, k, groups, sigmoid):
    """Biases near the ends of the type, alone and among ordinary ones, -inf beside them."""
    rng = np.random.default_rng(E + k)
    far = np.array([LOWEST, -3e38, -2e38, -1.5e38, -9e37, -1e31, 1e30, 2e38, -LOWEST], np.float32)
    for T in (2, 37):
        x = draw(T, E, T + E)
        for share in (0.2, 0.6, 1.0):
            for these in (far[:1], far[:6], far):
                bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
                at = rng.random(E) < share
                bias[at] = rng.choice(these, int(at.sum()))
                bias[rng.integers(0, E)] = -np.inf
                for keep in {1, max(1, groups // 2), groups}:
                    if k <= keep * (E // groups):
                        for best in (1, 2):
                            check_route(x, k, sigmoid, True, bias=bias, groups=groups, keep=keep, best=best)


# ------------------------------------------------------------------------- weights of far logits
def far_logits(T, E, low, high, seed):
    """Logits over the whole range, with a full mantissa each."""
    return np.random.default_rng(seed).uniform(low, high, (T, E)).astype(np.float32)


# Bound, in u = 2^-24.  A chosen expert's exponential: 2 (the function) and 1 (its argument's rounding put back); a
# sigmoid's quotient 4 more; the sum of up to 16 of them 4 additions, or over all logits 22 and (3 |x - max| + 2) a
# term, which the terms' own size keeps below 3 log 1024 + 2; quotient 1, scale 1: 50 of 64 at most.  Below fp32's
# normal range a score has steps of 2^-149, which the scale multiplies.
@pytest.mark.parametrize("T,E,k,groups", [(4, 256, 8, 8), (500, 16, 8, 1), (500, 64, 6, 4), (300, 256, 16, 2), (40, 600, 9, 1), (60, 40, 20, 1)])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_weights_of_far_logits(T, E, k, groups, sigmoid):
    for low, high in ((-40, 40), (-85, 2), (-100, 0), (-150, 90), (-9, 9)):
        x = far_logits(T, E, low, high, E - low)
        bias = np.random.default_rng(E).uniform(0.1, 4, E).astype(np.float32)   # the choice does not go by the scores alone
        for b in (None, bias):
            for renorm in (True, False):
                sd = desc(T, E, k, sigmoid, renorm, 2.5, groups, max(1, groups // 2), 2)
                got = run_route(sd, dev(x), None if b is None else dev(b), None)
                for t in range(T):
                    ids = got["ids"][t]
                    w = S.weights(x[t], ids, sigmoid, renorm, 2.5)
                    assert_close(f"w[{t}]", torch.from_numpy(got["w"][t]), w, w * 2.0 ** -18 + 2.0 ** -147)


# ------------------------------------------------------------- gradient of confident tokens
def softmax_gradient(x, ids, g):
    """d_e = s_e sum_f s_f (G_e - G_f) over all experts f, G the sum of an expert's g: nothing cancels but what does in
    the gradient itself.  And s_e times the terms' magnitudes, those of chosen f without what cancels among them."""
    T, E = x.shape
    d, size, s_all = np.zeros((T, E)), np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s, G = S.scores(x[t], False), np.zeros(E)
        np.add.at(G, ids[t], g[t].astype(np.float64))
        among = np.zeros(E, bool)
        among[ids[t]] = True
        inner = (s[None, :] * (G[:, None] - G[None, :]) * among[None, :]).sum(1)   # over the chosen f
        outer = np.abs(G) * s[~among].sum()
        d[t], size[t], s_all[t] = s * (inner + G * s[~among].sum()), s * (np.abs(inner) + outer), s
    return d, size, s_all


def units(x):
    """The relative bound below, of each token."""
    far = np.where(np.isinf(x), 0, x.max(1, keepdims=True) - x).max(1, keepdims=True).astype(np.float64)
    return (12 + 2 * far) * 2.0 ** -24


@pytest.mark.parametrize("T,E,k", [(6, 64, 1), (40, 64, 1), (40, 64, 6), (30, 100, 20), (5000, 32, 2), (9, 1024, 16), (5, 1000, 17)])
def test_softmax_gradient_of_confident_tokens(T, E, k):
    """Tokens whose chosen experts have nearly all of the softmax, down to 2^-24 of it left over.

    Bound, in u = 2^-24, of the terms that the gradient is made of: the other experts' exponentials |x - max| (the
    argument's rounding) and 2 (the function), twice where their sum counts too, a quotient or product 2 each, one
    rounding at the end: below 12 + 2 |x - max|.  The subtraction in 64 bits adds 2^-48 of s_e times the gradients'
    magnitudes (k terms, each of a few 2^-53)."""
    rng = np.random.default_rng(E + k)
    for gap in (0, 4, 8, 12, 17):
        x = draw(T, E, E + gap, 1.0)
        ids = np.argsort(rng.random((T, E)), 1)[:, :k]
        np.put_along_axis(x, ids, np.take_along_axis(x, ids, 1) + np.float32(gap), 1)
        if E > 64:
            x[::3, ::5] = np.where(np.isin(np.arange(E)[::5], ids[0]), x[::3, ::5], -100 - gap)   # far ones among the others
        if k > 1:
            ids[1::4, 1] = ids[1::4, 0]     # the same expert twice
        for g in (np.ones((T, k), np.float32), rng.standard_normal((T, k)).astype(np.float32)):
            got = run_backward(desc(T, E, k, False, False), dev(x), dev(ids, torch.int32), dev(g)).cpu().numpy()
            ref, size, s = softmax_gradient(x, ids, g)
            bound = size * units(x) + s * np.abs(g).astype(np.float64).sum(1, keepdims=True) * 2.0 ** -48 + 2.0 ** -140
            assert_close(f"gap {gap}", torch.from_numpy(got), ref, bound)
            assert (np.abs(got.astype(np.float64).sum(1)) <= bound.sum(1)).all()   # a softmax's gradient sums to 0


def test_softmax_gradient_beside_barred_experts():
    x = draw(30, 40, 2)
    x[:, 7:30:3] = -np.inf
    ids = np.tile(np.array([3, 39, 0]), (30, 1))
    g = np.random.default_rng(1).standard_normal((30, 3)).astype(np.float32)
    for k in (3, 17):
        more = np.full((30, k), -1)
        more[:, :3] = ids
        gk = np.full((30, k), np.nan, np.float32)
        gk[:, :3] = g
        got = run_backward(desc(30, 40, k, False, False), dev(x), dev(more, torch.int32), dev(gk)).cpu().numpy()
        ref, size, s = softmax_gradient(x, ids, g)
        assert (got[:, 7:30:3] == 0).all()
        assert_close("d", torch.from_numpy(got), ref, size * units(x) + s * np.abs(g).sum(1, keepdims=True) * 2.0 ** -48)


# ------------------------------------------------------------------ places without an expert
@pytest.mark.parametrize("each", range(2, 17))
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_every_expert_of_one_group_in_sixteen(each, sigmoid):
    """As many choices as the group that stays has experts, some of them too close for fp32: nothing else may come between."""
    for T in (3, 400):
        x = draw(T, 16 * each, each)
        x[::2] = np.round(x[::2] * 4) / 4
        for k in {each, max(1, each - 1)}:
            got = check_route(x, k, sigmoid, True, groups=16, keep=1, best=2)
            assert (got["ids"] // each == got["ids"][:, :1] // each).all()
            check_route(x, k, sigmoid, False, bias=np.full(16 * each, 0.25, np.float32), groups=16, keep=1, best=1)


@pytest.mark.parametrize("groups,more", [(16, 9), (8, 3), (8, 11), (4, 1), (4, 7), (2, 1)])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_barred_experts_behind_the_last_choice(groups, more, sigmoid):
    """256 experts, sixteen a lane.  Of one group the last two of each sixteen can be chosen, but of one sixteen `more` others;
    its last two, barred by their logits, have the largest bias.  All that there are are chosen, and all but one."""
    rng = np.random.default_rng(groups + more)
    lanes = 16 // groups
    for at in range(lanes):
        x, bias = np.full((200, 256), -np.inf, np.float32), np.zeros(256, np.float32)
        can = [16 * lane + r for lane in range(lanes) for r in ((14, 15) if lane != at else range(more))]
        x[:, can] = (0.5 + rng.standard_normal((200, len(can))) / 512).astype(np.float32)   # too close for fp32, but unlike
        bias[[16 * at + 14, 16 * at + 15]] = 2
        for k in (len(can), len(can) - 1):
            got = check_route(x, k, sigmoid, True, bias=bias, groups=groups, keep=1, best=2)
            assert np.isin(got["ids"], can).all()
            check_route(x, k, sigmoid, True, groups=groups, keep=1, best=2)
