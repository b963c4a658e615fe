"""Routing by scores where fp32 cannot tell a value from an empty place.  Against the fp64 oracle; the bounds are those
of test_gpu_score."""
import numpy as np
import pytest
import torch

from oracle import score_ref as S
from block_testlib import assert_close, dev
from test_gpu_score import check_route, desc, draw, run_route

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
