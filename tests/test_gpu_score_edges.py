"""Routing by scores where fp32 cannot tell a value from an empty place.  Against the fp64 oracle; the bounds are those
of test_gpu_score."""
import numpy as np
import pytest

from test_gpu_score import check_route, draw

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
