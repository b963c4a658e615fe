"""The balance loss's gradient where the logits are far from zero.

A softmax does not change when a constant is added to a row, so the gradient's p may not lose bits as
|lse| grows: lse in fp32 is off by half a unit of its own size (2^-11 at 8192, 2^-8 at 65536; above
2^27 the logarithm of E is lost whole), and exp(logit - lse) with it.

Bounds: p is a row's exponentials over their sum.  An exponent's argument is at most 32 from the
row's largest (smaller terms vanish beside the absolute slack below) and carries 2.5 of it times
2^-24; with exp2's 2 units a term is within 82 2^-24 of itself, the sum of up to 64 a lane and 4 steps
between lanes too, and 68 more: p is within 240 2^-24 < 2^-16.  Each of the gradient's terms is then
within 2^-15; d_in and the final rounding within 2^-23 of the terms' sizes."""
import numpy as np
import pytest

from oracle import block_ref as R
from block_testlib import assert_close, f64
from test_gpu_balance import make, run

SHIFTS = (0.0, 40.0, -300.0, 4096.0, -8192.0, 65536.0, -131072.0, 2e6, -1e9, 1e9, 1e30, -1e30)
LOWEST = np.finfo(np.float32).min


def far(T, E, k, seed, **more):
    c = make(T, E, k, seed, **more)
    shift = np.array(SHIFTS, np.float32)[np.arange(T) % len(SHIFTS)]
    c["logits"] = (c["logits"] + shift[:, None]).astype(np.float32)
    c["logits"][5] = LOWEST                 # every expert masked by the type's lowest value
    c["logits"][6] = np.finfo(np.float32).max
    c["logits"][7] = LOWEST
    c["logits"][7, E // 2] = 3.0            # all but one
    c["w"] = np.array([0.3, 0.0], np.float32)   # the squares of such lse leave fp32
    return c


def test_oracle_probabilities_sum_to_one():
    c = far(30, 12, 2, 1)
    b = R.balance(c["logits"], c["ids"])
    assert np.abs(b["p"].sum(1) - 1).max() < 1e-12
    assert np.abs(b["p"][5] - 1 / 12).max() < 1e-15


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1, 8, 60, 64, 65, 128, 200, 256, 385, 512, 1000, 1024])
@pytest.mark.parametrize("T,S", [(60, 1), (700, 4)])
def test_gradient_keeps_its_bits(T, S, E):
    print(f"[case] balance far logits T={T} S={S} E={E}", flush=True)
    c = far(T, E, min(4, E), 80 + E, S=S)
    o = run(c)
    b = R.balance(c["logits"], c["ids"], c["mask"], c["offsets"])
    d, size = R.balance_grad(b, c["k"], c["w"].astype(np.float64), c["d_in"])
    assert np.array_equal(f64(o["counts"]), b["counts"])
    top = np.abs(c["logits"].astype(np.float64)).max(1)
    assert_close("lse", o["lse"], b["lse"], 2.0 ** -16 * (1 + top))
    assert_close("losses", o["losses"][:1], b["losses"][:1], 2.0 ** -15 * b["losses"][0])
    assert_close("d_logits", o["d_logits"], d, 2.0 ** -15 * (size - np.abs(c["d_in"])) + 2.0 ** -23 * (size + np.abs(d)))


@pytest.mark.gpu
def test_a_constant_added_to_a_row_changes_nothing():
    """Logits on a grid that survives the shift: the gradient without the z-loss is the unshifted one's,
    each within the bound of the same terms."""
    print("[case] balance shifted rows", flush=True)
    T, E, k = 200, 96, 4
    c = make(T, E, k, 5, add=False)
    c["logits"] = np.round(c["logits"] * 16) / 16
    c["w"] = np.array([1.0, 0.0], np.float32)
    near = f64(run(c)["d_logits"])
    b = R.balance(c["logits"], c["ids"])
    _, size = R.balance_grad(b, k, (1.0, 0.0))
    for shift in (4096.0, -65536.0, 2.0 ** 19):
        moved = dict(c, logits=(c["logits"] + np.float32(shift)).astype(np.float32))
        assert_close(f"shift {shift}", run(moved)["d_logits"], near, 2.0 ** -14 * size)
