"""Routing by scores with the plan, its gradient and the bias's step, against the fp64 oracle.

Bounds.  The choice and the plan: equal.  A weight: fp32 exponentials of differences of logits (the
argument's rounding, |x| 2^-24 for |x| < 16, and the function's 2 units), a sum of up to 1024 such
terms in a tree of 16 sequential and 6 pairwise steps, a quotient: below 2^-17 in the worst case.
The tests' logits lie within +-8 of each other's mean, and the bound taken is 2^-18 relative to the
weight.  The gradient: the oracle gives the sum of each element's terms' magnitudes, and each term is
a product of at most four such factors: 2^-16 of that sum."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
import oracle
from oracle import score_ref as S
from block_testlib import Guarded, assert_close, dev, workspace

pytestmark = pytest.mark.gpu
KINDS = {True: moe.MOE_SCORE_SIGMOID, False: moe.MOE_SCORE_SOFTMAX}
I32, F32 = torch.int32, torch.float32


def desc(T, E, k, sigmoid, renorm, scale=1.0, groups=1, keep=1, best=1):
    return moe.score_desc(T, E, k, KINDS[sigmoid], renorm, scale, groups, keep, best)


def buffers(T, E, k):
    return {"ids": Guarded((T, k), I32, fill=77), "w": Guarded((T, k), F32), "counts": Guarded((E,), I32, fill=77),
            "offsets": Guarded((E + 1,), I32, fill=77), "perm": Guarded((max(T * k, 1),), I32, fill=77),
            "inv_perm": Guarded((max(T * k, 1),), I32, fill=77)}


def run_route(sd, logits, bias, mask, ws=None, o=None):
    o = o or buffers(sd.T, sd.E, sd.k)
    ws = workspace(moe.moe_score_workspace_bytes(sd)) if ws is None else ws
    moe.moe_score_route(sd, logits, bias, mask, *[o[n].t for n in ("ids", "w", "counts", "offsets", "perm", "inv_perm")], ws)
    torch.cuda.synchronize()
    return {n: g.check().cpu().numpy() for n, g in o.items()}


def check_plan(got, ids, E):
    pl = oracle.plan(ids, E)
    assert np.array_equal(got["counts"], pl.counts) and np.array_equal(got["offsets"], pl.offsets)
    n = pl.perm.size
    assert np.array_equal(got["perm"][:n], pl.perm) and np.all(got["perm"][n:] == 77)   # behind the last: as it was
    assert np.array_equal(got["inv_perm"][:ids.size], pl.inv_perm)


def check_route(logits, k, sigmoid, renorm, scale=1.0, bias=None, mask=None, groups=1, keep=1, best=1):
    T, E = logits.shape
    sd = desc(T, E, k, sigmoid, renorm, scale, groups, keep, best)
    got = run_route(sd, dev(logits), None if bias is None else dev(bias), None if mask is None else dev(mask, torch.uint8))
    ids, w = S.route(logits, k, sigmoid, renorm, float(np.float32(scale)), bias, mask, groups, keep, best)
    assert np.array_equal(got["ids"], ids)
    assert_close("w", torch.from_numpy(got["w"]), w, np.abs(w) * 2.0 ** -18)
    check_plan(got, ids, E)
    return got


def draw(T, E, seed, spread=1.5):
    return np.clip(np.random.default_rng(seed).standard_normal((T, E)) * spread, -8, 8).astype(np.float32)


# (T, E, k, groups, keep, best): single experts, odd numbers, the borders of a lane's share, the largest
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 7, 7, 1, 1, 1), (5, 8, 2, 1, 1, 1), (4, 8, 3, 8, 3, 2), (33, 63, 9, 9, 4, 1),
          (17, 64, 6, 4, 2, 2), (64, 65, 5, 5, 2, 2), (9, 100, 11, 2, 1, 1), (130, 128, 8, 1, 1, 1), (66, 129, 3, 3, 2, 1),
          (65, 160, 6, 8, 3, 1), (257, 256, 8, 8, 4, 2), (31, 255, 16, 15, 7, 2), (40, 257, 17, 1, 1, 1), (21, 320, 10, 64, 20, 2),
          (70, 384, 8, 1, 1, 1), (12, 512, 64, 4, 3, 2), (6, 1000, 12, 50, 9, 2), (5, 1024, 64, 64, 64, 1), (1100, 32, 4, 4, 2, 2)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_route(shape, sigmoid):
    T, E, k, groups, keep, best = shape
    print(f"[case] route {shape} sigmoid={sigmoid}", flush=True)
    logits = draw(T, E, 11 + E)
    rng = np.random.default_rng(E)
    for bias, renorm, scale, masked in ((None, True, 1.0, False), ((rng.standard_normal(E) * 0.1).astype(np.float32), False, 2.5, True)):
        x, mask = logits.copy(), None
        if masked:
            mask = (rng.random(T) < 0.7).astype(np.uint8)
            x[mask == 0] = np.nan
            if T > 2:
                x[2] = np.inf if mask[2] == 0 else x[2]
        check_route(x, k, sigmoid, renorm, scale, bias, mask, groups, keep, best)


@pytest.mark.parametrize("E,groups", [(8, 1), (16, 4), (128, 8), (256, 8), (300, 6), (600, 1)])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_barred_experts(E, groups, sigmoid):
    """Logits of -inf, down to a token that has none left, and biases of -inf; slots without an expert."""
    rng = np.random.default_rng(E)
    T, k = 40, 6
    x = draw(T, E, 3)
    for t in range(T):
        x[t, rng.random(E) < t / (T - 2)] = -np.inf
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    bias[rng.integers(0, E)] = -np.inf
    keep = max(1, groups // 2)
    got = check_route(x, k, sigmoid, True, 1.0, bias, None, groups, keep, 2)
    assert (got["ids"][-1] == -1).all() and (got["w"][-1] == 0).all()
    check_route(x, k, sigmoid, False, 1.0, np.full(E, -np.inf, np.float32), None, groups, keep, 1)   # nothing for anyone
    lowest = x.copy()
    lowest[np.isinf(x)] = np.finfo(np.float32).min   # the type's lowest value is a logit like others: its score is 0
    check_route(lowest, k, sigmoid, True, 1.0, bias, None, groups, keep, 2)


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,best", [(8, 1, 1), (64, 4, 2), (128, 1, 1), (256, 8, 2), (512, 8, 1)])
def test_equal_and_neighbouring_values(E, groups, best, sigmoid):
    """Logits that are equal (the lower id goes first) or differ in their last bit, in all orders."""
    rng = np.random.default_rng(E)
    T, k = 50, 6
    x = rng.choice(np.array([-1.0, 0.25, 2.0], np.float32), (T, E))
    check_route(x, k, sigmoid, True, 1.0, None, None, groups, max(1, groups // 2), best)
    bias = rng.choice(np.array([0.0, 0.125], np.float32), E)
    check_route(x, k, sigmoid, True, 1.0, bias, None, groups, max(1, groups // 2), best)
    near = np.float32(0.75)
    steps = [near]
    for _ in range(5):
        steps.append(np.nextafter(steps[-1], np.float32(2)))
    x = rng.choice(np.array(steps, np.float32), (T, E))
    check_route(x, k, sigmoid, True, 1.0, None, None, groups, max(1, groups // 2), best)
    # a bias that puts unequal scores within a few 2^-26 of each other
    x = draw(T, E, 5, 1.0)
    x[:] = x[0]
    bias = (0.9 - S.scores(x[0], sigmoid)).astype(np.float32)
    check_route(x, k, sigmoid, True, 1.0, bias, None, groups, max(1, groups // 2), best)


@pytest.mark.parametrize("E,groups", [(16, 4), (128, 1), (256, 8), (700, 7)])
def test_bad_values(E, groups):
    """A NaN, or +inf in a softmax: no expert and NaN weights, for that token alone."""
    T, k = 12, 4
    x = draw(T, E, 9)
    x[1, 3] = np.nan
    x[4, E - 1] = np.inf
    x[6] = np.nan
    x[7, :] = -np.inf
    x[8, 2] = np.nan
    x[8, 3] = -np.inf
    for sigmoid in (True, False):
        got = check_route(x, k, sigmoid, True, 1.0, None, None, groups, max(1, groups // 2), 2)
        assert (got["ids"][1] == -1).all() and np.isnan(got["w"][1]).all()
        assert np.isnan(got["w"][4]).all() != sigmoid
        check_route(x, k, sigmoid, False, 1.0, np.zeros(E, np.float32), None, groups, max(1, groups // 2), 1)
    bias = np.zeros(E, np.float32)
    bias[E // 2] = np.nan
    got = check_route(x, k, True, True, 1.0, bias, None, groups, max(1, groups // 2), 2)
    assert (got["ids"] == -1).all() and (got["counts"] == 0).all()
    bias[E // 2] = np.inf   # an expert that every token takes
    got = check_route(draw(T, E, 9), k, True, False, 1.0, bias, None, groups, max(1, groups // 2), 2)
    assert (got["ids"][:, 0] == E // 2).all()


@pytest.mark.parametrize("E", [132, 160, 256])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 32, 33, 65])
def test_few_tokens(T, E):
    rng = np.random.default_rng(T + E)
    bias, mask = (rng.standard_normal(E) * 0.05).astype(np.float32), (rng.random(T) < 0.7).astype(np.uint8)
    for groups, keep, best in ((1, 1, 1), (2, 1, 2), (4, 3, 1), (4, 2, 2), (8, 4, 2), (16, 5, 2)):
        if E % groups:
            continue
        for k in (1, 8, 16):
            if k > E // groups * keep:
                continue
            for sigmoid in (True, False):
                x = draw(T, E, T + k)
                check_route(x, k, sigmoid, k > 1, 2.5, bias, mask, groups, keep, best)
                check_route(np.round(x * 2) / np.float32(2), k, sigmoid, k > 1, 1.0, None, None, groups, keep, best)


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_logits_whose_scores_are_equal_in_64_bits(sigmoid):
    """Logits that differ while their scores do not: tiny ones, and far ones whose scores underflow."""
    rng = np.random.default_rng(8)
    for E, k in ((32, 6), (128, 8), (256, 8), (512, 4)):
        x = (rng.standard_normal((40, E)) * 2.0 ** rng.integers(-126, -40, (40, E))).astype(np.float32)
        x[:, 5] = 3.0
        x[20:30, ::3] = rng.standard_normal((10, x[:, ::3].shape[1])).astype(np.float32) * np.float32(2.0 ** -30)
        x[30:, 7:] = -np.abs(rng.standard_normal((10, E - 7)).astype(np.float32)) * 100 - 900
        check_route(x, k, sigmoid, True)
        check_route(x, k, sigmoid, False, bias=np.zeros(E, np.float32))


def test_small_sigmoids_in_groups():
    """Scores far below one, with no bias, with a bias of their own size and with a larger one: what fp32 exponentials are off
    there is more than the scores' distances."""
    rng = np.random.default_rng(12)
    T, E = 400, 256
    for low in (-6, -12, -20, -45, -66):
        x = (low + rng.standard_normal((T, E)) * 1e-3).astype(np.float32)
        for bias in (None, rng.standard_normal(E).astype(np.float32) * np.float32(np.exp(low) * 1e-3),
                     rng.standard_normal(E).astype(np.float32) * np.float32(1e-5)):
            check_route(x, 8, True, True, bias=bias, groups=8, keep=4, best=2)
            check_route(x, 8, True, False, bias=bias)


def test_far_logits():
    """Scores that underflow or saturate in 32 bits, and in 64: weights stay quotients."""
    x = np.stack([np.linspace(-80, 80, 16), np.linspace(-120, -90, 16), np.linspace(30, 36, 16), np.linspace(-900, -800, 16),
                  np.full(16, -700.0), np.linspace(-3, 700, 16)]).astype(np.float32)
    for sigmoid in (True, False):
        sd = desc(6, 16, 4, sigmoid, True)
        got = run_route(sd, dev(x), None, None)
        for t in range(6):
            ids = got["ids"][t]
            ref = S.choose(x[t], 4, sigmoid)
            if not (sigmoid and t in (0, 2, 3, 5)):   # scores that saturate: which of them goes first is a matter of 64 bits' last
                assert list(ids) == ref, t
            # arguments up to 2^10 long: their rounding, 2^-14, is a relative error of the exponential
            assert_close("w", torch.from_numpy(got["w"][t]), S.weights(x[t], ids, sigmoid, True), 2.0 ** -12)


@pytest.mark.parametrize("T,E,k,groups", [(16384, 128, 8, 1), (21804, 256, 8, 8), (70001, 64, 2, 4), (3001, 1024, 16, 32)])
def test_many_tokens(T, E, k, groups):
    """Whole batches: the choice equal to the 64-bit one, computed on the GPU by torch."""
    torch.manual_seed(T)
    x = torch.randn(T, E, device="cuda")
    bias = torch.randn(E, device="cuda") * 0.02
    keep = max(1, groups // 2)
    for sigmoid in (True, False):
        got = run_route(desc(T, E, k, sigmoid, True, 1.0, groups, keep, 2), x, bias, None)
        s = torch.sigmoid(x.double()) if sigmoid else torch.softmax(x.double(), 1)
        c = s + bias.double()
        if groups > 1:
            best = torch.sort(c.view(T, groups, -1), 2, descending=True).values[:, :, :2].sum(2)
            stay = torch.zeros(T, groups, dtype=torch.bool, device="cuda")
            stay.scatter_(1, torch.sort(best, dim=1, descending=True, stable=True).indices[:, :keep], True)
            c = torch.where(stay[:, :, None], c.view(T, groups, -1), -torch.inf).view(T, E)
        ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
        assert np.array_equal(got["ids"], ids.cpu().numpy())
        w = s.gather(1, ids)
        w = (w / w.sum(1, keepdim=True)).cpu().numpy()
        assert_close("w", torch.from_numpy(got["w"]), w, w * 2.0 ** -18)
        check_plan(got, got["ids"], E)


def test_no_tokens():
    got = run_route(desc(0, 8, 2, True, True), torch.zeros(16, device="cuda"), None, None)
    assert (got["counts"] == 0).all() and (got["offsets"] == 0).all() and (got["perm"] == 77).all()
    x = torch.full((9, 8), float("nan"), device="cuda")
    got = run_route(desc(9, 8, 2, True, True), x, None, torch.zeros(9, dtype=torch.uint8, device="cuda"))
    assert (got["ids"] == -1).all() and (got["w"] == 0).all() and (got["offsets"] == 0).all() and (got["inv_perm"] == -1).all()


# -------------------------------------------------------------------------------- gradient
def run_backward(sd, logits, ids, d_w):
    d = Guarded((sd.T, sd.E), F32)
    moe.moe_score_backward(sd, logits, ids, d_w, d.t)
    torch.cuda.synchronize()
    return d.check()


@pytest.mark.parametrize("shape", [s[:3] for s in SHAPES], ids=str)
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
def test_backward(shape, sigmoid, renorm):
    T, E, k = shape
    rng = np.random.default_rng(T + E)
    x = draw(T, E, 21)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int64)
    ids[rng.random((T, k)) < 0.2] = -1
    ids[T // 2] = -1
    x[T // 2] = np.nan          # a token without a slot: not read
    g = rng.standard_normal((T, k)).astype(np.float32)
    g[ids < 0] = np.nan         # nor is the gradient of a slot without an expert
    got = run_backward(desc(T, E, k, sigmoid, renorm, 2.5), dev(x), dev(ids, I32), dev(g))
    ref, size = S.backward(x, ids, g, sigmoid, renorm, 2.5)
    assert_close("d_logits", got, ref, size * 2.0 ** -16 + 1e-37)


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
def test_backward_by_differences(sigmoid, renorm):
    """The gradient against differences of the forward call's own weights: a step of 2^-6 in a logit, whose
    cube's share is 2^-12 of third derivatives below 1, and twice the weights' 2^-18 over the step."""
    T, E, k = 6, 16, 4
    sd = desc(T, E, k, sigmoid, renorm)
    x = draw(T, E, 33)
    got = run_route(sd, dev(x), None, None)
    g = np.random.default_rng(4).standard_normal((T, k)).astype(np.float32)
    d = run_backward(sd, dev(x), dev(got["ids"], I32), dev(g)).cpu().numpy()
    h = 2.0 ** -6
    for e in range(E):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        v = []
        for y in (up, down):
            r = run_route(sd, dev(y), None, None)
            same = (np.sort(r["ids"], 1) == np.sort(got["ids"], 1)).all(1)
            order = np.argsort(r["ids"], 1)[np.arange(T)[:, None], np.argsort(np.argsort(got["ids"], 1), 1)]
            v.append(np.where(same, (np.take_along_axis(r["w"].astype(np.float64), order, 1) * g).sum(1), np.nan))
        diff = (v[0] - v[1]) / (2 * h)
        ok = ~np.isnan(diff)
        assert ok.any()
        bound = np.abs(g).sum(1) * (h * h + 2.0 ** -18 / h)
        assert (np.abs(diff - d[:, e])[ok] <= bound[ok]).all()


@pytest.mark.parametrize("sigmoid,renorm", [(True, True), (False, True), (False, False)])
def test_backward_of_tokens_without_a_slot(sigmoid, renorm):
    """Rows of zeros where no id is an expert's, with NaN and infinities for logits; their neighbours as ever."""
    for T in (7, 5000):
        x = draw(T, 40, 3)
        ids = np.tile(np.array([3, 39, 0], np.int32), (T, 1))
        clean = run_backward(desc(T, 40, 3, sigmoid, renorm), dev(x), dev(ids, I32), dev(np.ones((T, 3)))).cpu().numpy()
        gone = np.arange(0, T, 3)
        ids[gone] = -1
        x[gone] = np.array([np.nan, np.inf, -np.inf, 1], np.float32)[np.arange(40) % 4]
        got = run_backward(desc(T, 40, 3, sigmoid, renorm), dev(x), dev(ids, I32), dev(np.ones((T, 3)))).cpu().numpy()
        assert (got[gone] == 0).all()
        keep = np.setdiff1d(np.arange(T), gone)
        assert np.array_equal(got[keep], clean[keep])


def test_backward_of_ids_out_of_range_and_repeated():
    x, g = draw(3, 10, 1), np.ones((3, 3), np.float32)
    ids = np.array([[10, 5, -7], [1 << 30, -1, 12], [4, 4, 2]])
    got = run_backward(desc(3, 10, 3, True, False), dev(x), dev(ids, I32), dev(g)).cpu().numpy()
    ref, _ = S.backward(x, ids, g, True, False)
    assert np.allclose(got, ref, rtol=2.0 ** -16) and (got[1] == 0).all() and got[2, 4] != 0


# ------------------------------------------------------------------------------------ bias
@pytest.mark.parametrize("E", [1, 2, 63, 64, 65, 256, 1000, 1024])
def test_bias_update(E):
    rng = np.random.default_rng(E)
    for counts in (rng.integers(0, 50, E), np.full(E, 2 ** 31 - 1), np.arange(E)):
        bias = rng.standard_normal(E).astype(np.float32)
        b, c = dev(bias), dev(counts, I32)
        out = Guarded((E,), F32)
        moe.moe_bias_update(c, 1e-3, b, out.t)
        torch.cuda.synchronize()
        ref = S.bias_update(counts, float(np.float32(1e-3)), bias)
        assert_close("bias", out.check(), ref, np.abs(ref) * 2.0 ** -24)
        moe.moe_bias_update(c, 1e-3, b, b)
        assert torch.equal(b, out.t)


# --------------------------------------------------------------------- streams, graphs, repeats
def test_graph_replays_streams_and_repeats():
    """A captured route, bias step and gradient, replayed with eager work between the replays; the same on
    four streams at once with a workspace each; every one bit for bit the eager call's."""
    T, E, k = 1500, 256, 8
    sd = desc(T, E, k, True, True, 2.5, 8, 4, 2)
    x, bias = dev(draw(T, E, 2)), dev(np.random.default_rng(3).standard_normal(E).astype(np.float32) * 0.02)
    g = dev(np.random.default_rng(4).standard_normal((T, k)).astype(np.float32))
    names = ("ids", "w", "counts", "offsets", "perm", "inv_perm", "bias", "d")

    def new():
        i = lambda *s: torch.full(s, 5, dtype=I32, device="cuda")  # noqa: E731
        f = lambda *s: torch.full(s, 5.0, device="cuda")  # noqa: E731
        return [i(T, k), f(T, k), i(E), i(E + 1), i(T * k), i(T * k), f(E), f(T, E), workspace(moe.moe_score_workspace_bytes(sd))]

    def step(o):
        moe.moe_score_route(sd, x, bias, None, *o[:6], o[8])
        moe.moe_bias_update(o[2], 1e-3, bias, o[6])
        moe.moe_score_backward(sd, x, o[0], g, o[7])

    ref = new()
    step(ref)
    torch.cuda.synchronize()

    def same(o):
        torch.cuda.synchronize()
        for n, a, b in zip(names, ref, o):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
            b.zero_()

    o = new()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(o)
    torch.cuda.current_stream().wait_stream(side)
    same(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o)
    for _ in range(3):
        graph.replay()
        same(o)
        step(o)
        same(o)
    streams, outs = [torch.cuda.Stream() for _ in range(4)], [new() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, q in zip(streams, outs):
            with torch.cuda.stream(s):
                step(q)
    for q in outs:
        same(q)
