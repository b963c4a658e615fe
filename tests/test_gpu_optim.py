"""Gradient norm and AdamW over lists of tensors, fp32 and 8-bit states, against the fp64 oracle.

Bounds.  m and v are sums of two products: four and five roundings, within 2^-21 of their terms'
sizes.  The update rate m / (root inv + eps) has eight more and the bias factors' rounding to fp32:
within 2^-19 of itself where m has not cancelled, and m's own error over the denominator else; the
weight's own products and sum add 2^-22 of its size.  An 8-bit code is one of the two e4m3 values
around the exact one; where it was exactly known in fp32 (betas of 0) the code is known too.  A mean
of N roundings with the remainder's probability is within 5 / sqrt(4 N) steps of 0."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from oracle import block_ref as R
from block_testlib import GUARD, HALF, assert_close, dev, f64, workspace

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U8 = torch.uint8


class Param:
    """One parameter with guards around everything the step writes."""

    def __init__(self, n, rng, p=F32, g=F32, master=False, eight=False, decay=0.0, fresh=False, gscale=1e-2):
        self.n, self.pt, self.eight, self.decay = n, p, eight, decay
        blocks = (n + 255) // 256
        w = rng.standard_normal(n).astype(np.float32) * 0.1
        self.whole, self.t = {}, {}

        def put(name, values, dtype):
            k = values.shape[0]
            whole = torch.zeros(k + 2 * GUARD, dtype=dtype, device="cuda")
            raw = whole.view(U8) if dtype in (F8, U8) else whole
            raw.fill_(9)
            whole[GUARD:GUARD + k] = torch.from_numpy(values).to("cuda").to(dtype)
            self.whole[name], self.t[name] = (raw, whole[GUARD:GUARD + k])

        put("p", w, p)
        self.g = dev(rng.standard_normal(n).astype(np.float32) * gscale, g)
        if master:
            put("master", w, F32)
        m = np.zeros(n, np.float32) if fresh else (rng.standard_normal(n) * 1e-2).astype(np.float32)
        r = np.zeros(n, np.float32) if fresh else (np.abs(rng.standard_normal(n)) * 1e-2 + 1e-4).astype(np.float32)
        if eight:
            for name, x in (("m", m), ("v", r)):
                pad = np.concatenate([x, np.zeros(blocks * 256 - n, np.float32)]).reshape(blocks, 256)
                s = (np.abs(pad).max(1) / 448).astype(np.float32) if not fresh else np.zeros(blocks, np.float32)
                put(name, x / np.repeat(np.maximum(s, 1e-30), 256)[:n], F8)
                put(name + "_scale", s, F32)
        else:
            put("m", m, F32)
            put("v", r * r, F32)
        self.row = moe.adamw_tensor(self.g, weight_decay=decay, **self.t)
        self.before = self.values()

    def codes(self, name):
        return self.t[name].view(U8).cpu().numpy()

    def values(self):
        o = {n: f64(t) for n, t in self.t.items() if n in ("p", "master")}
        if self.eight:
            o["m"] = R.decode_state(self.codes("m"), f64(self.t["m_scale"]))
            o["v"] = R.decode_state(self.codes("v"), f64(self.t["v_scale"])) ** 2
        else:
            o["m"], o["v"] = f64(self.t["m"]), f64(self.t["v"])
        return o

    def guards(self):
        for name, raw in self.whole.items():
            ends = torch.cat([raw[:GUARD], raw[-GUARD:]])
            assert torch.all(ends == 9), f"{name}: written outside"


def step(params, lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, t=3, seed=1, stochastic=False, scale=None, **more):
    hp = moe.adamw_hyper(lr, b1, b2, eps, t, seed, stochastic, d_grad_scale=scale, **more)
    moe.moe_adamw_step(hp, moe.adamw_tensors([p.row for p in params]))
    torch.cuda.synchronize()


def check(p, lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, t=3, scale=1.0, stochastic=False):
    b, a, g = p.before, p.values(), f64(p.g) * scale
    w0 = b.get("master", b["p"])
    w, m, v = R.adamw(w0, f64(p.g), b["m"], b["v"], lr, b1, b2, eps, t, p.decay, scale)
    em = 2.0 ** -21 * (np.abs(b1 * b["m"]) + np.abs((1 - b1) * g))
    ev = 2.0 ** -21 * v
    den = np.sqrt(v / (1 - b2 ** t)) + eps
    upd = lr / (1 - b1 ** t) / den
    ew = 2.0 ** -22 * (np.abs(w0) + np.abs(w)) + upd * em + 2.0 ** -19 * upd * np.abs(m)
    if "master" in a:
        assert_close("master", p.t["master"], w, ew)
        assert torch.equal(p.t["p"], p.t["master"].to(BF16)), "p is not its master's rounding"
    elif p.pt == BF16 and stochastic:
        # one of the two bf16 values around w: less than a whole step (two halves) away
        assert_close("p", p.t["p"], w, ew + 2 * HALF[BF16] * (np.abs(w) + ew))
    else:
        assert_close("p", p.t["p"], w, ew + HALF[p.pt] * (np.abs(w) + ew))
    if not p.eight:
        assert_close("m", p.t["m"], m, em)
        assert_close("v", p.t["v"], v, ev)
        return
    for name, x, ex in (("m", m, em), ("v", np.sqrt(v), 2.0 ** -21 * np.sqrt(v))):
        blocks = (p.n + 255) // 256
        pad = lambda q: np.concatenate([q, np.zeros(blocks * 256 - p.n)]).reshape(blocks, 256)  # noqa: E731
        top = pad(np.abs(x)).max(1)
        scale_ref = np.where(top > 0, np.maximum(top / 448, 2.0 ** -126), 1.0)
        s = f64(p.t[name + "_scale"])
        assert_close(name + "_scale", p.t[name + "_scale"], scale_ref, pad(ex).max(1) / 448 + 2.0 ** -23 * scale_ref)
        y = np.abs(x) / np.repeat(s, 256)[:p.n]
        got = np.abs(R.decode_state(p.codes(name), np.ones(blocks)))
        slack = 2.0 ** -20 * y + ex / np.repeat(s, 256)[:p.n]
        low, _ = R.e4m3_below(np.maximum(y - slack, 0))
        high, up = R.e4m3_below(y + slack)
        floor = np.where((name == "v") & (y > 0), 2.0 ** -9, 0.0)   # a root above 0 stays above 0
        assert np.all((got >= np.maximum(low, 0)) & (got <= np.maximum(high + up, floor))), f"{name}: not a neighbouring code"
        assert np.all(got >= floor) and np.all(got <= 448)
        sign = R.decode_state(p.codes(name), np.ones(blocks))
        assert np.all((sign * x >= 0) | (np.abs(x) <= ex))


SIZES = [1, 3, 4, 255, 256, 257, 1023, 4096, 4097, 70001]
TYPES = {
    "f32": dict(), "bf16g": dict(g=BF16), "bf16_master": dict(p=BF16, g=BF16, master=True),
    "bf16_master_f32g": dict(p=BF16, master=True), "bf16": dict(p=BF16, g=BF16),
    "f32_8bit": dict(eight=True), "bf16_master_8bit": dict(p=BF16, g=BF16, master=True, eight=True),
    "bf16_8bit": dict(p=BF16, g=BF16, eight=True),
}


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_step_parity(kind, stochastic):
    print(f"[case] adamw {kind} stochastic={stochastic}", flush=True)
    rng = np.random.default_rng(21)
    params = [Param(n, rng, decay=0.1 * (i % 2), **TYPES[kind]) for i, n in enumerate(SIZES)]
    scale = dev(np.array([0.5], np.float32))
    step(params, stochastic=stochastic, scale=scale)
    for p in params:
        p.guards()
        check(p, scale=0.5, stochastic=stochastic)


@pytest.mark.parametrize("kind", ["f32", "bf16_8bit"])
def test_first_step_from_zero_states(kind):
    print(f"[case] adamw first step {kind}", flush=True)
    rng = np.random.default_rng(22)
    params = [Param(n, rng, fresh=True, **TYPES[kind]) for n in (5, 256, 3001)]
    params[1].g[:] = 0        # no gradient yet either: nothing moves but the decay
    step(params, t=1)
    for p in params:
        p.guards()
        check(p, t=1)
    assert not params[1].values()["m"].any() and not params[1].values()["v"].any()


def test_many_tensors_in_one_list():
    """More tensors than a launch's arguments hold, empty ones among them, types mixed."""
    print("[case] adamw list of 150", flush=True)
    rng = np.random.default_rng(23)
    kinds = list(TYPES.values())
    params = [Param(0 if i % 11 == 3 else int(rng.integers(1, 9000)), rng, **kinds[i % len(kinds)]) for i in range(150)]
    step(params)
    for p in params:
        p.guards()
        if p.n:
            check(p)


@pytest.mark.parametrize("n", [1, 54, 55, 64, 65, 129])
@pytest.mark.parametrize("eight", [False, True])
def test_lists_around_a_launch(n, eight):
    """As many tensors as a launch holds and one more, without and with 8-bit states; the last one empty."""
    print(f"[case] adamw list of {n}, 8-bit {eight}", flush=True)
    rng = np.random.default_rng(40 + n)
    kinds = [k for k in TYPES.values() if not k.get("eight")]
    params = [Param(int(rng.integers(1, 1200)), rng, **kinds[i % len(kinds)]) for i in range(n)]
    if eight:
        params[n // 2] = Param(700, rng, eight=True)
    params.append(Param(0, rng))
    step(params)
    for p in params[:-1]:
        p.guards()
        check(p)


def test_repeated_steps_are_bitwise_reproducible():
    print("[case] adamw repeat", flush=True)
    out = []
    for _ in range(2):
        rng = np.random.default_rng(24)
        params = [Param(n, rng, **TYPES[k]) for n in (777, 12345) for k in ("bf16_8bit", "bf16_master")]
        for t in (1, 2, 3):
            step(params, t=t, stochastic=True)
        out.append([t.view(U8).clone() for p in params for t in p.t.values()])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_codes_where_the_arithmetic_is_exact():
    """betas of 0: m = g and sqrt(v) = |g| to the last bit, so scale, remainder, random bits and code follow
    from integers and single fp32 operations."""
    print("[case] adamw exact codes", flush=True)
    rng = np.random.default_rng(25)
    n = 5000
    p = Param(n, rng, eight=True)
    g = (2.0 ** rng.uniform(-22, 0, n) * rng.choice([-1, 1], n)).astype(np.float32)
    g[100:110] = 0
    p.g.copy_(torch.from_numpy(g))
    step([p], b1=0.0, b2=0.0, t=5, seed=77)
    u, _ = R.noise(77, 5, 0, n)
    pad = np.concatenate([np.abs(g), np.zeros(-n % 256, np.float32)]).reshape(-1, 256)
    s = (pad.max(1) * np.float32(1.0 / 448)).astype(np.float32)
    inv = (np.float32(1) / s).astype(np.float32)
    y = np.minimum(np.abs(g) * np.repeat(inv, 256)[:n], np.float32(448)).astype(np.float32)
    low = y < np.float32(2.0 ** -6)
    bits = np.where(low, y + np.float32(2.0 ** -6), y).astype(np.float32).view(np.uint32).astype(np.int64)
    for name, r in (("m", u & 0xFFFF), ("v", u >> 16)):
        code = ((bits + (r.astype(np.int64) << 4)) >> 20) - np.where(low, 968, 960)
        if name == "v":
            code = np.where((code == 0) & (y > 0), 1, code)
        else:
            code |= (g < 0).astype(np.int64) << 7
        assert np.array_equal(p.codes(name), code.astype(np.uint8)), name
        assert np.array_equal(p.t[name + "_scale"].cpu().numpy(), s), name


def test_stochastic_rounding_has_the_right_mean():
    """Over many values the remainder's probability shows: codes (normal and subnormal) and bf16 weights."""
    print("[case] adamw rounding mean", flush=True)
    rng = np.random.default_rng(26)
    n = 1 << 20
    p = Param(n, rng, eight=True)
    g = rng.uniform(0.0, 1.0, n).astype(np.float32) * 2.0 ** rng.integers(-16, 0, n).astype(np.float32)
    g[::256] = 1.0
    p.g.copy_(torch.from_numpy(g))
    step([p], b1=0.0, b2=0.0, seed=3)
    for name in ("m", "v"):
        y = g.astype(np.float64) * 448
        got = R.decode_state(p.codes(name), np.ones(n // 256))
        _, st = R.e4m3_below(y)
        use = (st > 0) & ((name == "m") | (y > 2.0 ** -9))
        err = (got - y)[use] / st[use]
        assert np.all(np.abs(err) < 1 + 2.0 ** -16)
        assert abs(err.mean()) < 5 / np.sqrt(4 * use.sum()) + 2.0 ** -16
        low = use & (y < 2.0 ** -6)
        assert abs(((got - y)[low] * 512).mean()) < 5 / np.sqrt(4 * low.sum()) + 2.0 ** -12
    # bf16 weights: no gradient, a decay that takes 2^-9 of each weight off: two bits below bf16's last
    q = Param(n, rng, p=BF16, fresh=True, decay=1.0)
    q.g.zero_()
    step([q], lr=2.0 ** -9, stochastic=True, seed=4)
    w = q.before["p"] * (1 - 2.0 ** -9)
    st = 2.0 ** (np.floor(np.log2(np.abs(w))) - 7)
    err = (f64(q.t["p"]) - w) / st
    assert np.all(np.abs(err) < 1) and abs(err.mean()) < 5 / np.sqrt(4 * n)
    assert abs((err * np.sign(w)).mean()) < 5 / np.sqrt(4 * n) + 2.0 ** -16


def test_eight_bit_average_moves_where_nearest_would_stick():
    """sqrt(v) halves its distance to |g| as its average should: steps of 2.5 % stay below half an e4m3 step."""
    print("[case] adamw moving average", flush=True)
    n, steps, b2 = 1 << 16, 40, 0.95
    rng = np.random.default_rng(27)
    p = Param(n, rng, eight=True, fresh=True)
    p.g.fill_(1.0)
    p.g[::256] = 4.0                      # keeps each block's scale
    r0 = np.full(n, 2.0)
    r0[::256] = 4.0
    p.t["v_scale"].fill_(4.0 / 448)
    p.t["v"].copy_(torch.from_numpy((r0 / 4 * 448).astype(np.float32)).to("cuda").to(F8))
    for t in range(1, steps + 1):
        step([p], b1=0.0, b2=b2, t=t, seed=t)
    v = p.values()["v"].reshape(-1, 256)[:, 1:]
    want = 1 + (4 - 1) * b2 ** steps
    # the root is rounded without bias, its square gains the rounding's variance: at most (step/2)^2 = (1/16)^2
    # of v a step (steps of 1/8 of the root's binade), over 1 / (1 - b2) steps' memory 20 / 256 of v
    assert abs(v.mean() - want) < want * (20 / 256 + 0.01)


def test_a_step_to_skip_changes_nothing():
    print("[case] adamw skipped", flush=True)
    rng = np.random.default_rng(28)
    for bad in (float("nan"), float("inf"), -float("inf")):
        params = [Param(3001, rng, **TYPES[k]) for k in ("f32", "bf16_8bit", "bf16_master")]
        before = [t.view(U8).clone() for p in params for t in p.t.values()]
        step(params, scale=dev(np.array([bad], np.float32)), stochastic=True)
        for a, t in zip(before, [t for p in params for t in p.t.values()]):
            assert torch.equal(a, t.view(U8))


def test_step_and_rate_on_the_device():
    print("[case] adamw device step", flush=True)
    for t in (1, 2, 7, 1000, 123457):
        rng = np.random.default_rng(29)
        params = [Param(4097, rng, **TYPES[k]) for k in ("f32", "bf16_master_8bit", "bf16")]
        step(params, lr=0.0, t=0, d_lr=dev(np.array([1e-2], np.float32)),
             d_step=torch.tensor([t], dtype=torch.int64, device="cuda"))
        for p in params:
            p.guards()
            check(p, lr=float(np.float32(1e-2)), t=t)
    p = Param(300, rng)                  # betas of 0 have no bias
    step([p], b1=0.0, b2=0.0, t=0, d_step=torch.tensor([9], dtype=torch.int64, device="cuda"))
    check(p, b1=0.0, b2=0.0, t=9)


def test_extreme_gradients():
    """Tiny gradients whose squares vanish in fp32, zeros, and large ones: no NaN."""
    print("[case] adamw extremes", flush=True)
    rng = np.random.default_rng(30)
    for kind in ("f32", "f32_8bit"):
        p = Param(1024, rng, fresh=True, **TYPES[kind])
        p.g[:256] = 1e-30
        p.g[256:512] = 0
        p.g[512:768] = 1e15
        p.g[768:] = 1e-38
        step([p], t=1)
        for t in p.t.values():
            assert torch.isfinite(t.float()).all()
        assert torch.isfinite(p.t["p"]).all()


@pytest.mark.parametrize("g", [F32, BF16])
@pytest.mark.parametrize("sizes", [[1], [4, 255, 256, 0, 4097], [70001, 3], [1000] * 400, [9_000_001, 5]])
def test_grad_norm_parity(sizes, g):
    """Sums in 64 bits: the norm's own rounding to fp32, and the scale's."""
    print(f"[case] grad_norm {len(sizes)} {g}", flush=True)
    rng = np.random.default_rng(31)
    gs = [dev(rng.standard_normal(n).astype(np.float32), g) for n in sizes]
    tl = moe.adamw_tensors([moe.adamw_tensor(t) for t in gs])
    nb = moe.moe_grad_norm_workspace_bytes(tl)
    ref, _ = R.grad_norm([f64(t) for t in gs], 1.0)
    for max_norm in (0.25 * ref, 4.0 * ref):
        max_norm = float(np.float32(max_norm))
        out = torch.full((2 + 2 * GUARD,), 9.0, device="cuda")
        ws = workspace(nb + 256)
        moe.moe_grad_norm(tl, max_norm, out[GUARD:GUARD + 1], out[GUARD + 1:GUARD + 2], ws, nb)
        torch.cuda.synchronize()
        assert torch.all(out[:GUARD] == 9) and torch.all(out[-GUARD:] == 9) and torch.all(ws[nb:] == 0xA5)
        scale = min(1.0, max_norm / (ref + 1e-6))
        assert_close("norm", out[GUARD:GUARD + 1], [ref], 2.0 ** -23 * ref)
        assert_close("scale", out[GUARD + 1:GUARD + 2], [scale], 2.0 ** -23 * scale)


def test_not_a_number_stays_one():
    """A NaN of any payload in a gradient or a parameter gives a NaN: the random bits that round a bf16
    parameter do not carry over its exponent and sign."""
    print("[case] adamw NaN", flush=True)
    rng = np.random.default_rng(33)
    for eight in (False, True):
        p = Param(300, rng, p=BF16, g=F32, eight=eight)     # a whole run and a tail
        at = torch.tensor([0, 5, 130, 255, 256, 299], device="cuda")
        p.g.view(torch.int32)[at] = torch.tensor([0x7FFFFFFF, -1, 0x7F800001, 0x7FC00000, 0x7FFFFFFF, -1],
                                                 dtype=torch.int32, device="cuda")
        p.t["p"].view(torch.int16)[[9, 290]] = torch.tensor([0x7FFF, -1], dtype=torch.int16, device="cuda")
        for seed in range(8):
            step([p], seed=seed, stochastic=True)
            nan = torch.isnan(p.t["p"])
            assert nan[at].all() and nan[[9, 290]].all() and (eight or int(nan.sum()) == 8)
        p.guards()


def test_grad_norm_far_sizes_and_bad_values():
    """Squares beyond fp32's range both ways are fine in 64 bits; a NaN, an infinity and a norm beyond
    fp32 give a scale that skips the step."""
    print("[case] grad_norm far", flush=True)

    def norm(values, g=F32):
        t = dev(np.array(values, np.float32), g)
        tl = moe.adamw_tensors([moe.adamw_tensor(t)])
        o = torch.empty(2, device="cuda")
        moe.moe_grad_norm(tl, 1.0, o[:1], o[1:], workspace(moe.moe_grad_norm_workspace_bytes(tl)))
        return f64(o)

    a = norm([3e-30, 4e-30])
    assert abs(a[0] - 5e-30) < 2e-36 and a[1] == 1.0
    a = norm([3e30, 4e30])
    assert abs(a[0] / 5e30 - 1) < 1e-6 and abs(a[1] * 5e30 - 1) < 1e-6
    a = norm([0.0, 0.0])
    assert a[0] == 0 and a[1] == 1.0
    a = norm([3e38, 3e38])
    assert np.isinf(a[0]) and np.isnan(a[1])
    a = norm([1.0, float("inf")])
    assert np.isinf(a[0]) and np.isnan(a[1])
    a = norm([1.0, float("nan")], BF16)
    assert np.isnan(a[0]) and np.isnan(a[1])
    o = torch.full((1,), 5.0, device="cuda")
    moe.moe_grad_norm(moe.adamw_tensors([]), 1.0, o, None, workspace(256))
    assert float(o) == 0.0
