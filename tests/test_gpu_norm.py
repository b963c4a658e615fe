"""Norms before and after a block, with gate and residual, forward and backward, against the fp64 oracle.

Bounds.  A row's sum of squares has positive terms added in a tree of at most 32 sequential and 10
pairwise steps: 42 roundings, 2^-18 with the squares' own; half of it in the reciprocal root, plus
2 units: 2^-18.  Every output is a sum of products of such factors and the inputs; the oracle adds
up the sizes of the terms, and each term is within 2^-16 of itself (a dozen roundings and up to
four statistics).  A sum over T tokens adds T / 1024 sequential terms in a block, then 64 and 16:
at most 2^-16 more for the tokens here.  The output's own rounding is half a step of its type."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from oracle import block_ref as R
from block_testlib import GUARD, HALF, MOE_TYPE, Guarded, assert_close, dev, f64, workspace

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
KINDS = {None: moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL, "token": moe.MOE_GATE_TOKEN, "full": moe.MOE_GATE_FULL}


def make(T, d, h=BF16, w=BF16, gate=None, post=True, pre=True, seed=0, res=1.0, out=1.0, eps=1e-6, scale=1.0):
    """post: True (norm behind the block), False (its output without a norm), None (no block output)."""
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    c = dict(T=T, d=d, ht=h, wt=w, kind=gate, eps=eps, res=res, out=out,
             h=dev(n(T, d) * scale, h), y=None, w_post=None, gate=None, w_pre=None,
             ch=dev(n(T, d), h), cx=None)
    if post is not None:
        c["y"] = dev(n(T, d) * scale, BF16)
        if post:
            c["w_post"] = dev(1 + 0.3 * n(d), w)
        if gate:
            c["gate"] = dev(0.5 + n(*{"channel": (d,), "token": (T,), "full": (T, d)}[gate]), w)
    if pre:
        c["w_pre"] = dev(1 + 0.3 * n(d), w)
        c["cx"] = dev(n(T, d), BF16)
    return c


def desc(c):
    return moe.norm_desc(c["T"], c["d"], MOE_TYPE[c["ht"]], MOE_TYPE[c["wt"]], KINDS[c["kind"]], c["eps"], c["res"], c["out"])


def forward(c, inplace=False):
    T, d = c["T"], c["d"]
    h_out = Guarded((T, d), c["ht"]) if c["y"] is not None else None
    x = Guarded((T, d), BF16) if c["w_pre"] is not None else None
    h = c["h"]
    if inplace:
        h_out.t.copy_(h)
        h = h_out.t
    moe.moe_norm_forward(desc(c), c["y"], h, c["w_post"], c["gate"], c["w_pre"], h_out and h_out.t, x and x.t)
    torch.cuda.synchronize()
    return h_out and h_out.check(), x and x.check()


def backward(c, h_out, inplace=False, skip=(), dh_out=True):
    T, d, nd = c["T"], c["d"], desc(c)
    shapes = {"dh": ((T, d), c["ht"])}
    if c["y"] is not None:
        shapes["dy"] = ((T, d), BF16)
        if c["w_post"] is not None:
            shapes["dw_post"] = ((d,), c["wt"])
        if c["gate"] is not None:
            shapes["dgate"] = (tuple(c["gate"].shape), c["wt"])
    if c["w_pre"] is not None:
        shapes["dw_pre"] = ((d,), c["wt"])
    o = {n: Guarded(*s) for n, s in shapes.items() if n not in skip}
    t = {n: o[n].t if n in o else None for n in ("dh", "dy", "dw_post", "dgate", "dw_pre")}
    up = c["ch"] if dh_out else None
    if inplace:
        t["dh"].copy_(up)
        up = t["dh"]
    nb = moe.moe_norm_workspace_bytes(nd)
    ws = workspace(nb + 256)
    moe.moe_norm_backward(nd, c["y"], h_out if c["w_pre"] is not None else None, c["w_post"], c["gate"], c["w_pre"], up,
                          c["cx"], t["dh"], t["dy"], t["dw_post"], t["dgate"], t["dw_pre"], ws, nb)
    torch.cuda.synchronize()
    assert torch.all(ws[nb:] == 0xA5), "written behind the workspace"
    return {n: g.check() for n, g in o.items()}


def ref_kw(c):
    return dict(y=f64(c["y"]), w_post=f64(c["w_post"]), gate=None if c["gate"] is None else (c["kind"], f64(c["gate"])),
                w_pre=f64(c["w_pre"]), eps=float(np.float32(c["eps"])), res_scale=float(np.float32(c["res"])),
                out_scale=float(np.float32(c["out"])))


def check_forward(c, h_out, x):
    kw = ref_kw(c)
    ref_h, ref_x = R.norm_forward(f64(c["h"]), **kw)
    h = f64(c["h"])
    size = np.abs(h)
    if ref_h is not None:
        size = np.abs(kw["res_scale"] * h) + np.abs(ref_h - kw["res_scale"] * h)
        assert_close("h_out", h_out, ref_h, 2.0 ** -16 * size + HALF[c["ht"]] * np.abs(ref_h))
    if ref_x is not None:
        out = h if ref_h is None else ref_h
        rms = np.sqrt((out * out).mean(1, keepdims=True) + c["eps"])
        # the row's rms moves by at most its values' errors' rms
        e = 2.0 ** -16 * size
        err = np.abs(kw["w_pre"]) / rms * (e + np.abs(out) * np.sqrt((e * e).mean(1, keepdims=True)) / rms)
        assert_close("x", x, ref_x, err + 2.0 ** -16 * np.abs(ref_x) + HALF[BF16] * np.abs(ref_x))


def check_backward(c, h_out, o, dh_out=True):
    kw = ref_kw(c)
    g, s = R.norm_backward(f64(c["ch"]) if dh_out else None, h_out=f64(h_out) if c["w_pre"] is not None else None,
                           dx=f64(c["cx"]), **kw)
    types = {"dh": c["ht"], "dy": BF16, "dw_post": c["wt"], "dgate": c["wt"], "dw_pre": c["wt"]}
    for n, t in o.items():
        assert_close(n, t, g[n], 2.0 ** -15 * s[n] + HALF[types[n]] * (np.abs(g[n]) + 2.0 ** -15 * s[n]))


SHAPES = [(1, 8), (1, 2048), (3, 16), (40, 128), (33, 136), (9, 256), (19, 264), (5, 504), (7, 512), (130, 520), (4, 1024),
          (9, 1032), (3, 1536), (4, 1544), (33, 2048), (6, 2056), (4, 3000), (3, 3600), (5, 4096), (3, 4104), (2, 6144),
          (2, 6152), (2, 7168), (2, 8192), (2, 8200), (1, 16384)]


@pytest.mark.parametrize("T,d", SHAPES)
def test_shapes(T, d):
    """Every split of a row over waves and vectors, and rows that fill none of them."""
    for i, (h, w, gate) in enumerate([(BF16, BF16, "channel"), (F32, F32, "token")]):
        print(f"[case] norm T={T} d={d} {h} {gate}", flush=True)
        c = make(T, d, h, w, gate, seed=100 + d + i)
        h_out, x = forward(c)
        check_forward(c, h_out, x)
        check_backward(c, h_out, backward(c, h_out))


FORMS = [(g, post, pre) for g in KINDS for post, pre in [(True, True), (True, False), (False, True), (False, False)]]


@pytest.mark.parametrize("gate,post,pre", FORMS + [(None, None, True)])   # a gate needs the block's output
@pytest.mark.parametrize("h,w", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_forms(h, w, post, pre, gate):
    print(f"[case] norm form {h} {w} post={post} pre={pre} gate={gate}", flush=True)
    for d in (136, 1536):
        c = make(37, d, h, w, gate, post, pre, seed=7, res=0.75, out=1.5)
        h_out, x = forward(c)
        check_forward(c, h_out, x)
        stream = c["h"] if post is None else h_out
        o = backward(c, stream)
        check_backward(c, stream, o)
        if pre:   # no gradient from above: the block's input alone is used
            check_backward(c, stream, backward(c, stream, dh_out=False), dh_out=False)
        if post is not None:
            again, x2 = forward(c, inplace=True)
            assert torch.equal(again, h_out) and (x is None or torch.equal(x, x2))
        o2 = backward(c, stream, inplace=True)
        for n in o:
            assert torch.equal(o[n], o2[n]), f"{n}: in place differs"
        for n in o:   # one output left out changes no other
            o3 = backward(c, stream, skip=(n,))
            for q in o3:
                assert torch.equal(o[q], o3[q]), f"{q} without {n}"


def test_many_rows_sum_in_a_fixed_order():
    """More rows than blocks walk at once; weights' gradients bitwise the same from run to run."""
    for T, d, gate in ((20001, 64, "channel"), (9001, 200, "token"), (2600, 1024, "channel"), (2311, 2048, "full"),
                       (1100, 1536, "token"), (700, 4096, "channel"), (600, 8000, "full"), (520, 16384, "channel")):
        print(f"[case] norm rows T={T} d={d} {gate}", flush=True)
        c = make(T, d, BF16, F32, gate, seed=T)
        h_out, x = forward(c)
        check_forward(c, h_out, x)
        o = backward(c, h_out)
        check_backward(c, h_out, o)
        o2 = backward(c, h_out)
        for n in o:
            assert torch.equal(o[n], o2[n])


def test_rows_of_zeros_and_of_far_sizes():
    """eps carries a row of zeros; tiny and huge rows beside each other."""
    print("[case] norm zeros", flush=True)
    c = make(6, 256, F32, F32, None, seed=3, eps=1e-5)
    c["h"][0], c["y"][0] = 0, 0
    c["h"][1] *= 1e-4
    c["y"][1] *= 2.0 ** -20
    c["h"][2] *= 1e6
    c["y"][2] *= 2.0 ** 20
    h_out, x = forward(c)
    check_forward(c, h_out, x)
    assert torch.all(h_out[0] == 0) and torch.all(x[0] == 0)
    check_backward(c, h_out, backward(c, h_out))


def test_a_bad_row_stays_alone():
    print("[case] norm NaN row", flush=True)
    c = make(9, 1024, BF16, BF16, "token", seed=4)
    good, gx = forward(c)
    c["y"][4, 3] = float("nan")
    h_out, x = forward(c)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(h_out[keep], good[keep]) and torch.equal(x[keep], gx[keep])
    assert torch.isnan(h_out[4]).all() and torch.isnan(x[4]).all()


def test_no_rows_writes_zero_gradients():
    print("[case] norm T=0", flush=True)
    nd = moe.norm_desc(0, 64, gate=moe.MOE_GATE_CHANNEL)
    o = [Guarded((64,), BF16) for _ in range(3)]
    w = torch.ones(64, dtype=BF16, device="cuda")
    moe.moe_norm_forward(nd, w, None, w, None, w, None, None)
    moe.moe_norm_backward(nd, None, None, w, None, w, None, None, None, None, o[0].t, o[1].t, o[2].t, workspace(256))
    torch.cuda.synchronize()
    for g in o:
        assert not g.check().any()
    assert GUARD == 64


def test_gradient_against_differences():
    """Central differences of the forward on the GPU, fp32 stream: step 2^-6, the value's fp32
    rounding (terms of size up to S: 2^-22 S) over a step is 2^-16 S; x's bf16 rounding is kept out by
    differentiating h_out alone."""
    print("[case] norm differences", flush=True)
    c = make(3, 64, F32, F32, "channel", pre=False, seed=5, eps=0.1)
    o = backward(c, None)
    step = 2.0 ** -6

    def value():
        h_out, _ = forward(c)
        terms = f64(h_out) * f64(c["ch"])
        return terms.sum(), np.abs(terms).sum()

    for name, grad, i in (("h", "dh", (1, 5)), ("w_post", "dw_post", (9,)), ("gate", "dgate", (63,))):
        t = c[name]
        t[i] += step
        up, size = value()
        t[i] -= 2 * step
        down, _ = value()
        t[i] += step
        assert abs((up - down) / (2 * step) - float(o[grad][i])) <= 2.0 ** -16 * size


@pytest.mark.parametrize("d", [64, 200, 512, 1000, 1536, 2048, 2056, 4096, 5000, 8192, 8200])
def test_forward_many_rows(d):
    """More rows than the card holds at once, the last turn of the blocks ragged; the last size that fits."""
    lanes = next((n for n in (16, 32, 64, 128, 192, 256, 384, 512, 768) if d <= 8 * n), 1024)
    T = 256 * 2048 // lanes
    for i, (rows, h, w, gate) in enumerate([(T + 3, BF16, F32, "channel"), (T + 257, F32, BF16, "token"), (T, BF16, BF16, "full")]):
        print(f"[case] norm T={rows} d={d} {h} {gate}", flush=True)
        c = make(rows, d, h, w, gate, seed=500 + d + i, res=0.75, out=1.5)
        h_out, x = forward(c)
        check_forward(c, h_out, x)
        same = forward(c, inplace=True)
        assert torch.equal(same[0], h_out) and torch.equal(same[1], x)


@pytest.mark.parametrize("d,step", [(64, 32768), (520, 2048), (1536, 1024), (2048, 1024), (8192, 256), (8200, 256)])
def test_backward_many_rows(d, step):
    """Eight and more turns of 256 blocks, the last one ragged: every row once, in whatever order."""
    for i, (T, h, gate) in enumerate([(8 * step + 5, BF16, "channel"), (9 * step - 1, F32, "token")]):
        if T * d > 1 << 24:
            T = 8 * step + 1 if i == 0 else 8 * step
        print(f"[case] norm backward T={T} d={d} {h} {gate}", flush=True)
        c = make(T, d, h, BF16, gate, seed=700 + d + i)
        h_out, _ = forward(c)
        o = backward(c, h_out)
        check_backward(c, h_out, o)
        same = backward(c, h_out, inplace=True)
        assert all(torch.equal(o[n], same[n]) for n in o)
