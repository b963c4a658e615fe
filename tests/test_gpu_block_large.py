"""Sizes past 32 bits: offsets, grids that one launch cannot hold, long sums.  Samples against the
fp64 oracle or against the same call on a small copy, whole tensors against torch sums in 64 bits."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from oracle import block_ref as R
from block_testlib import assert_close, f64, workspace

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def fill(n, dtype, seed, scale):
    """Seeded values, drawn in pieces."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = torch.empty(n, dtype=dtype, device="cuda")
    for a in range(0, n, 1 << 28):
        z = min(n, a + (1 << 28))
        t[a:z] = (torch.randn(z - a, generator=gen, device="cuda") * scale).to(dtype)
    return t


def test_adamw_and_norm_of_a_tensor_past_32_bits():
    """More values than 2^32, so more blocks than a launch takes: the pieces around the launches' borders and
    the tail are what a small tensor of the same values gives."""
    n = (1 << 32) + 2 * 256 + 5
    print(f"[case] adamw n={n}", flush=True)
    g, p = fill(n, BF16, 1, 1e-2), fill(n, BF16, 2, 0.1)
    blocks = (n + 255) // 256
    m, v = (torch.zeros(n, dtype=F8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(blocks, device="cuda") for _ in range(2))
    tl = moe.adamw_tensors([moe.adamw_tensor(g, p, m, v, None, ms, vs, 0.1)])
    norm, scale = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_grad_norm(tl, 1.0, norm, scale, workspace(moe.moe_grad_norm_workspace_bytes(tl)))
    total = sum(float(g[a:a + (1 << 28)].double().square().sum()) for a in range(0, n, 1 << 28))
    assert abs(float(norm) - total ** 0.5) <= 2.0 ** -22 * total ** 0.5
    spots = [0, (1 << 30) - 512, 1 << 31, (1 << 32) - 1024, (1 << 32) - 256, 1 << 32, n - 5 - 256]
    size = 768
    before = [(p[a:a + size].clone(), g[a:a + size].clone()) for a in spots]
    hp = moe.adamw_hyper(1e-2, step=1, seed=5)
    moe.moe_adamw_step(hp, tl)
    torch.cuda.synchronize()
    for a, (p0, g0) in zip(spots, before):
        k = p0.numel()
        sm, sv = torch.zeros(k, dtype=F8, device="cuda"), torch.zeros(k, dtype=F8, device="cuda")
        s1, s2 = torch.zeros((k + 255) // 256, device="cuda"), torch.zeros((k + 255) // 256, device="cuda")
        moe.moe_adamw_step(hp, moe.adamw_tensors([moe.adamw_tensor(g0, p0, sm, sv, None, s1, s2, 0.1)]))
        assert torch.equal(p0, p[a:a + k]), a
        b = a // 256
        assert torch.equal(s1, ms[b:b + s1.numel()]) and torch.equal(s2, vs[b:b + s2.numel()]), a
        # codes: rounded with other random bits, so within one code of each other
        for x, y in ((sm, m), (sv, v)):
            x, y = x.view(torch.uint8).int(), y[a:a + k].view(torch.uint8).int()
            assert int((x - y).abs().max()) <= 1, a
    assert torch.isfinite(p[-4096:].float()).all()


def test_adamw_with_fp32_states_past_a_launch():
    """A tensor that three launches share, between small ones: around the launches' borders and in the tail
    the same bits as a small tensor of these values, and the tensors behind it have their own step."""
    n, head = (1 << 31) + 3 * 256 + 9, 1001
    print(f"[case] adamw fp32 states n={n}", flush=True)
    sizes = [head, n, 0, 777]
    ps = [fill(k, BF16, 10 + i, 0.1) for i, k in enumerate(sizes)]
    gs = [fill(k, BF16, 20 + i, 1e-2) for i, k in enumerate(sizes)]
    ms = [torch.zeros(k, device="cuda") for k in sizes]
    vs = [torch.zeros(k, device="cuda") for k in sizes]
    row = lambda p, g, m, v: moe.adamw_tensor(g, p, m, v, weight_decay=0.1)  # noqa: E731
    first = (1 << 30) - 4 * 256   # the first launch holds `head` in 4 blocks of 256 values
    spots = [(1, a) for a in (0, first - 512, (1 << 30) - 256, first + (1 << 30) - 512, 1 << 31, n - 9 - 256)]
    spots += [(0, 0), (3, 0)]
    size = 768
    before = [(ps[i][a:a + size].clone(), gs[i][a:a + size].clone()) for i, a in spots]
    hp = moe.adamw_hyper(1e-2, step=1)
    moe.moe_adamw_step(hp, moe.adamw_tensors([row(*q) for q in zip(ps, gs, ms, vs)]))
    torch.cuda.synchronize()
    for (i, a), (p0, g0) in zip(spots, before):
        k = p0.numel()
        m0, v0 = torch.zeros(k, device="cuda"), torch.zeros(k, device="cuda")
        moe.moe_adamw_step(hp, moe.adamw_tensors([row(p0, g0, m0, v0)]))
        assert torch.equal(p0, ps[i][a:a + k]), (i, a)
        assert torch.equal(m0, ms[i][a:a + k]) and torch.equal(v0, vs[i][a:a + k]), (i, a)
    for a in range(0, n, 1 << 28):    # no value left out
        assert int((vs[1][a:a + (1 << 28)] == 0).sum()) == int((gs[1][a:a + (1 << 28)] == 0).sum())


@pytest.mark.parametrize("T,d", [(40_000_003, 8), (2_200_001, 1032)])
def test_norm_rows_past_a_grid(T, d):
    """More rows than a grid's blocks, offsets past 32 bits: sampled rows, and the weight's gradient whole."""
    print(f"[case] norm T={T} d={d}", flush=True)
    h = fill(T * d, BF16, 3, 1.0).view(T, d)
    w = 1 + 0.1 * torch.arange(d, device="cuda") / d
    x = torch.empty_like(h)
    nd = moe.norm_desc(T, d, moe.MOE_BF16, moe.MOE_F32)
    moe.moe_norm_forward(nd, None, h, None, None, w, None, x)
    rows = torch.tensor([0, 1, 17, T // 2, (1 << 21) - 1, (1 << 21) + 1, T - 2, T - 1], device="cuda")
    _, ref = R.norm_forward(f64(h[rows]), w_pre=f64(w))
    assert_close("x", x[rows], ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * np.abs(ref))
    dx, dh = h, torch.empty_like(h)   # the gradient of x: the stream's own values serve
    dw = torch.empty(d, device="cuda")
    moe.moe_norm_backward(nd, None, h, None, None, w, None, dx, dh, None, None, None, dw,
                          workspace(moe.moe_norm_workspace_bytes(nd)))
    g, s = R.norm_backward(None, h_out=f64(h[rows]), w_pre=f64(w), dx=f64(dx[rows]))
    assert_close("dh", dh[rows], g["dh"], 2.0 ** -15 * s["dh"] + 2.0 ** -8 * np.abs(g["dh"]))
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for a in range(0, T, 1 << 18):
        q = h[a:a + (1 << 18)].double()
        want += (q * q * torch.rsqrt(q.square().mean(1, keepdim=True) + nd.eps)).sum(0)
    # every term is positive; a block adds T / 512 of them or less one after the other, with rounding
    # errors of either sign: within (T / 512) 2^-24 at most
    assert float(((dw.double() - want).abs() / want).max()) <= T / 512 * 2.0 ** -24


def test_balance_of_more_tokens_than_a_grid():
    T, E, k = (1 << 27) + 77, 2, 1
    print(f"[case] balance T={T}", flush=True)
    dm = moe.dims(T, 128, 128, E, k)
    logits = fill(T * E, torch.float32, 4, 1.0).view(T, E)
    ids = (logits[:, 1] > logits[:, 0]).to(torch.int32).view(T, 1).contiguous()
    counts, tokens = torch.empty((1, E), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    losses, lse, d = torch.empty(2, device="cuda"), torch.empty(T, device="cuda"), torch.empty((T, E), device="cuda")
    moe.moe_balance_forward(dm, logits, ids, None, None, 1, counts, tokens, losses, lse,
                            workspace(moe.moe_balance_workspace_bytes(dm, 1)))
    moe.moe_balance_backward(dm, logits, lse, None, 1, counts, tokens, torch.tensor([1.0, 0.5], device="cuda"), None, d)
    torch.cuda.synchronize()
    ones = int(ids.sum())
    assert counts.tolist() == [[T - ones, ones]] and tokens.tolist() == [T, T, 1]
    P, z = torch.zeros(E, dtype=torch.float64, device="cuda"), 0.0
    for a in range(0, T, 1 << 24):
        q = logits[a:a + (1 << 24)].double()
        l = torch.logsumexp(q, 1)
        P += torch.exp(q - l[:, None]).sum(0)
        z += float(l.square().sum())
    bal = E / (k * float(T) ** 2) * float((counts[0].double() * P).sum())
    # sums of at most T / 65536 / 16 terms in fp32 between sums in 64 bits, and the terms' own 2^-16
    assert abs(float(losses[0]) - bal) <= 2.0 ** -15 * bal and abs(float(losses[1]) - z / T) <= 2.0 ** -14 * z / T
    rows = torch.tensor([0, 5, T // 2, T - 1], device="cuda")
    l64 = f64(logits[rows])
    p = np.exp(l64 - np.log(np.exp(l64).sum(1, keepdims=True)))
    lse64 = np.log(np.exp(l64).sum(1, keepdims=True))
    c = np.array([T - ones, ones], np.float64)
    ref = p * (E / (k * float(T) ** 2) * (c - (c * p).sum(1, keepdims=True)) + lse64 / T)
    size = p * (E / (k * float(T) ** 2) * np.abs(c - T / 2) .max() * 2 + np.abs(lse64) / T)
    assert_close("d_logits", d[rows], ref, 2.0 ** -14 * size)
