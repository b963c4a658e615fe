"""Calls that are in flight at once, and sums over tokens that miss no row and take none twice."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from block_testlib import MOE_TYPE, dev, workspace
from test_gpu_balance import make

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Balance:
    """One batch's inputs, outputs and workspace; both directions enqueued without a wait."""

    def __init__(self, c):
        T, E = c["logits"].shape
        self.S, self.T = c["S"], T
        self.dm = moe.dims(T, 128, 128, E, c["k"])
        self.logits, self.ids = dev(c["logits"]), dev(c["ids"], torch.int32)
        self.mask = None if c["mask"] is None else dev(c["mask"], torch.uint8)
        self.goff = None if c["offsets"] is None else dev(c["offsets"], torch.int32)
        self.w, self.d_in = dev(c["w"]), dev(c["d_in"])
        i32 = dict(dtype=torch.int32, device="cuda")
        self.counts, self.tokens = torch.empty((self.S, E), **i32), torch.empty(self.S + 2, **i32)
        self.losses, self.lse = torch.empty(2, device="cuda"), torch.empty(T, device="cuda")
        self.d = torch.empty((T, E), device="cuda")
        self.ws = workspace(moe.moe_balance_workspace_bytes(self.dm, self.S))

    def enqueue(self):
        moe.moe_balance_forward(self.dm, self.logits, self.ids, self.mask, self.goff, self.S, self.counts, self.tokens,
                                self.losses, self.lse, self.ws)
        moe.moe_balance_backward(self.dm, self.logits, self.lse, self.goff, self.S, self.counts, self.tokens, self.w,
                                 self.d_in, self.d)

    def outputs(self):
        return [t.clone().view(torch.int32) for t in (self.counts, self.tokens, self.losses, self.lse, self.d)]

    def spoil(self):
        for t in (self.counts, self.tokens, self.losses, self.lse, self.d):
            t.fill_(-1)
        self.ws.fill_(0xFF)


@pytest.mark.parametrize("T,E,S", [(5000, 64, 3), (100, 128, 1), (40000, 256, 17)])
def test_balance_on_streams_at_once(T, E, S):
    """Four batches on four streams, all enqueued before the first wait, several rounds of them: the
    outputs of each alone, bit for bit."""
    print(f"[case] balance streams T={T} E={E} S={S}", flush=True)
    batches = [Balance(make(T, E, 4, 11 + i, S=S, mask=i % 2 == 0)) for i in range(4)]
    alone = []
    for b in batches:
        b.enqueue()
        torch.cuda.synchronize()
        alone.append(b.outputs())
        b.spoil()
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                b.enqueue()
    torch.cuda.synchronize()
    for b, want in zip(batches, alone):
        assert all(torch.equal(x, y) for x, y in zip(b.outputs(), want))


@pytest.mark.parametrize("h", [BF16, F32])
@pytest.mark.parametrize("T,d", [(8_000_003, 8), (3_000_001, 136), (1_500_007, 264), (600_001, 520), (300_007, 1032),
                                 (200_003, 1544), (150_001, 2056), (100_003, 4104), (70_001, 8192), (40_003, 16384)])
def test_norm_gradient_sums_every_row_once(T, d, h):
    """The gradient of a channel's gate without norms is a plain sum over rows.  With small integers every
    fp32 sum is a whole number below 2^24 and exact in any order: one row left out or taken twice shows."""
    print(f"[case] norm exact sums T={T} d={d} {h}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)

    def ints(high, dtype):
        t = torch.empty((T, d), dtype=dtype, device="cuda")
        for a in range(0, T, 1 << 16):
            t[a:a + (1 << 16)] = torch.randint(0, high, (min(1 << 16, T - a), d), generator=gen, device="cuda").to(dtype)
        return t

    y, D = ints(2, BF16), ints(3, h)
    gate, dgate = torch.ones(d, device="cuda"), torch.empty(d, device="cuda")
    nd = moe.norm_desc(T, d, MOE_TYPE[h], moe.MOE_F32, moe.MOE_GATE_CHANNEL)
    moe.moe_norm_backward(nd, y, None, None, gate, None, D, None, None, None, None, dgate, None,
                          workspace(moe.moe_norm_workspace_bytes(nd)))
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for a in range(0, T, 1 << 16):
        want += (y[a:a + (1 << 16)].double() * D[a:a + (1 << 16)].double()).sum(0)
    assert float(want.max()) < 2 ** 24
    assert torch.equal(dgate.double(), want)


@pytest.mark.parametrize("T,d,rows", [(40_000_003, 8, 64), (2_200_001, 1032, 4)])
def test_norm_weight_gradient_of_long_batches(T, d, rows):
    """A lane adds its block's rows of every turn (256 blocks of `rows` rows: T / (256 rows) terms), then
    the block's rows, 16 partial sums a wave and 16 waves follow: positive terms, so as many roundings
    bound the sum, and 2^-18 the terms' own."""
    print(f"[case] norm long sums T={T} d={d}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    h = torch.empty((T, d), dtype=BF16, device="cuda")
    for a in range(0, T, 1 << 18):
        h[a:a + (1 << 18)] = torch.randn((min(1 << 18, T - a), d), generator=gen, device="cuda").to(BF16)
    w, dw = torch.ones(d, device="cuda"), torch.empty(d, device="cuda")
    nd = moe.norm_desc(T, d, moe.MOE_BF16, moe.MOE_F32)
    moe.moe_norm_backward(nd, None, h, None, None, w, None, h, None, None, None, None, dw,
                          workspace(moe.moe_norm_workspace_bytes(nd)))
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for a in range(0, T, 1 << 18):
        q = h[a:a + (1 << 18)].double()
        want += (q * q * torch.rsqrt(q.square().mean(1, keepdim=True) + nd.eps)).sum(0)
    bound = (T / (256 * rows) + rows + 32) * 2.0 ** -24 + 2.0 ** -18
    assert float(((dw.double() - want).abs() / want).max()) <= bound
