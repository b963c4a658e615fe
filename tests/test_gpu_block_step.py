"""A whole training step of a block around the routed layer, as a program runs it: norm, gate scores,
routing, balance loss, experts, norm and gated residual; the way back; gradient norm and AdamW.
Against the fp64 oracle end to end, captured in a HIP graph whose replays move on, and on a stream
of its own.

Tolerance, end to end: the layer's own 2e-2 (largest error over largest value) and one bf16 rounding
of at most 2^-8 at each of the four tensors handed on in bf16 (x, y, dy, dx): 3.6e-2, so 4e-2."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
import oracle
from oracle import block_ref as R
from block_testlib import dev, f64
from moe_testlib import rel_err

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TOL = 4e-2
EPS, OUT_SCALE, MAX_NORM = 1e-5, 0.7, 0.5
LR, B1, B2, AEPS = 1e-2, 0.9, 0.95, 1e-8
D_LOSSES = (0.02, 0.003)


class Block:
    """Parameters, states and buffers of one block, and its step."""

    NAMES = ("W1", "W2", "Wg", "w_pre", "w_post", "gate")

    def __init__(self, T, d, f, E, k, seed, dtype=moe.MOE_BF16, eight=False, groups=None, mask=None):
        rng = np.random.default_rng(seed)
        n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        self.shape = (T, d, f, E, k)
        self.dm = moe.dims(T, d, f, E, k, dtype)
        p = {"W1": dev(n(E, d, 2 * f) / np.sqrt(d), BF16), "W2": dev(n(E, f, d) / np.sqrt(f), BF16),
             "Wg": dev(n(d, E) / np.sqrt(d), BF16), "w_pre": dev(1 + 0.2 * n(d)), "w_post": dev(1 + 0.2 * n(d)),
             "gate": dev(0.8 + 0.2 * n(d))}
        self.p = p
        self.g = {q: torch.empty_like(t) for q, t in p.items()}
        self.master = {q: t.float() if t.dtype == BF16 else None for q, t in p.items()}
        self.states, rows = {}, []
        for q in self.NAMES:
            m = p[q].numel()
            st = {}
            if eight and p[q].dtype == BF16:
                st = {"m": torch.zeros(m, dtype=torch.float8_e4m3fn, device="cuda"), "v": torch.zeros(m, dtype=torch.float8_e4m3fn, device="cuda"),
                      "m_scale": torch.zeros((m + 255) // 256, device="cuda"), "v_scale": torch.zeros((m + 255) // 256, device="cuda")}
            else:
                st = {"m": torch.zeros(m, device="cuda"), "v": torch.zeros(m, device="cuda")}
            self.states[q] = st
            rows.append(moe.adamw_tensor(self.g[q], p[q], master=self.master[q], weight_decay=0.1 if "W" in q else 0.0, **st))
        self.list = moe.adamw_tensors(rows)
        self.b = moe.alloc_layer_buffers(self.dm)
        self.h, self.dh_out = dev(n(T, d), F32), dev(n(T, d), F32)
        S = 1 if groups is None else len(groups) - 1
        self.S, self.goff = S, None if groups is None else dev(np.asarray(groups), torch.int32)
        self.mask = None if mask is None else dev(mask, torch.uint8)
        new = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        ws = lambda nb: torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.x, self.logits, self.h_out, self.dy, self.dh = new(T, d, t=BF16), new(T, E), new(T, d), new(T, d, t=BF16), new(T, d)
        self.counts, self.tokens, self.losses, self.lse = new(S, E, t=torch.int32), new(S + 2, t=torch.int32), new(2), new(T)
        self.d_losses = dev(np.array(D_LOSSES, np.float32))
        self.pre = moe.norm_desc(T, d, moe.MOE_F32, moe.MOE_F32, eps=EPS)
        self.post = moe.norm_desc(T, d, moe.MOE_F32, moe.MOE_F32, moe.MOE_GATE_CHANNEL, EPS, 1.0, OUT_SCALE)
        self.ws_bal = ws(moe.moe_balance_workspace_bytes(self.dm, S))
        self.ws_norm = ws(moe.moe_norm_workspace_bytes(self.post))
        self.ws_gate = ws(moe.moe_workspace_bytes(self.dm, moe.MOE_WS_ROUTER))
        self.ws_gn = ws(moe.moe_grad_norm_workspace_bytes(self.list))
        self.norm, self.scale = new(1), new(1)
        self.step_no = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.hyper = moe.adamw_hyper(LR, B1, B2, AEPS, seed=11, d_step=self.step_no, d_grad_scale=self.scale)

    def gradients(self):
        dm, b, p, g = self.dm, self.b, self.p, self.g
        moe.moe_norm_forward(self.pre, None, self.h, None, None, p["w_pre"], None, self.x)
        moe.moe_router_logits(dm, self.x, p["Wg"], self.logits)
        moe.moe_route(dm, self.logits, b["topk_ids"], b["topk_w"], b["counts"], b["offsets"], b["perm"], b["inv_perm"], b["ws_route"])
        moe.moe_balance_forward(dm, self.logits, b["topk_ids"], self.mask, self.goff, self.S, self.counts, self.tokens,
                                self.losses, self.lse, self.ws_bal)
        moe.moe_forward(dm, self.x, None, p["W1"], None, p["W2"], None, b["topk_w"], b["offsets"], b["perm"], b["inv_perm"],
                        b["y"], b["saved"], b["ws_fwd"])
        moe.moe_norm_forward(self.post, b["y"], self.h, p["w_post"], p["gate"], None, self.h_out, None)
        # the way back
        moe.moe_norm_backward(self.post, b["y"], None, p["w_post"], p["gate"], None, self.dh_out, None, self.dh, self.dy,
                              g["w_post"], g["gate"], None, self.ws_norm)
        moe.moe_backward(dm, self.dy, self.x, None, p["W1"], None, p["W2"], None, b["topk_ids"], b["topk_w"], b["offsets"],
                         b["perm"], b["inv_perm"], b["saved"], b["dx"], g["W1"], g["W2"], b["d_topk_w"], b["d_logits"], b["ws_bwd"])
        moe.moe_balance_backward(dm, self.logits, self.lse, self.goff, self.S, self.counts, self.tokens, self.d_losses,
                                 b["d_logits"], b["d_logits"])
        moe.moe_router_backward(dm, self.x, p["Wg"], b["d_logits"], b["dx"], g["Wg"], self.ws_gate)
        moe.moe_norm_backward(self.pre, None, self.h, None, None, p["w_pre"], self.dh, b["dx"], self.dh, None, None, None,
                              g["w_pre"], self.ws_norm)

    def update(self):
        moe.moe_grad_norm(self.list, MAX_NORM, self.norm, self.scale, self.ws_gn)
        self.step_no.add_(1)
        moe.moe_adamw_step(self.hyper, self.list)

    def step(self):
        self.gradients()
        self.update()

    def results(self):
        o = {"h_out": self.h_out, "dh": self.dh, "losses": self.losses, "counts": self.counts, "lse": self.lse,
             "norm": self.norm, "scale": self.scale, "step": self.step_no, "d_logits": self.b["d_logits"]}
        for q in self.NAMES:
            o["p." + q], o["g." + q] = self.p[q], self.g[q]
            if self.master[q] is not None:
                o["master." + q] = self.master[q]
            for s, t in self.states[q].items():
                o[s + "." + q] = t
        return o


CASES = {
    "small": dict(T=96, d=256, f=128, E=8, k=2, seed=60),
    "seqs": dict(T=300, d=384, f=256, E=32, k=4, seed=61, groups=[0, 7, 150, 150, 280], mask=True),
    "one_token": dict(T=1, d=128, f=128, E=16, k=4, seed=62),
}


def build(name, **more):
    c = dict(CASES[name], **more)
    if c.get("mask") is True:
        c["mask"] = (np.random.default_rng(9).random(c["T"]) > 0.2).astype(np.uint8)
    return Block(**c)


@pytest.mark.parametrize("name", list(CASES))
def test_step_against_the_oracle(name):
    print(f"[case] block step {name}", flush=True)
    bl = build(name)
    T, d, f, E, k = bl.shape
    p = {q: f64(t) for q, t in bl.p.items()}
    bl.gradients()
    torch.cuda.synchronize()
    h, dh_out = f64(bl.h), f64(bl.dh_out)
    # forward, from the inputs alone but for the chosen experts
    _, x = R.norm_forward(h, w_pre=p["w_pre"], eps=EPS)
    logits = oracle.router_logits(x, p["Wg"])
    ids = bl.b["topk_ids"].cpu().numpy()
    sel = np.take_along_axis(logits, ids.astype(np.int64), 1)
    w = np.exp(sel - sel.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    y = oracle.forward(x, p["W1"], p["W2"], ids, w)
    kw = dict(y=y, w_post=p["w_post"], gate=("channel", p["gate"]), eps=EPS, out_scale=OUT_SCALE)
    h_out, _ = R.norm_forward(h, **kw)
    bal = R.balance(logits, ids, None if bl.mask is None else f64(bl.mask), None if bl.goff is None else f64(bl.goff).astype(int))
    g1, _ = R.norm_backward(dh_out, **kw)
    ref = oracle.backward(x, p["W1"], p["W2"], ids, w, g1["dy"])
    dl, _ = R.balance_grad(bal, k, D_LOSSES, ref["d_logits"])
    dx_r, dWg = oracle.router_backward(x, p["Wg"], dl)
    g2, _ = R.norm_backward(g1["dh"], h_out=h, w_pre=p["w_pre"], dx=ref["dx"] + dx_r, eps=EPS)
    want = {"W1": ref["dW1"], "W2": ref["dW2"], "Wg": dWg, "w_pre": g2["dw_pre"], "w_post": g1["dw_post"], "gate": g1["dgate"]}
    errs = {"h_out": rel_err(f64(bl.h_out), h_out), "losses": rel_err(f64(bl.losses), bal["losses"]),
            "dh": rel_err(f64(bl.dh), g2["dh"]), "d_logits": rel_err(f64(bl.b["d_logits"]), dl)}
    errs.update({q: rel_err(f64(bl.g[q]), want[q]) for q in bl.NAMES})
    print(f"[case] block step {name}: " + ", ".join(f"{n}={v:.1e}" for n, v in errs.items()), flush=True)
    assert np.array_equal(f64(bl.counts), bal["counts"])
    bad = {n: v for n, v in errs.items() if not v <= TOL}
    assert not bad, bad
    # the update, from the gradients in hand
    before = {q: f64(bl.master[q] if bl.master[q] is not None else bl.p[q]) for q in bl.NAMES}
    bl.update()
    torch.cuda.synchronize()
    norm, scale = R.grad_norm([f64(bl.g[q]) for q in bl.NAMES], MAX_NORM)
    assert abs(float(bl.norm) - norm) <= 2.0 ** -22 * norm and abs(float(bl.scale) - scale) <= 2.0 ** -22 * scale
    for q in bl.NAMES:
        g = f64(bl.g[q])
        new, _, _ = R.adamw(before[q], g, 0 * g, 0 * g, LR, B1, B2, AEPS, 1, 0.1 if "W" in q else 0.0, float(bl.scale))
        got = f64(bl.master[q] if bl.master[q] is not None else bl.p[q])
        # the first step's rate is lr at most; its factors carry a dozen roundings
        assert np.all(np.abs(got - new) <= 2.0 ** -19 * LR + 2.0 ** -22 * np.abs(new)), q


GRAPHS = {"bf16": {}, "bf16_8bit": dict(eight=True), "mxfp8": dict(dtype=moe.MOE_MXFP8, d=256, f=256)}


@pytest.mark.parametrize("kind", list(GRAPHS))
def test_graph_replays_are_the_eager_steps(kind):
    """Three replays move the weights as three eager steps do, bit for bit, with the eager twin's work and
    waits between them; the step number counts on the device."""
    print(f"[case] block step graph {kind}", flush=True)
    eager, captured = build("seqs", **GRAPHS[kind]), build("seqs", **GRAPHS[kind])
    for bl in (eager, captured):        # a warm-up step each, of its own
        bl.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    torch.cuda.synchronize()
    for rep in range(3):
        eager.step()
        torch.cuda.synchronize()
        captured.h_out.fill_(float("nan"))
        captured.losses.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        a, b = eager.results(), captured.results()
        for n in a:
            assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), f"replay {rep}: {n}"
        # a changed input shows in the next replay
        for bl in (eager, captured):
            bl.h.mul_(1.01)
    assert int(captured.step_no) == 4


def test_two_blocks_on_two_streams():
    """Two blocks step at once, each on a stream and with workspaces of its own."""
    print("[case] block step two streams", flush=True)
    alone = [build("seqs", seed=70 + i) for i in range(2)]
    for bl in alone:
        bl.step()
        bl.step()
    torch.cuda.synchronize()
    both = [build("seqs", seed=70 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(2):
        for bl, s in zip(both, streams):
            with torch.cuda.stream(s):
                bl.step()
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        a, b = x.results(), y.results()
        for n in a:
            assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


def test_a_gradient_that_is_not_finite_skips_the_update():
    print("[case] block step skipped", flush=True)
    bl = build("small")
    bl.step()
    bl.gradients()
    bl.g["W2"].view(-1)[5] = float("inf")
    before = {n: t.clone() for n, t in bl.results().items() if n.split(".")[0] in ("p", "master", "m", "v")}
    bl.update()
    torch.cuda.synchronize()
    assert torch.isnan(bl.scale).all()
    for n, t in before.items():
        assert torch.equal(t, bl.results()[n]), n
