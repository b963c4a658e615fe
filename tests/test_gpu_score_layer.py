"""The routing by scores, the blockwise quantiser and the blockwise e4m3 product as a layer uses them, run
together: logits of the router, choice with groups, balance bias and a token mask, the experts' products forward
and backward, the gradient through the scores into the router, one step of the bias; beside them a dense expert that every token
runs through, as blockwise e4m3 products with their gradients.  Against the fp64 oracle, and the whole captured as
one graph and replayed.

Bounds.  The choice and the plan: equal, on the layer's own logits.  The experts' path and the router: the layer's
own comparison (largest error over largest value, 2e-2).  The dense expert, on the values the codes stand for: the
product's bound of an fp32 C, (128 + 2 blocks) 2^-23 of the terms' magnitudes."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
import oracle
from oracle import score_ref as S
from block_testlib import dev, f64, workspace
from moe_testlib import GpuLayer, TOL_BF16, bf16_dev, rel_err, to_np
from workloads import make_inputs

pytestmark = pytest.mark.gpu
F8, U8, BF16, F32 = torch.float8_e4m3fn, torch.uint8, torch.bfloat16, torch.float32
RATE = float(np.float32(1e-3))   # the call's argument is fp32: 1e-3 itself is up to 2^-24 off, enough for another rounding


def empty(*s, t=F32):
    return torch.empty(s, dtype=t, device="cuda")


class Layer:
    """The buffers of one layer and its step."""

    def __init__(self, T, d, f, E, k, seed, sigmoid, renorm, groups, keep):
        self.inp = inp = make_inputs(T, d, f, E, k, seed=seed)
        self.gl = GpuLayer(inp)
        self.dm, self.b = self.gl.dm, self.gl.b
        self.Wg = bf16_dev(inp.Wg)
        self.sd = moe.score_desc(T, E, k, moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX, renorm, 2.5, groups, keep, 2)
        rng = np.random.default_rng(seed)
        self.bias_np = (rng.standard_normal(E) * 0.05).astype(np.float32)
        self.mask_np = (rng.random(T) < 0.9).astype(np.uint8)
        self.bias, self.mask = dev(self.bias_np), dev(self.mask_np, U8)
        self.logits, self.d_logits, self.dWg, self.next_bias = empty(T, E), empty(T, E), empty(d, E, t=BF16), empty(E)
        self.ws = workspace(moe.moe_score_workspace_bytes(self.sd))
        self.ws_router = workspace(moe.moe_workspace_bytes(self.dm, moe.MOE_WS_ROUTER))
        # the dense expert: y = x W, W [d, N]; gradients of x (with W in the same form) and of W
        self.N = N = 2 * f
        self.W = dev(rng.standard_normal((d, N)) / np.sqrt(d))
        up = (T + 15) // 16 * 16
        self.wq, self.wqs = empty(d, N, t=U8), empty((d + 127) // 128, (N + 127) // 128)
        self.md = moe.matmul_desc(T, N, d, moe.MOE_B_KN, moe.MOE_F32)
        self.back = moe.matmul_desc(T, d, N, moe.MOE_B_NK, moe.MOE_F32)
        self.grad = moe.matmul_desc(d, N, up, moe.MOE_B_NK_ROWS, moe.MOE_F32)
        tb = (T + 127) // 128
        cb = lambda n: (n + 127) // 128  # noqa: E731
        self.dense = {"xq": empty(T, d, t=U8), "xs": empty(T, cb(d)), "y": empty(T, N), "gq": empty(T, N, t=U8), "gs": empty(T, cb(N)),
                      "dx": empty(T, d), "xt": empty(d, up, t=U8), "xts": empty(d, tb), "gt": empty(N, up, t=U8), "gts": empty(N, tb),
                      "dW": empty(d, N)}
        self.ws_dense = workspace(max(moe.moe_fp8_matmul_workspace_bytes(m) for m in (self.md, self.back, self.grad)))

    def step(self):
        gl, b, q, T, d, N = self.gl, self.b, self.dense, self.inp.T, self.inp.d, self.N
        moe.moe_router_logits(self.dm, gl.x, self.Wg, self.logits)
        moe.moe_score_route(self.sd, self.logits, self.bias, self.mask, b["topk_ids"], b["topk_w"], b["counts"], b["offsets"],
                            b["perm"], b["inv_perm"], self.ws)
        gl.forward()
        gl.backward(with_logits=False)
        moe.moe_score_backward(self.sd, self.logits, b["topk_ids"], b["d_topk_w"], self.d_logits)
        moe.moe_router_backward(self.dm, gl.x, self.Wg, self.d_logits, b["dx"], self.dWg, self.ws_router)
        moe.moe_bias_update(b["counts"], RATE, self.bias, self.next_bias)
        moe.moe_fp8_quantize(self.W, d, N, moe.MOE_BLOCK_TILES, self.wq, self.wqs)
        moe.moe_fp8_quantize(gl.x, T, d, moe.MOE_BLOCK_ROWS, q["xq"], q["xs"])
        moe.moe_fp8_matmul(self.md, q["xq"], q["xs"], self.wq, self.wqs, None, q["y"], self.ws_dense)
        moe.moe_fp8_quantize(q["y"], T, N, moe.MOE_BLOCK_ROWS, q["gq"], q["gs"])
        moe.moe_fp8_matmul(self.back, q["gq"], q["gs"], self.wq, self.wqs, None, q["dx"], self.ws_dense)
        moe.moe_fp8_quantize(gl.x, T, d, moe.MOE_BLOCK_TOKENS, q["xt"], q["xts"])
        moe.moe_fp8_quantize(q["y"], T, N, moe.MOE_BLOCK_TOKENS, q["gt"], q["gts"])
        moe.moe_fp8_matmul(self.grad, q["xt"], q["xts"], q["gt"], q["gts"], None, q["dW"], self.ws_dense)

    def outputs(self):
        names = ("topk_ids", "topk_w", "counts", "offsets", "y", "dx", "d_topk_w")
        return [self.b[n] for n in names] + [self.logits, self.d_logits, self.dWg, self.next_bias] + list(self.dense.values())


def values(codes, scales):
    v = codes.view(F8).double()
    t = scales.double().repeat_interleave(128, 1)[:, :v.shape[1]]
    if t.shape[0] != v.shape[0]:
        t = t.repeat_interleave(128, 0)[:v.shape[0]]
    return v * t


CASES = {
    # name: (T, d, f, E, k, seed, sigmoid, renormalised, groups, groups kept)
    "sigmoid_groups": (300, 256, 128, 32, 4, 70, True, True, 8, 4),
    "softmax": (77, 384, 128, 100, 5, 71, False, False, 1, 1),
    "one_token": (1, 256, 128, 16, 2, 72, True, False, 4, 2),
    "sigmoid_256": (40, 128, 256, 256, 8, 73, True, True, 8, 4),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_layer_routed_by_scores(name):
    T, d, f, E, k, seed, sigmoid, renorm, groups, keep = CASES[name]
    print(f"[case] {name}", flush=True)
    la = Layer(*CASES[name])
    if T == 1:
        la.mask_np[:] = 1
        la.mask.fill_(1)
    la.step()
    torch.cuda.synchronize()
    inp, b = la.inp, la.b
    x, Wg, W1, W2, dy = (oracle.bf16_to_f64(a) for a in (inp.x, inp.Wg, inp.W1, inp.W2, inp.dy))
    logits = to_np(la.logits)
    ids, w = S.route(logits, k, sigmoid, renorm, 2.5, la.bias_np, la.mask_np, groups, keep, 2)
    assert np.array_equal(to_np(b["topk_ids"]), ids)
    assert (ids[la.mask_np == 0] == -1).all() and (ids[la.mask_np == 1] >= 0).all()
    pl = oracle.plan(ids, E)
    assert np.array_equal(to_np(b["counts"]), pl.counts) and np.array_equal(to_np(b["offsets"]), pl.offsets)
    assert np.array_equal(to_np(la.next_bias), np.asarray(S.bias_update(pl.counts, RATE, la.bias_np), np.float32))
    ref = oracle.backward(x, W1, W2, ids, w, dy, logits_routed=False)
    # through the scores, on the layer's own gradient of the weights and on the oracle's
    dl, _ = S.backward(logits, ids, to_np(b["d_topk_w"]), sigmoid, renorm, 2.5)
    dl_ref, _ = S.backward(logits, ids, ref["d_topk_w"], sigmoid, renorm, 2.5)
    dx_r, dWg = oracle.router_backward(x, Wg, dl_ref)
    errs = {"logits": rel_err(logits, oracle.router_logits(x, Wg)), "w": rel_err(to_np(b["topk_w"]), w),
            "y": rel_err(to_np(b["y"]), oracle.forward(x, W1, W2, ids, w)), "d_w": rel_err(to_np(b["d_topk_w"]), ref["d_topk_w"]),
            "d_logits": rel_err(to_np(la.d_logits), dl), "dx": rel_err(to_np(b["dx"]), ref["dx"] + dx_r), "dWg": rel_err(to_np(la.dWg), dWg)}
    print(f"[case] {name}: " + ", ".join(f"{n}={v:.2e}" for n, v in errs.items()), flush=True)
    bad = {n: v for n, v in errs.items() if not v <= TOL_BF16}
    assert not bad, bad
    # the dense expert
    q = la.dense
    xv, wv, gv = values(q["xq"], q["xs"]), values(la.wq, la.wqs), values(q["gq"], q["gs"])
    xt, gt = values(q["xt"], q["xts"]), values(q["gt"], q["gts"])
    for got, a, bm, K in ((q["y"], xv, wv, d), (q["dx"], gv, wv.t().contiguous(), la.N), (q["dW"], xt, gt.t().contiguous(), xt.shape[1])):
        want, size = f64(a @ bm), f64(a.abs() @ bm.abs())
        assert (np.abs(f64(got) - want) <= size * (128 + 2 * ((K + 127) // 128)) * 2.0 ** -23 + np.abs(want) * 2.0 ** -24).all()
    assert np.abs(f64(xv) - x).max() <= np.abs(x).max() * 2.0 ** -4


def test_layer_in_a_graph():
    """The step captured once and replayed, with eager steps between the replays; bit for bit the first one's."""
    la = Layer(*CASES["sigmoid_groups"])
    la.step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in la.outputs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        la.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.step()
    for turn in range(6):
        for t in la.outputs():
            t.zero_()
        graph.replay() if turn % 2 == 0 else la.step()
        torch.cuda.synchronize()
        for i, (a, c) in enumerate(zip(ref, la.outputs())):
            assert torch.equal(a.view(U8), c.view(U8)), (turn, i)
