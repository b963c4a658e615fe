"""The blockwise e4m3 quantiser against the fp8 layer itself: the layer fed with what the quantiser writes, and the codes
that the layer makes of its own inputs."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from block_testlib import dev
from moe_testlib import GpuLayer, TOL_FP8, check_full_parity, oracle_full
from workloads import make_prerouted_fp8

pytestmark = pytest.mark.gpu
U8, F32, BF16 = torch.uint8, torch.float32, torch.bfloat16


def quantize(src, form):
    rows, cols = src.shape
    blocks = lambda n: (n + 127) // 128  # noqa: E731
    codes = torch.empty(rows, cols, dtype=U8, device="cuda")
    scales = torch.empty(rows if form == moe.MOE_BLOCK_ROWS else blocks(rows), blocks(cols), device="cuda")
    moe.moe_fp8_quantize(src, rows, cols, form, codes, scales)
    return codes, scales


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_layer_fed_by_the_quantiser(dtype):
    """x by rows and the experts' weights in tiles, quantised on the device; the layer's outputs and gradients against the
    oracle on the values that the codes stand for, within the fp8 layer's tolerance."""
    inp = make_prerouted_fp8(256, 16, 4, 256, 512, 4, 51)
    T, d, f, E = inp.T, inp.d, inp.f, inp.E
    print(f"[case] T={T} d={d} f={f} E={E}", flush=True)
    rng = np.random.default_rng(2)
    x = dev(rng.standard_normal((T, d)), dtype)
    inp.x, inp.x_scale = (t.cpu().numpy() for t in quantize(x, moe.MOE_BLOCK_ROWS))
    for e in range(E):
        w1, w2 = dev(rng.standard_normal((d, 2 * f)) / np.sqrt(d), dtype), dev(rng.standard_normal((f, d)) / np.sqrt(f), dtype)
        inp.W1[e], inp.W1_scale[e] = (t.cpu().numpy() for t in quantize(w1, moe.MOE_BLOCK_TILES))
        inp.W2[e], inp.W2_scale[e] = (t.cpu().numpy() for t in quantize(w2, moe.MOE_BLOCK_TILES))
    check_full_parity(GpuLayer(inp).run(), oracle_full(inp), tol=TOL_FP8)


def test_the_layer_makes_the_same_codes():
    """The backward pass quantises dy by rows into its workspace: the quantiser's codes and scales are found there, bit for
    bit; ordinary values of all sizes, whole powers of two, blocks of zeros."""
    inp = make_prerouted_fp8(200, 8, 4, 512, 256, 2, 52)
    T, d = inp.T, inp.d
    gl = GpuLayer(inp)
    rng = np.random.default_rng(3)
    dy = rng.standard_normal((T, d)) * np.exp2(rng.integers(-40, 40, (T, 1)))
    dy[3, 128:256] = 0
    dy[5] = 0
    dy[7] = np.exp2(rng.integers(-20, 20, d))
    dy[rng.random((T, d)) < 0.05] = 0
    gl.dy = dev(dy, BF16)
    gl.b["ws_bwd"].zero_()
    gl.run()
    codes, scales = quantize(gl.dy, moe.MOE_BLOCK_ROWS)
    ws = gl.b["ws_bwd"].cpu().numpy().tobytes()
    at = ws.find(codes.cpu().numpy().tobytes())
    assert at >= 0, "the layer's codes are others"
    assert ws.find(scales.cpu().numpy().tobytes(), at) >= 0, "the layer's scales are others"
