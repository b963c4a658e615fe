"""The blockwise e4m3 quantiser and matrix product, against the fp64 oracle.

Bounds.  Quantiser: the oracle computes in the format's own fp32 steps (one quotient, one product), so
codes and scales are equal bit for bit.  Product: with codes of small whole numbers and scales that are
powers of two every sum is exact, and the result equal to the 64-bit one rounded to C's type.  With any
codes and scales: products of codes are exact, a sum over one block has at most 128 roundings and the sum
over ceil(K / 128) blocks two each; a matrix instruction may truncate, so each rounding counts a whole
step, 2^-23, of at most the sum of all terms' magnitudes; then half a step of C's type.  For a bf16 C the
matrix instruction works on eight products at a time, aligned to the largest, m: seven of them lose less
than 2^-13 m each, together less than 7 2^-13 m <= 7 2^-13 (the eight magnitudes' sum), so that over all
groups the result loses at most 7 2^-13 of the sum of all terms' magnitudes."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from oracle import score_ref as S
from block_testlib import HALF, MOE_TYPE, Guarded, assert_close, dev, f64, workspace

pytestmark = pytest.mark.gpu
BF16, F32, U8, F8 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn
FORMS = {"rows": moe.MOE_BLOCK_ROWS, "tokens": moe.MOE_BLOCK_TOKENS, "tiles": moe.MOE_BLOCK_TILES}
B_FORMS = {"kn": moe.MOE_B_KN, "nk": moe.MOE_B_NK, "rows": moe.MOE_B_NK_ROWS}


def up(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------------------- quantiser
def quantize(src, rows, cols, form, ld=None):
    shapes = {"rows": ((rows, cols), (rows, up(cols, 128) // 128)), "tiles": ((rows, cols), (up(rows, 128) // 128, up(cols, 128) // 128)),
              "tokens": ((cols, up(rows, 16)), (cols, up(rows, 128) // 128))}[form]
    codes, scales = Guarded(shapes[0], U8, fill=0x5A), Guarded(shapes[1], F32)
    moe.moe_fp8_quantize(src, rows, cols, FORMS[form], codes.t, scales.t, ld)
    torch.cuda.synchronize()
    return codes.check(), scales.check()


def check_quantize(x, form, dtype, ld=None):
    rows, cols = x.shape
    t = dev(x, dtype)
    wide = torch.full((rows, ld or cols), float("nan"), dtype=dtype, device="cuda")
    wide[:, :cols] = t
    codes, scales = quantize(wide, rows, cols, form, ld)
    ref_codes, ref_scales = S.quantize(t.float().cpu().numpy(), form)
    assert np.array_equal(scales.cpu().numpy(), ref_scales)
    assert np.array_equal(codes.cpu().numpy(), ref_codes)


QSHAPES = [(1, 16), (1, 128), (3, 144), (16, 112), (17, 7168), (127, 272), (128, 128), (129, 64), (130, 80), (257, 400), (300, 1040),
           (1, 2048), (2100, 16)]


@pytest.mark.parametrize("shape", QSHAPES, ids=str)
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantize(shape, form, dtype):
    print(f"[case] quantize {shape} {form} {dtype}", flush=True)
    rng = np.random.default_rng(shape[0] + shape[1])
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-8, 8, (shape[0], 1))) * np.exp(rng.standard_normal(shape[1]))
    x[rng.random(shape) < 0.05] = 0
    check_quantize(x.astype(np.float32), form, dtype)
    if shape[1] <= 400:
        check_quantize(x.astype(np.float32), form, dtype, ld=shape[1] + 24)


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantize_zeros_small_and_large_values(form, dtype):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((256, 256))
    x[:128, :128] = 0
    x[128:, :128] *= 2.0 ** -127        # below fp32's normal range, scale and all
    x[:128, 128:] *= 2.0 ** 124
    x[128:, 128:] *= 2.0 ** -118        # the least scale of a normal one
    check_quantize(x.astype(np.float32), form, dtype)
    for v in (1.0, 448.0, 0.75, 3.0e38, 2.0 ** -126):
        check_quantize(np.full((20, 32), v, np.float32), form, dtype)
    # every e4m3 value and the midpoints between neighbours: ties to even
    tab = np.sort(np.concatenate([S.e4m3_to_f64(np.arange(0x7F)), (S.e4m3_to_f64(np.arange(0x7E)) + S.e4m3_to_f64(np.arange(1, 0x7F))) / 2]))
    x = np.zeros((128, 256))
    x[0, :tab.size] = tab
    x[1, :tab.size] = -tab
    x[:, 0] = x[0, 128] = x[1, 128] = 448
    check_quantize(x.astype(np.float32), form, dtype)


def test_quantize_values_that_are_not_finite():
    x = np.ones((130, 256), np.float32)
    x[3, 5], x[4, 130], x[5, 7], x[5, 9] = np.nan, np.inf, -np.inf, np.nan
    for dtype in (BF16, F32):
        codes, scales = quantize(dev(x, dtype), 130, 256, "rows")
        codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
        v = S.values(codes, scales)
        assert np.isnan(v[3, 5]) and np.isfinite(np.delete(v[3], 5)).all() and scales[3, 0] == np.float32(1 / 448)
        assert np.isinf(scales[4, 1]) and np.isnan(v[4, 128:]).all() and np.isfinite(v[4, :128]).all()
        assert np.isinf(scales[5, 0]) and np.isnan(v[5, :128]).all()
        rest = np.delete(v, [3, 4, 5], 0)
        assert np.allclose(rest, 1, rtol=2.0 ** -23)
        codes, scales = quantize(dev(x, dtype), 130, 256, "tokens")
        v = S.values(codes.cpu().numpy(), scales.cpu().numpy())
        assert np.isnan(v[5, 3]) and np.isnan(v[130, :128]).all() and np.isfinite(v[130, 128:130]).all() and np.isnan(v[7, :128]).all()
        codes, scales = quantize(dev(x, dtype), 130, 256, "tiles")
        assert np.isinf(scales.cpu().numpy()[0]).all() and np.isfinite(scales.cpu().numpy()[1]).all()


def test_the_layers_codes_are_the_quantisers():
    """moe_forward's fp8 inputs as this call makes them: the values it was given, within half a step of e4m3."""
    x = torch.randn(64, 512, device="cuda", dtype=BF16)
    codes, scales = quantize(x, 64, 512, "rows")
    v = codes.view(F8).float().view(64, 4, 128) * scales[:, :, None]
    assert ((v - x.float().view(64, 4, 128)).abs() <= torch.maximum(x.float().abs().view(64, 4, 128) * 2.0 ** -4, scales[:, :, None] * 2.0 ** -10) * 1.001).all()


# --------------------------------------------------------------------------------- product
def operands(M, N, K, form, seed, exact):
    """codes and scales on the device.  exact: whole numbers up to 3 and scales that are powers of two."""
    gen = torch.Generator("cuda").manual_seed(seed)

    def make(shape, tiles):
        R, C = shape
        sr = up(R, 128) // 128 if tiles else R
        if exact:
            c = torch.randint(-3, 4, shape, generator=gen, device="cuda").float().to(F8)
            s = torch.exp2(torch.randint(-2, 3, (sr, up(C, 128) // 128), generator=gen, device="cuda").float())
        else:
            c = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.int32).to(U8)
            c = torch.where((c & 0x7F) == 0x7F, 0x38, c).to(U8).view(F8)
            s = torch.exp(torch.randn((sr, up(C, 128) // 128), generator=gen, device="cuda"))
        return c, s

    a, sa = make((M, K), False)
    b, sb = make((K, N) if form == "kn" else (N, K), form != "rows")
    return a, sa, b, sb


def values(c, s):
    v = c.double()
    t = s.double().repeat_interleave(128, 1)[:, :v.shape[1]]
    if t.shape[0] != v.shape[0]:
        t = t.repeat_interleave(128, 0)[:v.shape[0]]
    return v * t


def strided(t, ld, fill):
    """t with `ld` values from one row to the next; what lies between is `fill`."""
    w = torch.full((t.shape[0], ld), fill, dtype=t.dtype, device="cuda") if t.dtype != F8 else \
        torch.full((t.shape[0], ld), fill, dtype=U8, device="cuda").view(F8)
    w[:, :t.shape[1]] = t
    return w


def product(M, N, K, form, dtype, a, sa, b, sb, c_in=None, pad=0, in_place=False):
    """C of the call, checked for what lies around it.  pad: 16s of codes between rows, which hold NaN."""
    lda, ldb, ldc = a.shape[1] + 16 * pad, b.shape[1] + 16 * pad, N + 8 * pad
    if pad:
        a, b = strided(a, lda, 0x7F), strided(b, ldb, 0x7F)
    md = moe.matmul_desc(M, N, K, B_FORMS[form], MOE_TYPE[dtype], lda, ldb, ldc)
    c = Guarded((M, ldc), dtype)
    if c_in is not None and pad:
        c_in = strided(c_in, ldc, 7.0)
    if in_place:
        c.t.copy_(c_in)
        c_in = c.t
    moe.moe_fp8_matmul(md, a, sa, b, sb, c_in, c.t, workspace(moe.moe_fp8_matmul_workspace_bytes(md)))
    torch.cuda.synchronize()
    c.check()
    assert (c.t[:, N:] == 7).all(), "written between two rows"
    return c.t[:, :N]


def check_exact(M, N, K, form, dtype, seed=0, pad=0, add=False):
    a, sa, b, sb = operands(M, N, K, form, seed, True)
    av, bv = values(a, sa), values(b, sb)
    ref = av @ (bv if form == "kn" else bv.t().contiguous())
    c_in = None
    if add:
        c_in = torch.randint(-50, 50, (M, N), device="cuda").to(dtype)
        ref = ref + c_in.double()
    # below 2^24 times the least product of two scales: every partial sum is a whole multiple of 2^-4
    assert float((av.abs() @ (bv.abs() if form == "kn" else bv.abs().t().contiguous())).max()) + 50 < 2.0 ** 20
    for in_place in ((False, True) if add else (False,)):
        got = product(M, N, K, form, dtype, a, sa, b, sb, c_in, pad, in_place)
        assert torch.equal(got, ref.to(F32).to(dtype))   # the sum fits fp32; one rounding


def check_any(M, N, K, form, dtype, seed=0):
    a, sa, b, sb = operands(M, N, K, form, seed, False)
    av, bv = values(a, sa), values(b, sb)
    if form != "kn":
        bv = bv.t().contiguous()
    got = product(M, N, K, form, dtype, a, sa, b, sb)
    ref, size = f64(av @ bv), f64(av.abs() @ bv.abs())
    dropped = 7 * 2.0 ** -13 if dtype == BF16 else 0.0
    assert_close("C", got, ref, size * ((128 + 2 * up(K, 128) // 128) * 2.0 ** -23 + dropped) + np.abs(ref) * HALF[dtype])


# every border of the tiles, of a block of K and of the rows that one token or a decode batch has
MS = [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 200, 255, 256, 257, 385]
NKS = [(16, 16), (48, 112), (112, 128), (128, 144), (144, 48), (256, 256), (272, 400), (528, 640), (64, 1040), (1040, 272)]


@pytest.mark.parametrize("form", sorted(B_FORMS))
@pytest.mark.parametrize("nk", NKS, ids=str)
def test_product_exact(form, nk):
    N, K = nk
    for i, M in enumerate(MS):
        print(f"[case] product {form} {M}x{N}x{K}", flush=True)
        check_exact(M, N, K, form, (BF16, F32)[i % 2], M, pad=i % 3, add=i % 4 == 1)


@pytest.mark.parametrize("form", sorted(B_FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_product_any_values(form, dtype):
    for M, N, K in ((1, 16, 16), (1, 512, 1024), (7, 144, 272), (16, 256, 2048), (33, 80, 4096), (64, 1024, 512), (100, 272, 1168),
                    (256, 256, 256), (300, 528, 1040), (513, 768, 896)):
        print(f"[case] product {form} {M}x{N}x{K}", flush=True)
        check_any(M, N, K, form, dtype, M)


# long K, few and many rows, wide and narrow: the listed workloads' kinds at whole sizes
LARGE = [("kn", 1, 4096, 7168), ("kn", 16, 7168, 2048), ("nk", 1, 7168, 4096), ("nk", 48, 7168, 2048), ("nk", 5, 2048, 16384),
         ("kn", 33, 1024, 8192), ("nk", 1023, 7168, 4096), ("kn", 4099, 4096, 2048), ("kn", 777, 2064, 7168), ("rows", 2048, 1408, 4112),
         ("rows", 528, 512, 16400), ("rows", 7, 512, 8192), ("nk", 8200, 1040, 1024), ("kn", 2050, 16384, 512), ("kn", 130, 400, 10000),
         ("nk", 300, 64, 16384), ("rows", 64, 4096, 4096)]


@pytest.mark.parametrize("case", LARGE, ids=str)
def test_product_large(case):
    form, M, N, K = case
    check_exact(M, N, K, form, BF16 if M % 2 else F32, 5, add=M % 3 == 0)


# tiles of every shape: whole ones, all of them cut along K, and a card full of whole ones with cut ones behind; a
# stop of K inside a block where a part ends there; rows and columns that end inside a tile
TILES = [(128, 4096, 3100), (300, 8192, 8192), (1023, 4104, 1040), (1500, 2048, 4096), (4099, 4096, 2064), (4100, 4112, 1024),
         (2100, 8192, 1936), (2048, 2048, 7168), (700, 512, 20000), (33000, 272, 656)]


@pytest.mark.parametrize("form", sorted(B_FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_product_tiles(form, dtype):
    for M, N, K in TILES:
        N, K = up(N, 16), up(K, 16)
        print(f"[case] product {form} {M}x{N}x{K}", flush=True)
        check_exact(M, N, K, form, dtype, N, pad=M % 2, add=M % 4 == 0)


def test_product_nan_and_infinite_scales_stay_in_their_rows():
    M, N, K = 70, 144, 272
    for form in B_FORMS:
        a, sa, b, sb = operands(M, N, K, form, 3, True)
        clean = product(M, N, K, form, F32, a, sa, b, sb)
        a.view(U8)[5, 271] = 0x7F
        sa[9, 1] = float("nan")
        got = product(M, N, K, form, F32, a, sa, b, sb)
        assert torch.isnan(got[5]).all() and torch.isnan(got[9]).all()
        keep = [r for r in range(M) if r not in (5, 9)]
        assert torch.equal(got[keep], clean[keep])


def test_rows_do_not_depend_on_the_others():
    """A token's row is the same in every batch that runs the same split of K: here alone and with itself
    repeated; and a call repeated gives the same bits."""
    N, K = 512, 1040
    for form in B_FORMS:
        a, sa, b, sb = operands(300, N, K, form, 8, False)
        first = product(300, N, K, form, F32, a, sa, b, sb)
        assert torch.equal(first, product(300, N, K, form, F32, a, sa, b, sb))
        twice = product(300, N, K, form, F32, a[:1].expand(300, -1).contiguous(), sa[:1].expand(300, -1).contiguous(), b, sb)
        assert (twice == twice[:1]).all() and torch.equal(twice[0], first[0])


def test_offsets_past_32_bits():
    """Operands and results whose last rows lie past 2^31 and 2^32 bytes: a long stride, and a tall product."""
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GiB of GPU memory")
    M, N, K = 40, 32, 144
    for form in ("kn", "nk"):
        a, sa, b, sb = operands(M, N, K, form, 4, True)
        ref = product(M, N, K, form, F32, a, sa, b, sb)
        ld = (1 << 27) + 16
        wide = torch.empty(K * ld, dtype=U8, device="cuda")
        av = torch.as_strided(wide, (M, K), (ld, 1))
        av.copy_(a.view(U8))
        md = moe.matmul_desc(M, N, K, B_FORMS[form], moe.MOE_F32, lda=ld)
        c = torch.empty(M, N, device="cuda")
        ws = workspace(moe.moe_fp8_matmul_workspace_bytes(md))
        moe.moe_fp8_matmul(md, wide, sa, b, sb, None, c, ws)
        assert torch.equal(c, ref)
        bv = torch.as_strided(wide, tuple(b.shape), (ld, 1))
        bv.copy_(b.view(U8))
        md = moe.matmul_desc(M, N, K, B_FORMS[form], moe.MOE_F32, ldb=ld)
        moe.moe_fp8_matmul(md, a, sa, wide, sb, None, c, ws)
        assert torch.equal(c, ref)
        md = moe.matmul_desc(M, N, K, B_FORMS[form], moe.MOE_F32, ldc=1 << 25)
        cw = wide.view(F32)
        moe.moe_fp8_matmul(md, a, sa, b, sb, None, cw, ws)
        assert torch.equal(torch.as_strided(cw, (M, N), (1 << 25, 1)), ref)
        del wide, av, bv, cw
    M, N, K = (1 << 21) + 5, 16, 1040     # A of 2.2e9 bytes
    a = torch.zeros(M, K, dtype=U8, device="cuda")
    a[-3:] = 0x38
    sa = torch.ones(M, 9, device="cuda")
    b, sb = torch.full((N, K), 0x38, dtype=U8, device="cuda"), torch.ones(1, 9, device="cuda")
    got = product(M, N, K, "nk", F32, a.view(F8), sa, b.view(F8), sb)
    assert (got[:-3] == 0).all() and (got[-3:] == K).all()
    # the quantiser, over a source of 4.3e9 bytes
    rows, cols = (1 << 20) + 3, 2048
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[-1] = 3.0
    for form in FORMS:
        codes, scales = quantize(x, rows, cols, form)
        v = codes.view(F8)
        last = v[:, rows - 1] if form == "tokens" else v[-1]
        scale = scales[:, -1] if form == "tokens" else scales[-1].repeat_interleave(128)
        assert torch.allclose(last.float() * scale, torch.full_like(scale, 3.0), rtol=2.0 ** -22)
        assert int((codes != 0).sum()) == cols


# --------------------------------------------------------------------- streams, graphs, repeats
def test_graph_replays_and_streams():
    """A captured quantise and product of every form, replayed with eager work between the replays; the same
    calls on four streams at once with a workspace each; each bit for bit the eager call's."""
    x = torch.randn(70, 2048, device="cuda", dtype=BF16)
    w = torch.randn(2048, 512, device="cuda") / 45
    wq, ws_ = quantize(w, 2048, 512, "tiles")
    md = moe.matmul_desc(70, 512, 2048)
    back = moe.matmul_desc(70, 2048, 512, moe.MOE_B_NK)
    grad = moe.matmul_desc(2048, 512, 80, moe.MOE_B_NK_ROWS, moe.MOE_F32)

    def new():
        e = lambda *s, t=U8: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        return {"q": e(70, 2048), "qs": e(70, 16, t=F32), "y": e(70, 512, t=BF16), "yq": e(70, 512), "ys": e(70, 4, t=F32),
                "dx": e(70, 2048, t=BF16), "xt": e(2048, 80), "xts": e(2048, 1, t=F32), "yt": e(512, 80), "yts": e(512, 1, t=F32),
                "dw": e(2048, 512, t=F32), "ws": workspace(max(moe.moe_fp8_matmul_workspace_bytes(d) for d in (md, back, grad)))}

    def step(o):
        moe.moe_fp8_quantize(x, 70, 2048, moe.MOE_BLOCK_ROWS, o["q"], o["qs"])
        moe.moe_fp8_matmul(md, o["q"], o["qs"], wq, ws_, None, o["y"], o["ws"])
        moe.moe_fp8_quantize(o["y"], 70, 512, moe.MOE_BLOCK_ROWS, o["yq"], o["ys"])
        moe.moe_fp8_matmul(back, o["yq"], o["ys"], wq, ws_, None, o["dx"], o["ws"])
        moe.moe_fp8_quantize(x, 70, 2048, moe.MOE_BLOCK_TOKENS, o["xt"], o["xts"])
        moe.moe_fp8_quantize(o["y"], 70, 512, moe.MOE_BLOCK_TOKENS, o["yt"], o["yts"])
        moe.moe_fp8_matmul(grad, o["xt"], o["xts"], o["yt"], o["yts"], None, o["dw"], o["ws"])

    ref = new()
    step(ref)
    torch.cuda.synchronize()

    def same(o):
        torch.cuda.synchronize()
        for n in ref:
            if n != "ws":
                assert torch.equal(ref[n].view(U8), o[n].view(U8)), n
            o[n].zero_() if n != "ws" else o[n].fill_(0xA5)

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
    # the gradient of the weights against the 64-bit one of the same quantised values
    xv = values(ref["xt"].view(F8), ref["xts"])
    yv = values(ref["yt"].view(F8), ref["yts"])
    got, want, size = f64(ref["dw"]), f64(xv @ yv.t().contiguous()), f64(xv.abs() @ yv.abs().t().contiguous())
    assert (np.abs(got - want) <= size * 130 * 2.0 ** -23 + np.abs(want) * 2.0 ** -24).all()
