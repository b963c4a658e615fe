"""The blockwise e4m3 quantiser and product at the ends of their documented ranges: the longest K, the widest N, the tallest
M, strides of 2^31 values, and scales from one end of fp32 to the other.  Operands are zeros but for a few places, so that
results are exact and the reference is small."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from block_testlib import Guarded, workspace
from test_gpu_fp8_dense import B_FORMS, FORMS, operands, product, quantize, values

pytestmark = pytest.mark.gpu
BF16, F32, U8, F8 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn
ONE = 0x38   # the code of 1


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


@pytest.mark.parametrize("form", sorted(B_FORMS))
@pytest.mark.parametrize("M", [3, 40, 70, 300])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_longest_k(form, M, dtype):
    """K = 2^24: whole numbers at 600 places of K, others zero; every sum is exact."""
    N, K = 32, 1 << 24
    print(f"[case] product {form} {M}x{N}x{K}", flush=True)
    gen = torch.Generator("cuda").manual_seed(M)
    at = torch.randint(0, K, (600,), generator=gen, device="cuda").unique()
    at[0], at[-1] = 0, K - 1
    a, b = torch.zeros(M, K, dtype=U8, device="cuda"), torch.zeros((K, N) if form == "kn" else (N, K), dtype=U8, device="cuda")
    av = torch.randint(-3, 4, (M, at.numel()), generator=gen, device="cuda").float()
    bv = torch.randint(-3, 4, (at.numel(), N), generator=gen, device="cuda").float()
    a[:, at] = av.to(F8).view(U8)
    if form == "kn":
        b[at] = bv.to(F8).view(U8)
    else:
        b[:, at] = bv.t().contiguous().to(F8).view(U8)
    KB = K // 128
    sa = torch.exp2(torch.randint(-2, 3, (M, KB), generator=gen, device="cuda").float())
    shape = {"kn": (KB, 1), "nk": (1, KB), "rows": (N, KB)}[form]
    sb = torch.exp2(torch.randint(-2, 3, shape, generator=gen, device="cuda").float())
    got = product(M, N, K, form, dtype, a.view(F8), sa, b.view(F8), sb)
    bs = sb[at // 128].expand(-1, N) if form == "kn" else sb[:, at // 128].expand(N, -1).t()
    ref = (av * sa[:, at // 128]).double() @ (bv * bs).double().contiguous()
    assert torch.equal(got, ref.to(F32).to(dtype))


@pytest.mark.parametrize("form", sorted(B_FORMS))
@pytest.mark.parametrize("M", [2, 33, 100])
def test_widest_n(form, M):
    """N = 2^24: columns far apart have their own values, the rest are zero."""
    room(40)
    N, K = 1 << 24, 48
    print(f"[case] product {form} {M}x{N}x{K}", flush=True)
    gen = torch.Generator("cuda").manual_seed(M)
    cols = torch.tensor([0, 1, 127, 128, (1 << 23) - 1, 1 << 23, N - 129, N - 16, N - 1], device="cuda")
    a, sa, _, _ = operands(M, 16, K, form, M, True)
    bv = torch.randint(-3, 4, (K, cols.numel()), generator=gen, device="cuda").float()
    b = torch.zeros((K, N) if form == "kn" else (N, K), dtype=U8, device="cuda")
    if form == "kn":
        b[:, cols] = bv.to(F8).view(U8)
    else:
        b[cols] = bv.t().contiguous().to(F8).view(U8)
    sb = torch.exp2(torch.randint(-2, 3, (N if form == "rows" else N // 128,), generator=gen, device="cuda").float())
    c = Guarded((M, N), BF16)
    md = moe.matmul_desc(M, N, K, B_FORMS[form], moe.MOE_BF16)
    moe.moe_fp8_matmul(md, a, sa, b, sb.view(1, -1) if form == "kn" else sb.view(-1, 1), None, c.t,
                       workspace(moe.moe_fp8_matmul_workspace_bytes(md)))
    torch.cuda.synchronize()
    got = c.check()
    ref = values(a, sa) @ (bv * (sb[cols] if form == "rows" else sb[cols // 128])).double()
    assert torch.equal(got[:, cols], ref.to(F32).to(BF16))
    assert int((got != 0).sum()) == int((got[:, cols] != 0).sum())


@pytest.mark.parametrize("form", sorted(B_FORMS))
def test_tallest_m(form):
    """M = 2^30: rows far apart have values, the rest are zero."""
    room(120)
    M, N, K = 1 << 30, 16, 16
    print(f"[case] product {form} {M}x{N}x{K}", flush=True)
    rows = torch.tensor([0, 1, 255, 256, (1 << 27) + 5, 1 << 28, (1 << 29) - 1, M - 257, M - 1], device="cuda")
    a, sa = torch.zeros(M, K, dtype=U8, device="cuda"), torch.ones(M, 1, device="cuda")
    a[rows] = ONE
    sa[rows, 0] = torch.exp2(torch.arange(rows.numel(), device="cuda").float())
    b, sb = torch.full((N, K), ONE, dtype=U8, device="cuda"), torch.ones(N if form == "rows" else 1, 1, device="cuda")
    c = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    md = moe.matmul_desc(M, N, K, B_FORMS[form])
    moe.moe_fp8_matmul(md, a, sa, b, sb, None, c, workspace(moe.moe_fp8_matmul_workspace_bytes(md)))
    torch.cuda.synchronize()
    assert torch.equal(c[rows], (16 * sa[rows]).expand(-1, N).to(BF16))
    seen = sum(int(torch.count_nonzero(c[i:i + (1 << 27)])) for i in range(0, M, 1 << 27))
    assert seen == rows.numel() * N


@pytest.mark.parametrize("shape", [(1 << 24, 1008), (1008, 1 << 24)], ids=["tall", "wide"])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_largest_source(shape, form):
    """Nearly 2^34 values, 34 GB; ones in the first and last rows and columns."""
    room(130)
    rows, cols = shape
    print(f"[case] quantize {shape} {form}", flush=True)
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[0, 0] = x[-1, -1] = x[rows // 2 + 1, 5] = 2.0
    codes, scales = quantize(x, rows, cols, form)
    if form == "tokens":
        codes, scales = codes.t(), scales.t()
    c = rows // 2 + 1
    for i, j in ((0, 0), (rows - 1, cols - 1), (c, 5)):
        si, sj = {"rows": (i, j // 128), "tokens": (i // 128, j), "tiles": (i // 128, j // 128)}[form]
        assert int(codes[i, j]) == 0x7E and float(scales[si, sj]) == float(np.float32(2) / np.float32(448))
    n = sum(int(torch.count_nonzero(p)) for p in torch.chunk(codes, 16, int(cols > rows)))
    assert n == 3 and int((scales != 1).sum()) == 3


def test_longest_stride_of_a_source():
    room(30)
    ld, rows, cols = 1 << 31, 3, 272
    wide = torch.empty((rows - 1) * ld + cols, dtype=BF16, device="cuda")
    x = torch.randn(rows, cols, device="cuda").to(BF16)
    torch.as_strided(wide, (rows, cols), (ld, 1)).copy_(x)
    for form in FORMS:
        got, want = quantize(wide, rows, cols, form, ld), quantize(x, rows, cols, form)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("form", sorted(B_FORMS))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_scales_from_end_to_end(form, dtype):
    """Powers of two as scales whose products lie between 2^-120 and 2^100: exact where a row's blocks share one."""
    for M in (5, 40, 130):
        N, K = 144, 400
        a, sa, b, sb = operands(M, N, K, form, M, True)
        for ea, eb in ((-110, -10), (-10, -110), (-60, -60), (90, 10), (10, 90), (-120, 120), (100, -120)):
            ta, tb = torch.full_like(sa, 2.0 ** ea), torch.full_like(sb, 2.0 ** eb)
            got = product(M, N, K, form, dtype, a, ta, b, tb)
            bv = b.double() if form == "kn" else b.double().t().contiguous()
            assert torch.equal(got, (a.double() @ bv * 2.0 ** (ea + eb)).to(F32).to(dtype))
