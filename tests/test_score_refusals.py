"""Refusals of the scored routing, quantiser and product calls: every host-side check returns its code
without launching anything (no GPU needed)."""
import ctypes
import os

import pytest
import torch

import grouped_gemm_expert_router_amd as moe

F = 1 << 20   # a non-null, 256-aligned address that is never dereferenced on error paths
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return moe.load_library()


def size(fn, desc):
    out = ctypes.c_size_t(0)
    return fn(ctypes.byref(desc) if desc is not None else None, ctypes.byref(out)), out.value


ROUTE = ("logits", "bias", "mask", "ids", "w", "counts", "offsets", "perm", "inv", "ws")


def route(lib, sd, over=None, nb=1 << 40):
    a = dict.fromkeys(ROUTE, F) | (over or {})
    return lib.moe_score_route(ctypes.byref(sd), *[a[n] for n in ROUTE], nb, None)


def back(lib, sd, over=None):
    a = dict(logits=F, ids=F, d_w=F, d=F) | (over or {})
    return lib.moe_score_backward(ctypes.byref(sd), a["logits"], a["ids"], a["d_w"], a["d"], None)


def changed(sd, **over):
    for n, v in over.items():
        setattr(sd, n, v)
    return sd


def test_score_desc_refusals(lib):
    make = lambda **o: changed(moe.score_desc(64, 32, 4, groups=4, group_topk=2, group_best=2), **o)  # noqa: E731
    rc, need = size(lib.moe_score_workspace_bytes, make())
    assert rc == 0 and need > 0 and need % 256 == 0
    bad = [dict(T=-1), dict(T=1 << 31), dict(T=1 << 30), dict(E=0), dict(E=1025), dict(E=30), dict(k=0), dict(k=33),
           dict(k=17), dict(k=65, E=128), dict(score=2), dict(score=-1), dict(renormalise=2), dict(renormalise=-1),
           dict(groups=0), dict(groups=65, E=650), dict(groups=3), dict(group_topk=0), dict(group_topk=5), dict(group_best=0),
           dict(group_best=3), dict(scale=NAN), dict(scale=INF), dict(reserved=1)]
    for over in bad:
        sd = make(**over)
        assert size(lib.moe_score_workspace_bytes, sd)[0] == moe.MOE_ERR_SHAPE, over
        assert route(lib, sd) == back(lib, sd) == moe.MOE_ERR_SHAPE, over
    assert size(lib.moe_score_workspace_bytes, None)[0] == moe.MOE_ERR_NULL
    assert lib.moe_score_workspace_bytes(ctypes.byref(make()), None) == moe.MOE_ERR_NULL


def test_score_pointer_refusals(lib):
    sd = moe.score_desc(64, 32, 4)
    need = size(lib.moe_score_workspace_bytes, sd)[1]
    for name in ROUTE:
        if name not in ("bias", "mask"):
            assert route(lib, sd, {name: None}) == moe.MOE_ERR_NULL, name
    assert route(lib, sd, nb=need - 1) == moe.MOE_ERR_WORKSPACE
    for name, off in dict(logits=4, bias=2, ids=2, w=1, counts=2, offsets=2, perm=2, inv=1, ws=16).items():
        assert route(lib, sd, {name: F + off}) == moe.MOE_ERR_ALIGN, name
    for name in ("logits", "ids", "d_w", "d"):
        assert back(lib, sd, {name: None}) == moe.MOE_ERR_NULL, name
    for name, off in dict(logits=8, ids=2, d_w=2, d=4).items():
        assert back(lib, sd, {name: F + off}) == moe.MOE_ERR_ALIGN, name
    none = moe.score_desc(0, 32, 4)
    assert back(lib, none, dict(logits=None, d=None)) == moe.MOE_OK
    assert route(lib, none, dict(counts=None)) == moe.MOE_ERR_NULL


def test_bias_update_refusals(lib):
    call = lambda E=8, counts=F, rate=1e-3, bias=F, out=F: lib.moe_bias_update(E, counts, rate, bias, out, None)  # noqa: E731
    for over in (dict(E=0), dict(E=-1), dict(E=1025), dict(rate=NAN), dict(rate=INF)):
        assert call(**over) == moe.MOE_ERR_SHAPE, over
    for name in ("counts", "bias", "out"):
        assert call(**{name: None}) == moe.MOE_ERR_NULL
        assert call(**{name: F + 2}) == moe.MOE_ERR_ALIGN


def test_quantize_refusals(lib):
    def call(rows=8, cols=32, ld=32, form=0, dtype=moe.MOE_BF16, src=F, codes=F, scales=F):
        return lib.moe_fp8_quantize(src, dtype, rows, cols, ld, form, codes, scales, None)
    for dtype in (moe.MOE_FP8_E4M3, moe.MOE_MXFP8, -1, 4):
        assert call(dtype=dtype) == moe.MOE_ERR_DTYPE
    for over in (dict(form=-1), dict(form=3), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(cols=0), dict(cols=8), dict(cols=40),
                 dict(cols=-16), dict(cols=(1 << 24) + 16, ld=1 << 25), dict(rows=1 << 20, cols=1 << 14, ld=1 << 14),
                 dict(ld=24), dict(ld=36), dict(ld=(1 << 31) + 8)):
        assert call(**over) == moe.MOE_ERR_SHAPE, over
    for name in ("src", "codes", "scales"):
        assert call(**{name: None}) == moe.MOE_ERR_NULL, name
    for name, off in dict(src=8, codes=8, scales=2).items():
        assert call(**{name: F + off}) == moe.MOE_ERR_ALIGN, name
    assert call(rows=0, src=None) == moe.MOE_OK


MM = ("a", "sa", "b", "sb", "c_in", "c", "ws")


def mm(lib, md, over=None, nb=1 << 40):
    a = dict.fromkeys(MM, F) | (over or {})
    return lib.moe_fp8_matmul(ctypes.byref(md), *[a[n] for n in MM], nb, None)


def test_matmul_refusals(lib):
    make = lambda **o: changed(moe.matmul_desc(40, 64, 96), **o)  # noqa: E731
    bad = [dict(M=-1), dict(M=(1 << 30) + 1), dict(N=0), dict(N=8), dict(N=72), dict(N=(1 << 24) + 16, ldb=1 << 25, ldc=1 << 25),
           dict(K=0), dict(K=8), dict(K=100), dict(K=(1 << 24) + 16, lda=1 << 25), dict(M=1 << 30, N=64), dict(lda=80), dict(lda=104),
           dict(lda=(1 << 28) + 16), dict(ldb=48), dict(ldb=72), dict(ldb=(1 << 28) + 16), dict(ldc=56), dict(ldc=68), dict(ldc=1 << 32),
           dict(b_form=-1), dict(b_form=3), dict(b_form=moe.MOE_B_NK), dict(b_form=moe.MOE_B_NK_ROWS), dict(reserved=1)]
    for over in bad:   # the two forms [N, K] want ldb >= K = 96
        md = make(**over)
        assert size(lib.moe_fp8_matmul_workspace_bytes, md)[0] == mm(lib, md) == moe.MOE_ERR_SHAPE, over
    for t in (moe.MOE_FP8_E4M3, moe.MOE_MXFP8, 4, -1):
        assert size(lib.moe_fp8_matmul_workspace_bytes, make(c_dtype=t))[0] == mm(lib, make(c_dtype=t)) == moe.MOE_ERR_DTYPE
    assert size(lib.moe_fp8_matmul_workspace_bytes, None)[0] == moe.MOE_ERR_NULL
    for name in ("a", "sa", "b", "sb", "c"):
        assert mm(lib, make(), {name: None}) == moe.MOE_ERR_NULL, name
    for name, off in dict(a=8, sa=2, b=4, sb=1, c_in=8, c=4, ws=16).items():
        assert mm(lib, make(), {name: F + off}) == moe.MOE_ERR_ALIGN, name
    assert mm(lib, make(M=0), dict(a=None, c=None)) == moe.MOE_OK


def test_matmul_workspace(lib):
    """A workspace that is asked for has to be there and of its size."""
    seen = 0
    for M, N, K in ((1, 16, 16), (1, 2048, 7168), (16, 4096, 7168), (48, 7168, 2048), (700, 1024, 16384), (1 << 20, 4096, 4096)):
        for form in (moe.MOE_B_KN, moe.MOE_B_NK, moe.MOE_B_NK_ROWS):
            md = moe.matmul_desc(M, N, K, form)
            rc, need = size(lib.moe_fp8_matmul_workspace_bytes, md)
            assert rc == 0 and need % 256 == 0 and need <= 1 << 28, (M, N, K, form)
            if need:
                seen += 1
                assert mm(lib, md, dict(ws=None)) == moe.MOE_ERR_NULL
                assert mm(lib, md, nb=need - 1) == moe.MOE_ERR_WORKSPACE
    assert seen >= 6


class Elsewhere:
    """A tensor's look, as the binding sees it, on device `index` (-1: the host)."""

    def __init__(self, index):
        self.index, self.device = index, "cpu" if index < 0 else f"cuda:{index}"

    def get_device(self):
        return self.index

    def data_ptr(self):
        return F

    def numel(self):
        return 16

    def element_size(self):
        return 4


def places():
    """Calls by name: their tensors' names and the call with those."""
    sd, md = moe.score_desc(4, 16, 2), moe.matmul_desc(4, 16, 16)
    return {
        "moe_score_route": (ROUTE, lambda a: moe.moe_score_route(sd, *[a[n] for n in ROUTE])),
        "moe_score_backward": (("logits", "ids", "d_w", "d"),
                               lambda a: moe.moe_score_backward(sd, a["logits"], a["ids"], a["d_w"], a["d"])),
        "moe_bias_update": (("counts", "bias", "out"), lambda a: moe.moe_bias_update(a["counts"], 1e-3, a["bias"], a["out"])),
        "moe_fp8_quantize": (("src", "codes", "scales"),
                             lambda a: moe.moe_fp8_quantize(a["src"], 4, 16, 0, a["codes"], a["scales"], src_dtype=moe.MOE_F32)),
        "moe_fp8_matmul": (MM, lambda a: moe.moe_fp8_matmul(md, *[a[n] for n in MM])),
    }


@pytest.mark.parametrize("fn", sorted(places()))
def test_every_tensor_of_a_call_is_on_the_current_device(fn, monkeypatch):
    """A tensor in the host's memory or on another GPU, in any one place, is refused before the call; the
    same call with all of them on the current device goes through."""
    calls = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    lib = Recorder()
    monkeypatch.setattr(moe, "load_library", lambda: lib)
    monkeypatch.setattr(moe, "_torch", (lambda device: 0, lambda: 0))
    names, call = places()[fn]
    here = {n: Elsewhere(0) for n in names}
    call(here)
    assert calls == [fn]
    for n in names:
        for index in (-1, 1):
            with pytest.raises(ValueError, match="not on the current GPU"):
                call(dict(here, **{n: Elsewhere(index)}))
    assert calls == [fn]


def test_a_source_of_another_type_is_refused(lib):
    """The binding takes the type from the tensor; one that is neither bf16 nor fp32 is the library's to refuse."""
    if torch.cuda.is_available():
        pytest.skip("shown without a GPU")
    half = torch.zeros(4, 16, dtype=torch.float16)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_fp8_quantize(half.data_ptr(), 4, 16, 0, F, F, src_dtype=-1, stream=0)
    assert e.value.status == moe.MOE_ERR_DTYPE
