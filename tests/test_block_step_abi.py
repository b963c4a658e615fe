"""Refusals of the balance loss, norm, gradient norm and AdamW calls: every host-side check returns
its code without launching anything (no GPU needed)."""
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


def size(fn, *a):
    out = ctypes.c_size_t(0)
    return fn(*a, ctypes.byref(out)), out.value


# ------------------------------------------------------------------ balance
def bal_fwd(lib, dm, over=None, S=2, nb=1 << 40):
    a = dict(logits=F, ids=F, mask=F, goff=F, counts=F, tokens=F, losses=F, lse=F, ws=F)
    a.update(over or {})
    return lib.moe_balance_forward(ctypes.byref(dm), a["logits"], a["ids"], a["mask"], a["goff"], S, a["counts"],
                                   a["tokens"], a["losses"], a["lse"], a["ws"], nb, None)


def bal_bwd(lib, dm, over=None, S=2):
    a = dict(logits=F, lse=F, goff=F, counts=F, tokens=F, w=F, d_in=F, d=F)
    a.update(over or {})
    return lib.moe_balance_backward(ctypes.byref(dm), a["logits"], a["lse"], a["goff"], S, a["counts"], a["tokens"],
                                    a["w"], a["d_in"], a["d"], None)


def test_balance_refusals(lib):
    dm = moe.dims(64, 128, 128, 8, 2)
    rc, need = size(lib.moe_balance_workspace_bytes, ctypes.byref(dm), 2)
    assert rc == 0 and need > 0 and need % 256 == 0
    for S in (0, -1, 65536):
        assert size(lib.moe_balance_workspace_bytes, ctypes.byref(dm), S)[0] == moe.MOE_ERR_SHAPE
        assert bal_fwd(lib, dm, S=S) == bal_bwd(lib, dm, S=S) == moe.MOE_ERR_SHAPE
    assert lib.moe_balance_workspace_bytes(ctypes.byref(dm), 1, None) == moe.MOE_ERR_NULL
    assert bal_fwd(lib, moe.dims(64, 128, 128, 8, 9)) == moe.MOE_ERR_SHAPE
    assert bal_fwd(lib, moe.dims(-1, 128, 128, 8, 2)) == moe.MOE_ERR_SHAPE
    for name in ("logits", "ids", "goff", "counts", "tokens", "losses", "lse", "ws"):
        assert bal_fwd(lib, dm, {name: None}) == moe.MOE_ERR_NULL, name
    for name in ("logits", "lse", "goff", "counts", "tokens", "w", "d"):
        assert bal_bwd(lib, dm, {name: None}) == moe.MOE_ERR_NULL, name
    assert bal_fwd(lib, dm, nb=need - 1) == moe.MOE_ERR_WORKSPACE
    for name, off in (("logits", 4), ("ids", 4), ("counts", 8), ("lse", 4), ("goff", 2), ("tokens", 1), ("losses", 2), ("ws", 16)):
        assert bal_fwd(lib, dm, {name: F + off}) == moe.MOE_ERR_ALIGN, name
    for name, off in (("logits", 4), ("d_in", 4), ("d", 8), ("counts", 4), ("lse", 8), ("w", 2), ("goff", 1), ("tokens", 2)):
        assert bal_bwd(lib, dm, {name: F + off}) == moe.MOE_ERR_ALIGN, name
    assert bal_bwd(lib, moe.dims(0, 128, 128, 8, 2), dict(logits=None, d=None)) == moe.MOE_OK   # nothing to add


def test_fp32_is_no_type_of_the_layer(lib):
    dm = moe.dims(64, 256, 256, 8, 2, moe.MOE_F32)
    assert size(lib.moe_workspace_bytes, ctypes.byref(dm), moe.MOE_WS_FORWARD)[0] == moe.MOE_ERR_DTYPE
    assert size(lib.moe_balance_workspace_bytes, ctypes.byref(dm), 1)[0] == moe.MOE_ERR_DTYPE


def test_balance_workspace_is_bounded(lib):
    big = lambda T, S, E=256: size(lib.moe_balance_workspace_bytes, ctypes.byref(moe.dims(T, 128, 128, E, 1)), S)[1]  # noqa: E731
    assert big(1 << 19, 1) == big(1 << 16, 1)                 # 1024 tiles
    assert big(1 << 15, 64) > big(1 << 15, 1)
    assert big((1 << 31) - 1, 1, 8) <= (1 << 16) * (8 * 8 + 8) + 8192   # 65536 tiles at most


# ------------------------------------------------------------------ norms
def nfwd(lib, nd, over=None):
    a = dict(y=F, h=F, w_post=F, gate=None, w_pre=F, h_out=F, x=F)
    a.update(over or {})
    return lib.moe_norm_forward(ctypes.byref(nd), a["y"], a["h"], a["w_post"], a["gate"], a["w_pre"], a["h_out"], a["x"], None)


def nbwd(lib, nd, over=None, nb=1 << 40):
    a = dict(y=F, h_out=F, w_post=F, gate=None, w_pre=F, dh_out=F, dx=F, dh=F, dy=F, dw_post=F, dgate=None, dw_pre=F, ws=F)
    a.update(over or {})
    return lib.moe_norm_backward(ctypes.byref(nd), *(a[n] for n in ("y", "h_out", "w_post", "gate", "w_pre", "dh_out", "dx",
                                                                     "dh", "dy", "dw_post", "dgate", "dw_pre", "ws")), nb, None)


def test_norm_shapes_and_types(lib):
    ok = moe.norm_desc(4, 64)
    assert size(lib.moe_norm_workspace_bytes, ctypes.byref(ok))[0] == 0
    bad = [moe.norm_desc(4, 0), moe.norm_desc(4, 4), moe.norm_desc(4, 100), moe.norm_desc(4, 16392), moe.norm_desc(-1, 64),
           moe.norm_desc(1 << 31, 64), moe.norm_desc(1 << 30, 2048), moe.norm_desc(4, 64, gate=4), moe.norm_desc(4, 64, gate=-1),
           moe.norm_desc(4, 64, eps=0.0), moe.norm_desc(4, 64, eps=-1e-6), moe.norm_desc(4, 64, eps=NAN),
           moe.norm_desc(4, 64, eps=INF), moe.norm_desc(4, 64, res_scale=INF), moe.norm_desc(4, 64, out_scale=NAN)]
    r = moe.norm_desc(4, 64)
    r.reserved = 1
    for nd in bad + [r]:
        assert size(lib.moe_norm_workspace_bytes, ctypes.byref(nd))[0] == moe.MOE_ERR_SHAPE
        assert nfwd(lib, nd) == nbwd(lib, nd) == moe.MOE_ERR_SHAPE
    for nd in (moe.norm_desc(4, 64, h_dtype=1), moe.norm_desc(4, 64, w_dtype=2), moe.norm_desc(4, 64, h_dtype=9)):
        assert nfwd(lib, nd) == nbwd(lib, nd) == moe.MOE_ERR_DTYPE
    assert lib.moe_norm_forward(None, F, F, F, None, F, F, F, None) == moe.MOE_ERR_NULL
    assert lib.moe_norm_workspace_bytes(ctypes.byref(ok), None) == moe.MOE_ERR_NULL


def test_norm_argument_errors(lib):
    nd, gated = moe.norm_desc(4, 64), moe.norm_desc(4, 64, gate=moe.MOE_GATE_TOKEN)
    assert nfwd(lib, nd, dict(h=None)) == moe.MOE_ERR_NULL
    assert nfwd(lib, nd, dict(h_out=None)) == moe.MOE_ERR_NULL
    assert nfwd(lib, nd, dict(x=None)) == nfwd(lib, nd, dict(w_pre=None)) == moe.MOE_ERR_NULL
    assert nfwd(lib, nd, dict(y=None)) == moe.MOE_ERR_SHAPE          # the part behind a block without its output
    assert nfwd(lib, nd, dict(y=None, w_post=None)) == moe.MOE_ERR_SHAPE
    assert nfwd(lib, gated, dict(y=None, w_post=None, h_out=None)) == moe.MOE_ERR_SHAPE
    assert nfwd(lib, nd, dict(y=None, w_post=None, h_out=None, w_pre=None, x=None)) == moe.MOE_ERR_NULL   # nothing to do
    assert nfwd(lib, gated) == moe.MOE_ERR_NULL
    assert nfwd(lib, nd, dict(gate=F)) == moe.MOE_ERR_NULL
    for name in ("y", "h", "w_post", "w_pre", "h_out", "x"):
        assert nfwd(lib, nd, {name: F + 8}) == moe.MOE_ERR_ALIGN, name
    assert nfwd(lib, gated, dict(gate=F + 2)) == moe.MOE_ERR_ALIGN
    assert nbwd(lib, nd, dict(h_out=None)) == nbwd(lib, nd, dict(dx=None)) == moe.MOE_ERR_NULL
    assert nbwd(lib, nd, dict(w_pre=None)) == moe.MOE_ERR_SHAPE
    assert nbwd(lib, nd, dict(w_pre=None, h_out=None, dx=None, dw_pre=None, dh_out=None)) == moe.MOE_ERR_NULL   # no gradient
    assert nbwd(lib, nd, dict(y=None)) == moe.MOE_ERR_SHAPE
    assert nbwd(lib, nd, dict(w_post=None)) == moe.MOE_ERR_NULL       # a gradient of a weight that is not there
    assert nbwd(lib, gated) == moe.MOE_ERR_NULL
    assert nbwd(lib, nd, dict(dgate=F)) == moe.MOE_ERR_NULL
    rc, need = size(lib.moe_norm_workspace_bytes, ctypes.byref(nd))
    assert need > 0 and nbwd(lib, nd, nb=need - 1) == moe.MOE_ERR_WORKSPACE
    assert nbwd(lib, nd, dict(ws=None)) == moe.MOE_ERR_NULL
    assert nbwd(lib, nd, dict(ws=F + 16)) == moe.MOE_ERR_ALIGN
    for name in ("y", "h_out", "w_post", "w_pre", "dh_out", "dx", "dh", "dy", "dw_post", "dw_pre"):
        assert nbwd(lib, nd, {name: F + 4}) == moe.MOE_ERR_ALIGN, name


# ------------------------------------------------------------------ optimiser
def tensor(**over):
    a = dict(p=F, g=F, m=F, v=F, m_scale=None, v_scale=None, master=None, n=100, p_dtype=moe.MOE_F32,
             g_dtype=moe.MOE_F32, state=moe.MOE_STATE_F32, weight_decay=0.0)
    a.update(over)
    return moe.MoeTensor(*a.values())


def adam(lib, hp=None, tensors=None, n=None):
    ts = [tensor()] if tensors is None else tensors
    arr = (moe.MoeTensor * max(len(ts), 1))(*ts)
    return lib.moe_adamw_step(ctypes.byref(hp or moe.adamw_hyper(1e-3)), arr, len(ts) if n is None else n, None)


EIGHT = dict(state=moe.MOE_STATE_8BIT, m_scale=F, v_scale=F)


def test_adamw_hyper_refusals(lib):
    for kw in (dict(lr=-1.0), dict(lr=NAN), dict(lr=INF), dict(lr=1e39), dict(beta1=1.0), dict(beta1=-0.1),
               dict(beta2=1.0 - 1e-12), dict(beta2=NAN), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-60), dict(eps=1e-40), dict(eps=INF),
               dict(step=0), dict(step=-5)):
        a = dict(lr=1e-3)
        a.update(kw)
        assert adam(lib, moe.adamw_hyper(**a)) == moe.MOE_ERR_SHAPE, kw
    hp = moe.adamw_hyper(1e-3)
    hp.reserved = 1
    assert adam(lib, hp) == moe.MOE_ERR_SHAPE
    hp = moe.adamw_hyper(1e-3)
    hp.stochastic = 2
    assert adam(lib, hp) == moe.MOE_ERR_SHAPE
    for kw in (dict(d_lr=F + 2), dict(d_step=F + 4), dict(d_grad_scale=F + 1)):
        assert adam(lib, moe.adamw_hyper(1e-3, **kw)) == moe.MOE_ERR_ALIGN, kw
    assert lib.moe_adamw_step(None, None, 0, None) == moe.MOE_ERR_NULL
    assert adam(lib, n=-1) == moe.MOE_ERR_SHAPE
    assert lib.moe_adamw_step(ctypes.byref(moe.adamw_hyper(1e-3)), None, 1, None) == moe.MOE_ERR_NULL
    assert adam(lib, tensors=[]) == moe.MOE_OK                       # an empty list
    assert adam(lib, tensors=[tensor(n=0, p=None, g=None, m=None, v=None)]) == moe.MOE_OK


def test_adamw_tensor_refusals(lib):
    E = moe
    cases = [(dict(n=-1), E.MOE_ERR_SHAPE), (dict(n=(1 << 40) + 1), E.MOE_ERR_SHAPE), (dict(weight_decay=-0.1), E.MOE_ERR_SHAPE),
             (dict(weight_decay=NAN), E.MOE_ERR_SHAPE), (dict(p=None), E.MOE_ERR_NULL), (dict(g=None), E.MOE_ERR_NULL),
             (dict(m=None), E.MOE_ERR_NULL), (dict(v=None), E.MOE_ERR_NULL), (dict(p_dtype=1), E.MOE_ERR_DTYPE),
             (dict(g_dtype=2), E.MOE_ERR_DTYPE), (dict(state=2), E.MOE_ERR_DTYPE), (dict(master=F), E.MOE_ERR_DTYPE),
             (dict(m_scale=F), E.MOE_ERR_DTYPE), (dict(EIGHT, m_scale=None), E.MOE_ERR_NULL),
             (dict(EIGHT, v_scale=None), E.MOE_ERR_NULL), (dict(EIGHT, v_scale=F + 2), E.MOE_ERR_ALIGN),
             (dict(p=F + 4), E.MOE_ERR_ALIGN), (dict(g=F + 2), E.MOE_ERR_ALIGN), (dict(m=F + 8), E.MOE_ERR_ALIGN),
             (dict(v=F + 1), E.MOE_ERR_ALIGN), (dict(p_dtype=0, master=F + 4), E.MOE_ERR_ALIGN)]
    for over, code in cases:
        assert adam(lib, tensors=[tensor(), tensor(**over)]) == code, over
    for over, code in cases[:1] + [(dict(g=None), E.MOE_ERR_NULL), (dict(g_dtype=1), E.MOE_ERR_DTYPE), (dict(g=F + 4), E.MOE_ERR_ALIGN)]:
        arr = (moe.MoeTensor * 1)(tensor(**over))
        assert size(lib.moe_grad_norm_workspace_bytes, arr, 1)[0] == code
        assert lib.moe_grad_norm(arr, 1, 1.0, F, F, F, 1 << 30, None) == code


def test_grad_norm_refusals(lib):
    arr = (moe.MoeTensor * 1)(tensor(p=None, m=None, v=None, n=1 << 20))
    rc, need = size(lib.moe_grad_norm_workspace_bytes, arr, 1)
    assert rc == 0 and need > 0
    for m in (0.0, -1.0, NAN, INF):
        assert lib.moe_grad_norm(arr, 1, m, F, F, F, need, None) == moe.MOE_ERR_SHAPE
    assert lib.moe_grad_norm(arr, 1, 1.0, None, F, F, need, None) == moe.MOE_ERR_NULL
    assert lib.moe_grad_norm(arr, 1, 1.0, F, F, None, need, None) == moe.MOE_ERR_NULL
    assert lib.moe_grad_norm(arr, 1, 1.0, F, F, F, need - 1, None) == moe.MOE_ERR_WORKSPACE
    assert lib.moe_grad_norm(arr, 1, 1.0, F + 2, F, F, need, None) == moe.MOE_ERR_ALIGN
    assert lib.moe_grad_norm(arr, 1, 1.0, F, F + 1, F, need, None) == moe.MOE_ERR_ALIGN
    assert lib.moe_grad_norm(arr, 1, 1.0, F, F, F + 8, need, None) == moe.MOE_ERR_ALIGN
    assert lib.moe_grad_norm(arr, -1, 1.0, F, F, F, need, None) == moe.MOE_ERR_SHAPE
    assert lib.moe_grad_norm_workspace_bytes(arr, 1, None) == moe.MOE_ERR_NULL


def test_adamw_tensor_checks_torch_tensors():
    z = lambda n, t=torch.float32: torch.zeros(n, dtype=t)  # noqa: E731
    row, _ = moe.adamw_tensor(z(300, torch.bfloat16), z(300, torch.bfloat16), z(300, torch.float8_e4m3fn),
                              z(300, torch.uint8), z(300), z(2), z(2), 0.1)
    assert row.n == 300 and row.p_dtype == row.g_dtype == moe.MOE_BF16 and row.state == moe.MOE_STATE_8BIT
    row, _ = moe.adamw_tensor(z(10))
    assert row.g_dtype == moe.MOE_F32 and row.state == moe.MOE_STATE_F32 and not row.p
    for kw in (dict(p=z(9)), dict(p=z(20)[::2]), dict(p=z(10, torch.float16)), dict(p=z(10), m=z(10, torch.bfloat16)),
               dict(p=z(10), master=z(10, torch.bfloat16)), dict(p=z(10), m=z(10), v=z(10), m_scale=z(1)),
               dict(p=z(10), m=z(10, torch.uint8), m_scale=z(2), v_scale=z(1))):
        with pytest.raises(ValueError):
            moe.adamw_tensor(z(10), **kw)
    with pytest.raises(ValueError):
        moe.adamw_tensor(z(10, torch.float16))


def test_tensors_of_another_device_are_refused():
    z = torch.zeros(64)
    nd, dm = moe.norm_desc(1, 64, moe.MOE_F32, moe.MOE_F32), moe.dims(8, 128, 128, 8, 2)
    tl = moe.adamw_tensors([moe.adamw_tensor(z, z, z, z)])
    for call in (lambda: moe.moe_norm_forward(nd, None, z, None, None, z, None, z),
                 lambda: moe.moe_norm_backward(nd, None, z, None, None, z, z, z, z, None, None, None, z, z),
                 lambda: moe.moe_balance_forward(dm, z, z, None, None, 1, z, z, z, z, z),
                 lambda: moe.moe_balance_backward(dm, z, z, None, 1, z, z, z, None, z),
                 lambda: moe.moe_grad_norm(tl, 1.0, z, None, z), lambda: moe.moe_adamw_step(moe.adamw_hyper(1e-3), tl)):
        with pytest.raises(ValueError, match="not on the current GPU"):
            call()
    with pytest.raises(ValueError, match="more than one device"):
        moe.adamw_tensors([moe.adamw_tensor(z), moe.adamw_tensor(torch.zeros(3, device="meta"))])
