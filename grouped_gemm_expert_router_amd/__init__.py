"""Python binding of libmoe.so, the MI355X dropless MoE layer (see include/moe.h).

Argument marshalling only: every step of the layer runs in the library's HIP kernels.  PyTorch
provides device memory and the current HIP stream.  Importing this package does not need a GPU;
calling an entry point without the built library raises (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_BF16, MOE_FP8_E4M3, MOE_MXFP8, MOE_F32 = 0, 1, 2, 3
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3
MOE_STATE_F32, MOE_STATE_8BIT = 0, 1
MOE_WS_ROUTE, MOE_WS_FORWARD, MOE_WS_BACKWARD, MOE_WS_ROUTER = 0, 1, 2, 3
MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_WORKSPACE, MOE_ERR_HIP, MOE_ERR_ALIGN = 0, -1, -2, -3, -4, -5, -6

ENTRY_POINTS = ("moe_workspace_bytes", "moe_saved_bytes", "moe_route", "moe_route_noalloc", "moe_plan",
                "moe_forward", "moe_forward_fused", "moe_backward", "moe_router_logits", "moe_router_backward",
                "moe_permute", "moe_combine", "moe_mxfp8_quantize", "moe_mxfp8_quantize_weights",
                "moe_balance_workspace_bytes", "moe_balance_forward", "moe_balance_backward",
                "moe_norm_workspace_bytes", "moe_norm_forward", "moe_norm_backward",
                "moe_grad_norm_workspace_bytes", "moe_grad_norm", "moe_adamw_step", "moe_set_stage_hook",
                "moe_status_string")


class MoeDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("f", ctypes.c_int64), ("E", ctypes.c_int64),
                ("k", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def __repr__(self):
        return f"MoeDims(T={self.T}, d={self.d}, f={self.f}, E={self.E}, k={self.k}, dtype={self.dtype})"


class MoeNormDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("h_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("reserved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("out_scale", ctypes.c_float)]


class MoeTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "m_scale", "v_scale", "master")] + [
        ("n", ctypes.c_int64), ("p_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32), ("state", ctypes.c_int32),
        ("weight_decay", ctypes.c_float)]


class MoeAdamW(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps")] + [
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint64), ("stochastic", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("d_lr", ctypes.c_void_p), ("d_step", ctypes.c_void_p),
        ("d_grad_scale", ctypes.c_void_p)]


# void hook(const char* stage, int begin, void* stream, void* user)
STAGE_HOOK = ctypes.CFUNCTYPE(None, ctypes.c_char_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed with status {status}: {text}")
        self.status = status


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmoe.so (built in-tree by grouped_gemm_expert_router_amd.build)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m grouped_gemm_expert_router_amd.build`")
    lib = ctypes.CDLL(p)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    dp = ctypes.POINTER(MoeDims)
    lib.moe_workspace_bytes.argtypes = [dp, i32, ctypes.POINTER(sz)]
    lib.moe_saved_bytes.argtypes = [dp, ctypes.POINTER(sz)]
    lib.moe_route.argtypes = [dp] + [vp] * 8 + [sz, vp]
    lib.moe_route_noalloc.argtypes = [dp] + [vp] * 7 + [vp]
    lib.moe_plan.argtypes = [dp] + [vp] * 6 + [sz, vp]
    lib.moe_forward.argtypes = [dp] + [vp] * 13 + [sz, vp]
    lib.moe_forward_fused.argtypes = [dp] + [vp] * 10 + [sz, vp]
    lib.moe_backward.argtypes = [dp] + [vp] * 19 + [sz, vp]
    lib.moe_router_logits.argtypes = [dp, vp, vp, vp, vp]
    lib.moe_router_backward.argtypes = [dp] + [vp] * 6 + [sz, vp]
    lib.moe_permute.argtypes = [dp, vp, vp, vp, vp]
    lib.moe_combine.argtypes = [dp, vp, vp, vp, vp]
    lib.moe_mxfp8_quantize.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, i32, vp, vp, vp]
    lib.moe_mxfp8_quantize_weights.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64] + [vp] * 5
    i64, szp = ctypes.c_int64, ctypes.POINTER(sz)
    np_, tp, ap = ctypes.POINTER(MoeNormDesc), ctypes.POINTER(MoeTensor), ctypes.POINTER(MoeAdamW)
    lib.moe_balance_workspace_bytes.argtypes = [dp, i64, szp]
    lib.moe_balance_forward.argtypes = [dp] + [vp] * 4 + [i64] + [vp] * 5 + [sz, vp]
    lib.moe_balance_backward.argtypes = [dp] + [vp] * 3 + [i64] + [vp] * 5 + [vp]
    lib.moe_norm_workspace_bytes.argtypes = [np_, szp]
    lib.moe_norm_forward.argtypes = [np_] + [vp] * 7 + [vp]
    lib.moe_norm_backward.argtypes = [np_] + [vp] * 13 + [sz, vp]
    lib.moe_grad_norm_workspace_bytes.argtypes = [tp, i64, szp]
    lib.moe_grad_norm.argtypes = [tp, i64, ctypes.c_float, vp, vp, vp, sz, vp]
    lib.moe_adamw_step.argtypes = [ap, tp, i64, vp]
    lib.moe_set_stage_hook.argtypes = [STAGE_HOOK, vp]
    lib.moe_status_string.argtypes = [i32]
    lib.moe_status_string.restype = ctypes.c_char_p
    for name in ENTRY_POINTS[:-1]:
        getattr(lib, name).restype = i32
    if path is None:
        _lib = lib
    return lib


def dims(T: int, d: int, f: int, E: int, k: int, dtype: int = MOE_BF16) -> MoeDims:
    return MoeDims(T, d, f, E, k, dtype, 0)


def _ptr(t) -> Optional[int]:
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


_torch = None  # (handle of a device's current stream, current device), once they are needed


def _torch_calls():
    global _torch
    if _torch is None:
        import torch
        torch.cuda.current_device()  # sets up the runtime
        # not public: where they are missing, the public calls behind them
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        _torch = (raw or (lambda index: torch.cuda.current_stream(index).cuda_stream), device or torch.cuda.current_device)
    return _torch


def _stream(stream) -> Optional[int]:
    """A stream's handle; None is torch's current stream of the current device.  The handle is taken
    from torch directly: a torch.cuda.Stream object around it costs 2.8 us, most of a small call."""
    if stream is None:
        raw, device = _torch or _torch_calls()
        return raw(device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoEError(fn, rc, load_library().moe_status_string(rc).decode())


def _elsewhere(fn: str, t):
    raise ValueError(f"{fn}: tensors on {t.device}, not on the current GPU")


def _device() -> Optional[int]:
    """torch's current device, None without a GPU."""
    if _torch is None:
        import torch
        if not torch.cuda.is_available():
            return None
    return _torch_calls()[1]()


def _arguments(fn: str, stream, tensors: tuple) -> list:
    """Addresses of a call's tensors (None and plain addresses stay) and the stream's handle.  Refuses a tensor
    that is not on the current device: the kernels go to a stream of that one, and would fault on the host's
    memory.  A small call's time is the host's, so no step here is more than that needs."""
    here = _torch[1]() if _torch is not None else _device()
    try:
        a = [None if t is None else t.data_ptr() if t.get_device() == here else _elsewhere(fn, t) for t in tensors]
    except AttributeError:   # a plain address among them
        a = [t if t is None or isinstance(t, int) else t.data_ptr() if t.get_device() == here else _elsewhere(fn, t)
             for t in tensors]
    a.append(_stream(stream) if stream is not None or here is None else _torch[0](here))
    return a


def status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def moe_workspace_bytes(dm: MoeDims, which: int) -> int:
    out = ctypes.c_size_t(0)
    _check("moe_workspace_bytes", load_library().moe_workspace_bytes(ctypes.byref(dm), which, ctypes.byref(out)))
    return out.value


def moe_saved_bytes(dm: MoeDims) -> int:
    out = ctypes.c_size_t(0)
    _check("moe_saved_bytes", load_library().moe_saved_bytes(ctypes.byref(dm), ctypes.byref(out)))
    return out.value


def moe_route(dm, logits, topk_ids, topk_w, counts, offsets, perm, inv_perm, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("moe_route", load_library().moe_route(
        ctypes.byref(dm), _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(perm),
        _ptr(inv_perm), _ptr(ws), nb, _stream(stream)))


def moe_route_noalloc(dm, logits, topk_ids, topk_w, counts, offsets, perm, inv_perm, stream=None):
    _check("moe_route_noalloc", load_library().moe_route_noalloc(
        ctypes.byref(dm), _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(perm),
        _ptr(inv_perm), _stream(stream)))


def moe_plan(dm, topk_ids, counts, offsets, perm, inv_perm, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("moe_plan", load_library().moe_plan(
        ctypes.byref(dm), _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv_perm), _ptr(ws), nb,
        _stream(stream)))


def moe_forward(dm, x, x_scale, W1, W1_scale, W2, W2_scale, topk_w, offsets, perm, inv_perm, y, saved, ws,
                ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("moe_forward", load_library().moe_forward(
        ctypes.byref(dm), _ptr(x), _ptr(x_scale), _ptr(W1), _ptr(W1_scale), _ptr(W2), _ptr(W2_scale), _ptr(topk_w),
        _ptr(offsets), _ptr(perm), _ptr(inv_perm), _ptr(y), _ptr(saved), _ptr(ws), nb, _stream(stream)))


def moe_forward_fused(dm, x, W1, W2, topk_w, offsets, perm, inv_perm, y, saved, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("moe_forward_fused", load_library().moe_forward_fused(
        ctypes.byref(dm), _ptr(x), _ptr(W1), _ptr(W2), _ptr(topk_w), _ptr(offsets), _ptr(perm), _ptr(inv_perm),
        _ptr(y), _ptr(saved), _ptr(ws), nb, _stream(stream)))


def moe_backward(dm, dy, x, x_scale, W1, W1_scale, W2, W2_scale, topk_ids, topk_w, offsets, perm, inv_perm, saved,
                 dx, dW1, dW2, d_topk_w, d_logits, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check("moe_backward", load_library().moe_backward(
        ctypes.byref(dm), _ptr(dy), _ptr(x), _ptr(x_scale), _ptr(W1), _ptr(W1_scale), _ptr(W2), _ptr(W2_scale),
        _ptr(topk_ids), _ptr(topk_w), _ptr(offsets), _ptr(perm), _ptr(inv_perm), _ptr(saved), _ptr(dx), _ptr(dW1),
        _ptr(dW2), _ptr(d_topk_w), _ptr(d_logits), _ptr(ws), nb, _stream(stream)))


def moe_router_logits(dm, x, Wg, logits, stream=None):
    _check("moe_router_logits", load_library().moe_router_logits(ctypes.byref(dm), _ptr(x), _ptr(Wg), _ptr(logits),
                                                                 _stream(stream)))


def moe_router_backward(dm, x, Wg, d_logits, dx, dWg, ws, ws_bytes=None, stream=None):
    nb = (ws.numel() * ws.element_size() if ws is not None else 0) if ws_bytes is None else ws_bytes
    _check("moe_router_backward", load_library().moe_router_backward(
        ctypes.byref(dm), _ptr(x), _ptr(Wg), _ptr(d_logits), _ptr(dx), _ptr(dWg), _ptr(ws), nb, _stream(stream)))


def moe_permute(dm, x, inv_perm, xp, stream=None):
    _check("moe_permute", load_library().moe_permute(ctypes.byref(dm), _ptr(x), _ptr(inv_perm), _ptr(xp),
                                                     _stream(stream)))


def moe_combine(dm, op, inv_perm, y, stream=None):
    _check("moe_combine", load_library().moe_combine(ctypes.byref(dm), _ptr(op), _ptr(inv_perm), _ptr(y),
                                                     _stream(stream)))


def moe_mxfp8_quantize(src, batch, rows, cols, block_axis, codes, exps, stream=None):
    _check("moe_mxfp8_quantize", load_library().moe_mxfp8_quantize(_ptr(src), batch, rows, cols, block_axis,
                                                                   _ptr(codes), _ptr(exps), _stream(stream)))


def moe_mxfp8_quantize_weights(src, batch, rows, cols, col_codes, col_exps, row_codes, row_words, stream=None):
    _check("moe_mxfp8_quantize_weights",
           load_library().moe_mxfp8_quantize_weights(_ptr(src), batch, rows, cols, _ptr(col_codes), _ptr(col_exps),
                                                     _ptr(row_codes), _ptr(row_words), _stream(stream)))


def moe_balance_workspace_bytes(dm: MoeDims, S: int) -> int:
    out = ctypes.c_size_t(0)
    _check("moe_balance_workspace_bytes",
           load_library().moe_balance_workspace_bytes(ctypes.byref(dm), S, ctypes.byref(out)))
    return out.value


def moe_balance_forward(dm, logits, topk_ids, token_mask, group_offsets, S, counts, group_tokens, losses, lse, ws,
                        ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    a = _arguments("moe_balance_forward", stream, (logits, topk_ids, token_mask, group_offsets, counts, group_tokens,
                                                   losses, lse, ws))
    a.insert(4, S)
    a.insert(-1, nb)
    _check("moe_balance_forward", load_library().moe_balance_forward(dm, *a))


def moe_balance_backward(dm, logits, lse, group_offsets, S, counts, group_tokens, d_losses, d_logits_in, d_logits,
                         stream=None):
    a = _arguments("moe_balance_backward", stream, (logits, lse, group_offsets, counts, group_tokens, d_losses,
                                                    d_logits_in, d_logits))
    a.insert(3, S)
    _check("moe_balance_backward", load_library().moe_balance_backward(dm, *a))


def norm_desc(T: int, d: int, h_dtype: int = MOE_BF16, w_dtype: int = MOE_BF16, gate: int = MOE_GATE_NONE,
              eps: float = 1e-6, res_scale: float = 1.0, out_scale: float = 1.0) -> MoeNormDesc:
    return MoeNormDesc(T, d, h_dtype, w_dtype, gate, 0, eps, res_scale, out_scale)


def moe_norm_workspace_bytes(nd: MoeNormDesc) -> int:
    out = ctypes.c_size_t(0)
    _check("moe_norm_workspace_bytes", load_library().moe_norm_workspace_bytes(ctypes.byref(nd), ctypes.byref(out)))
    return out.value


def moe_norm_forward(nd, y, h, w_post, gate, w_pre, h_out, x, stream=None):
    a = _arguments("moe_norm_forward", stream, (y, h, w_post, gate, w_pre, h_out, x))
    _check("moe_norm_forward", load_library().moe_norm_forward(nd, *a))


def moe_norm_backward(nd, y, h_out, w_post, gate, w_pre, dh_out, dx, dh, dy, dw_post, dgate, dw_pre, ws,
                      ws_bytes=None, stream=None):
    nb = (ws.numel() * ws.element_size() if ws is not None else 0) if ws_bytes is None else ws_bytes
    a = _arguments("moe_norm_backward", stream, (y, h_out, w_post, gate, w_pre, dh_out, dx, dh, dy, dw_post, dgate, dw_pre, ws))
    a.insert(-1, nb)
    _check("moe_norm_backward", load_library().moe_norm_backward(nd, *a))


class TensorList:
    """A host array of moe_tensor and the torch tensors it points to, which it keeps alive."""

    def __init__(self, rows):
        self.rows = list(rows)
        self.first = self.rows[0][1][0] if self.rows else None
        if any(keep[0].device != self.first.device for _, keep in self.rows):
            raise ValueError("adamw_tensors: tensors on more than one device")
        self.array = (MoeTensor * max(len(self.rows), 1))(*(r for r, _ in self.rows))

    def __len__(self):
        return len(self.rows)


def adamw_tensor(g, p=None, m=None, v=None, master=None, m_scale=None, v_scale=None, weight_decay: float = 0.0):
    """One row for adamw_tensors(): torch tensors of one parameter, its gradient and its states.  m and
    v with scales (float8_e4m3fn or uint8) are 8-bit states.  moe_grad_norm needs g alone."""
    import torch
    f32, types = torch.float32, {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
    n = g.numel()
    eight = m_scale is not None or v_scale is not None
    state = (torch.float8_e4m3fn, torch.uint8) if eight else (f32,)
    device = g.device

    def check(name, t, size, allowed):
        if t is None:
            return None
        if t.dtype not in allowed or t.numel() != size or not t.is_contiguous() or t.device != device:
            raise ValueError(f"adamw_tensor: {name} is {tuple(t.shape)} {t.dtype} on {t.device}, expected {size} "
                             f"contiguous values on {device} of {sorted(map(str, allowed))}")
        return t.data_ptr()

    blocks = (n + 255) // 256
    row = MoeTensor(check("p", p, n, types), check("g", g, n, types), check("m", m, n, state), check("v", v, n, state),
                    check("m_scale", m_scale, blocks, (f32,)), check("v_scale", v_scale, blocks, (f32,)),
                    check("master", master, n, (f32,)), n, types[p.dtype] if p is not None else MOE_F32,
                    types[g.dtype], MOE_STATE_8BIT if eight else MOE_STATE_F32, weight_decay)
    return row, (g, p, m, v, master, m_scale, v_scale)


def adamw_tensors(rows) -> TensorList:
    """The list that moe_grad_norm and moe_adamw_step take, from adamw_tensor() rows."""
    return TensorList(rows)


def adamw_hyper(lr: float, beta1: float = 0.9, beta2: float = 0.95, eps: float = 1e-8, step: int = 1, seed: int = 0,
                stochastic: bool = False, d_lr=None, d_step=None, d_grad_scale=None) -> MoeAdamW:
    hyper = MoeAdamW(lr, beta1, beta2, eps, step, seed, int(stochastic), 0, _ptr(d_lr), _ptr(d_step),
                     _ptr(d_grad_scale))
    hyper.keep = (d_lr, d_step, d_grad_scale)  # alive as long as their addresses are
    return hyper


def moe_grad_norm_workspace_bytes(tensors: TensorList) -> int:
    out = ctypes.c_size_t(0)
    _check("moe_grad_norm_workspace_bytes",
           load_library().moe_grad_norm_workspace_bytes(tensors.array, len(tensors), ctypes.byref(out)))
    return out.value


def moe_grad_norm(tensors: TensorList, max_norm, norm, scale, ws, ws_bytes=None, stream=None):
    nb = (ws.numel() * ws.element_size() if ws is not None else 0) if ws_bytes is None else ws_bytes
    _, *a = _arguments("moe_grad_norm", stream, (tensors.first, norm, scale, ws))   # the list is on its first's device
    a.insert(-1, nb)
    _check("moe_grad_norm", load_library().moe_grad_norm(tensors.array, len(tensors), max_norm, *a))


def moe_adamw_step(hyper: MoeAdamW, tensors: TensorList, stream=None):
    here = _device()
    for t in (tensors.first, *getattr(hyper, "keep", ())):
        if t is not None and not isinstance(t, int) and t.get_device() != here:
            _elsewhere("moe_adamw_step", t)
    _check("moe_adamw_step", load_library().moe_adamw_step(hyper, tensors.array, len(tensors), _stream(stream)))


_hook_ref = None


def moe_set_stage_hook(fn) -> None:
    """Install fn(stage: str, begin: bool, stream_ptr: int) as the library's profiling hook
    (None removes it).  The ctypes callback object is kept alive here."""
    global _hook_ref
    if fn is None:
        _hook_ref = None
        _check("moe_set_stage_hook", load_library().moe_set_stage_hook(STAGE_HOOK(), None))
        return

    def tramp(stage, begin, stream, user):
        fn(stage.decode(), bool(begin), stream or 0)

    _hook_ref = STAGE_HOOK(tramp)
    _check("moe_set_stage_hook", load_library().moe_set_stage_hook(_hook_ref, None))


# ------------------------------------------------------------------ buffer helpers (torch)
def alloc_layer_buffers(dm: MoeDims, device="cuda", backward: bool = True) -> dict:
    """Device buffers for one route/plan -> forward (-> backward) round, sized by the library."""
    import torch
    T, d, f, E, k = dm.T, dm.d, dm.f, dm.E, dm.k
    A = T * k
    i32 = dict(dtype=torch.int32, device=device)
    b = {
        "topk_ids": torch.empty((T, k), **i32),
        "topk_w": torch.empty((T, k), dtype=torch.float32, device=device),
        "counts": torch.empty((E,), **i32),
        "offsets": torch.empty((E + 1,), **i32),
        "perm": torch.empty((max(A, 1),), **i32),
        "inv_perm": torch.empty((max(A, 1),), **i32),
        "ws_route": torch.empty((max(moe_workspace_bytes(dm, MOE_WS_ROUTE), 256),), dtype=torch.uint8, device=device),
        "y": torch.empty((T, d), dtype=torch.bfloat16, device=device),
        "saved": torch.empty((max(moe_saved_bytes(dm), 256),), dtype=torch.uint8, device=device),
        "ws_fwd": torch.empty((max(moe_workspace_bytes(dm, MOE_WS_FORWARD), 256),), dtype=torch.uint8, device=device),
    }
    if backward:
        b.update({
            "dx": torch.empty((T, d), dtype=torch.bfloat16, device=device),
            "dW1": torch.empty((E, d, 2 * f), dtype=torch.bfloat16, device=device),
            "dW2": torch.empty((E, f, d), dtype=torch.bfloat16, device=device),
            "d_topk_w": torch.empty((T, k), dtype=torch.float32, device=device),
            "d_logits": torch.empty((T, E), dtype=torch.float32, device=device),
            "ws_bwd": torch.empty((max(moe_workspace_bytes(dm, MOE_WS_BACKWARD), 256),), dtype=torch.uint8,
                                  device=device),
        })
    return b


__all__ = ["MoeDims", "MoEError", "dims", "load_library", "status_string", "moe_workspace_bytes", "moe_saved_bytes",
           "moe_route", "moe_route_noalloc", "moe_plan", "moe_forward", "moe_forward_fused", "moe_backward",
           "moe_router_logits",
           "moe_router_backward", "moe_permute", "moe_combine",
           "moe_mxfp8_quantize", "moe_mxfp8_quantize_weights", "moe_set_stage_hook", "alloc_layer_buffers",
           "moe_balance_workspace_bytes", "moe_balance_forward", "moe_balance_backward", "MoeNormDesc", "norm_desc",
           "moe_norm_workspace_bytes", "moe_norm_forward", "moe_norm_backward", "MoeTensor", "MoeAdamW", "TensorList",
           "adamw_tensor", "adamw_tensors", "adamw_hyper", "moe_grad_norm_workspace_bytes", "moe_grad_norm",
           "moe_adamw_step", "MOE_F32", "MOE_GATE_NONE", "MOE_GATE_CHANNEL", "MOE_GATE_TOKEN", "MOE_GATE_FULL",
           "MOE_STATE_F32", "MOE_STATE_8BIT",
           "ENTRY_POINTS", "MOE_BF16",
           "MOE_FP8_E4M3", "MOE_MXFP8", "MOE_WS_ROUTE", "MOE_WS_FORWARD",
           "MOE_WS_BACKWARD", "MOE_WS_ROUTER", "MOE_OK", "MOE_ERR_NULL", "MOE_ERR_SHAPE", "MOE_ERR_DTYPE", "MOE_ERR_WORKSPACE",
           "MOE_ERR_HIP", "MOE_ERR_ALIGN"]
