"""Calls of the training step that are refused before anything is launched (no GPU needed)."""
import ctypes
import os

import pytest

import grouped_gemm_expert_router_amd as moe

F = 1 << 20   # a non-null, 256-aligned address that is never dereferenced on error paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return moe.load_library()


def test_norm_backward_of_neither_part_is_refused(lib):
    """Neither the norm before a block (w_pre) nor the part behind it (y): there is nothing to go back
    through, whatever comes in and is asked for.  The forward call refuses it with the same code."""
    names = ("y", "h_out", "w_post", "gate", "w_pre", "dh_out", "dx", "dh", "dy", "dw_post", "dgate", "dw_pre")
    for T in (1, 4, 4096):
        nd = moe.norm_desc(T, 64)
        for given in ((), ("dh_out",), ("dh_out", "dh"), ("dh",)):
            a = [F if n in given else None for n in names]
            for ws, nb in ((F, 1 << 40), (None, 0)):
                assert lib.moe_norm_backward(ctypes.byref(nd), *a, ws, nb, None) == moe.MOE_ERR_NULL, given
        assert lib.moe_norm_forward(ctypes.byref(nd), None, F, None, None, None, None, None, None) == moe.MOE_ERR_NULL


class Elsewhere:
    """A tensor's look, as the binding sees it, on device `index` (-1: the host)."""

    def __init__(self, index):
        self.index, self.device = index, "cpu" if index < 0 else f"cuda:{index}"

    def get_device(self):
        return self.index

    def data_ptr(self):
        return F

    def numel(self):
        return 1 << 20

    def element_size(self):
        return 4


class Recorder:
    """Takes every call of the library and launches nothing."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append(name)
            return 0
        return call


def places():
    """Calls by name: the tensors' argument names and the call with those."""
    nd, dm = moe.norm_desc(4, 64, gate=moe.MOE_GATE_CHANNEL), moe.dims(8, 128, 128, 8, 2)

    def listed(first):
        rows = moe.TensorList([])
        rows.first = first
        return rows

    def adamw(a):
        hp = moe.adamw_hyper(1e-3, d_lr=a["d_lr"], d_step=a["d_step"], d_grad_scale=a["d_grad_scale"])
        moe.moe_adamw_step(hp, listed(a["first"]))

    def positional(fn, names, head=(), at=None, value=None):
        def call(a):
            args = [a[n] for n in names]
            if at is not None:
                args.insert(at, value)
            fn(*head, *args)
        return names, call

    return {
        "moe_balance_forward": positional(moe.moe_balance_forward, ("logits", "ids", "mask", "offsets", "counts", "tokens",
                                                                    "losses", "lse", "ws"), (dm,), 4, 3),
        "moe_balance_backward": positional(moe.moe_balance_backward, ("logits", "lse", "offsets", "counts", "tokens",
                                                                      "d_losses", "d_in", "d_out"), (dm,), 3, 3),
        "moe_norm_forward": positional(moe.moe_norm_forward, ("y", "h", "w_post", "gate", "w_pre", "h_out", "x"), (nd,)),
        "moe_norm_backward": positional(moe.moe_norm_backward, ("y", "h_out", "w_post", "gate", "w_pre", "dh_out", "dx", "dh",
                                                                "dy", "dw_post", "dgate", "dw_pre", "ws"), (nd,)),
        "moe_grad_norm": (("first", "norm", "scale", "ws"),
                          lambda a: moe.moe_grad_norm(listed(a["first"]), 1.0, a["norm"], a["scale"], a["ws"])),
        "moe_adamw_step": (("first", "d_lr", "d_step", "d_grad_scale"), adamw),
    }


@pytest.mark.parametrize("fn", ["moe_balance_forward", "moe_balance_backward", "moe_norm_forward", "moe_norm_backward",
                                "moe_grad_norm", "moe_adamw_step"])
def test_every_tensor_of_a_call_is_on_the_current_device(fn, monkeypatch):
    """A tensor in the host's memory or on another GPU, in any one place, is refused before the call; the
    same call with all of them on the current device goes through."""
    lib = Recorder()
    monkeypatch.setattr(moe, "load_library", lambda: lib)
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(moe, "_torch", (lambda device: 0, lambda: 0))
    names, call = places()[fn]
    here = {n: Elsewhere(0) for n in names}
    call(here)
    assert lib.calls == [fn]
    for n in names:
        for index in (-1, 1):
            with pytest.raises(ValueError, match="not on the current GPU"):
                call(dict(here, **{n: Elsewhere(index)}))
    assert lib.calls == [fn]
    monkeypatch.setattr(moe, "_torch", (lambda device: 0, lambda: 1))   # all of them on another than the current one
    with pytest.raises(ValueError, match="not on the current GPU"):
        call(here)
    assert lib.calls == [fn]


def test_stream_handles_come_from_the_public_call_where_there_is_no_raw_one(monkeypatch):
    """torch's raw handle and device functions are not public: without them the same come from
    torch.cuda's own calls."""
    import torch

    class Stream:
        def __init__(self, device):
            self.cuda_stream = 4096 + device

    monkeypatch.setattr(moe, "_torch", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(3 if device is None else device))
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    assert moe._stream(None) == 4099
    assert moe._device() in (None, 3)   # None: no GPU here
