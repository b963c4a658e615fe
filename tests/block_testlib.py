"""Shared helpers of the tests of the training step around the layer: tensors to and from the
device and the elementwise comparison against a 64-bit value with a bound of its own."""
from __future__ import annotations

import numpy as np
import torch

import grouped_gemm_expert_router_amd as moe

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative to the value
MOE_TYPE = {torch.bfloat16: moe.MOE_BF16, torch.float32: moe.MOE_F32}
GUARD = 64   # values around every output that have to stay as they were


def dev(a, dtype=torch.float32, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(device)


def f64(t):
    """The device values, exactly, in fp64 (None stays None)."""
    return None if t is None else t.detach().double().cpu().numpy()


class Guarded:
    """An output buffer filled with a pattern between two guard bands."""

    def __init__(self, shape, dtype, device="cuda", fill=7.0):
        n = int(np.prod(shape))
        self.whole = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device=device)
        self.t = self.whole[GUARD:GUARD + n].view(shape)
        self.fill = fill

    def check(self):
        w = self.whole
        assert torch.all(w[:GUARD] == self.fill) and torch.all(w[-GUARD:] == self.fill), "written outside the output"
        return self.t


def assert_close(name, got, ref, bound):
    """|got - ref| <= bound for every element; non-finite values equal."""
    got, ref = f64(got).reshape(-1), np.asarray(ref, np.float64).reshape(-1)
    bound = np.broadcast_to(np.asarray(bound, np.float64), np.shape(bound)).reshape(-1)
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(got)), f"{name}: non-finite values differ"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), name
    over = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)) - bound, 0)
    if over.size and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{name}[{i}]: {got[i]} is not {ref[i]} within {bound[i]} ({(over > 0).sum()} of {got.size})")


def workspace(n, device="cuda"):
    return torch.full((max(int(n), 256),), 0xA5, dtype=torch.uint8, device=device)
