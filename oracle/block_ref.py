"""Plain fp64 CPU oracle of the training step around the routed layer.

TEST INFRASTRUCTURE ONLY (as ``moe_ref``): the gate's balance and z losses with their gradient,
the RMS norms before and after the block with gate and residual, the gradient norm and AdamW with
fp32 or 8-bit states.  Plain numpy in fp64, loops over groups and rows of tokens.

Conventions: ``gate`` is None, or ("channel" [d] | "token" [T] | "full" [T, d], values).
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_to_f64


# ------------------------------------------------------------------ balance loss
def _counted(logits, mask, offsets):
    """Each token's group, -1 where it does not count."""
    T = logits.shape[0]
    group = np.full(T, -1, np.int64)
    for g, (a, z) in enumerate(zip(offsets[:-1], offsets[1:])):
        group[a:z] = g
    for t in range(T):
        # a NaN is not -inf: its token counts
        if (mask is not None and mask[t] == 0) or np.all(logits[t] == -np.inf):
            group[t] = -1
    return group


def balance(logits, ids, mask=None, offsets=None):
    """losses [2], counts [S, E], tokens [S+2], lse [T], p [T, E] (zeros where a token does not count)."""
    T, E = logits.shape
    k = ids.shape[1]
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    S = len(offsets) - 1
    group = _counted(logits, mask, offsets)
    lse, p = np.full(T, -np.inf), np.zeros((T, E))
    counts, P, n = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    z = 0.0
    for t in np.flatnonzero(group >= 0):
        x = logits[t].astype(np.float64)
        top = x.max()
        e = np.exp(x - top)
        lse[t] = top + np.log(e.sum())
        p[t] = e / e.sum()
        g = group[t]
        n[g] += 1
        P[g] += p[t]
        z += lse[t] ** 2
        for e in ids[t]:
            if 0 <= e < E:
                counts[g, e] += 1
    full = np.flatnonzero(n)
    terms = [E / (k * float(n[g]) ** 2) * float((counts[g] * P[g]).sum()) for g in full]
    losses = np.array([np.mean(terms) if len(full) else 0.0, z / n.sum() if n.sum() else 0.0])
    return dict(losses=losses, counts=counts, tokens=np.concatenate([n, [n.sum(), len(full)]]), lse=lse, p=p,
                group=group)


def balance_grad(b, k, d_losses, d_in=None):
    """d_logits of d_losses . losses plus d_in, and a bound on what fp32 terms it is a sum of."""
    p, counts, tokens = b["p"], b["counts"].astype(np.float64), b["tokens"]
    T, E = p.shape
    d = np.zeros((T, E)) if d_in is None else d_in.astype(np.float64).copy()
    size = np.abs(d)
    G, N = tokens[-1], tokens[-2]
    for t in np.flatnonzero(b["group"] >= 0):
        g = b["group"][t]
        a = d_losses[0] * E / (k * float(tokens[g]) ** 2 * G)
        c = counts[g] - k * tokens[g] // E
        z = 2 * d_losses[1] * b["lse"][t] / N
        d[t] += p[t] * (a * (c - (c * p[t]).sum()) + z)
        size[t] += p[t] * (abs(a) * (np.abs(c) + (np.abs(c) * p[t]).sum()) + abs(z))
    return d, size


# ------------------------------------------------------------------ norms around a block
def _gate(gate, T, d):
    if gate is None:
        return np.ones((1, 1))
    kind, v = gate
    return {"channel": lambda: v.reshape(1, d), "token": lambda: v.reshape(T, 1), "full": lambda: v.reshape(T, d)}[kind]()


def norm_forward(h, y=None, w_post=None, gate=None, w_pre=None, eps=1e-6, res_scale=1.0, out_scale=1.0):
    """h_out (None without y), x (None without w_pre)."""
    T, d = h.shape
    out = h
    if y is not None:
        n = y if w_post is None else w_post * y / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        out = res_scale * h + out_scale * _gate(gate, T, d) * n
    x = None if w_pre is None else w_pre * out / np.sqrt((out * out).mean(1, keepdims=True) + eps)
    return (None if y is None else out), x


def norm_backward(dh_out, h_out=None, y=None, w_post=None, gate=None, w_pre=None, dx=None, eps=1e-6, res_scale=1.0,
                  out_scale=1.0):
    """Gradients by name, and under the same names the sizes of the terms each is a sum of."""
    T, d = (y if y is not None else h_out).shape
    D = np.zeros((T, d)) if dh_out is None else dh_out
    sD = np.abs(D)
    g, s = {}, {}
    if w_pre is not None:
        sp = 1 / np.sqrt((h_out * h_out).mean(1, keepdims=True) + eps)
        hh, t = h_out * sp, w_pre * dx
        D = D + sp * (t - hh * (hh * t).mean(1, keepdims=True))
        sD = sD + sp * (np.abs(t) + np.abs(hh) * np.abs(hh * t).mean(1, keepdims=True))
        g["dw_pre"], s["dw_pre"] = (dx * hh).sum(0), np.abs(dx * hh).sum(0)
    r = res_scale if y is not None else 1.0
    g["dh"], s["dh"] = r * D, abs(r) * sD
    if y is None:
        return g, s
    sq = np.ones((T, 1)) if w_post is None else 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    w = np.ones((1, d)) if w_post is None else w_post
    yh, G = y * sq, out_scale * _gate(gate, T, d)
    if gate is not None:
        each, size = out_scale * D * (w * yh), abs(out_scale) * sD * np.abs(w * yh)
        axis = {"channel": 0, "token": 1, "full": None}[gate[0]]
        g["dgate"], s["dgate"] = (each, size) if axis is None else (each.sum(axis), size.sum(axis))
    dn, sn = G * D, np.abs(G) * sD
    if w_post is None:
        g["dy"], s["dy"] = dn, sn
        return g, s
    g["dw_post"], s["dw_post"] = (dn * yh).sum(0), (sn * np.abs(yh)).sum(0)
    g["dy"] = sq * (w * dn - yh * (yh * w * dn).mean(1, keepdims=True))
    s["dy"] = sq * (np.abs(w) * sn + np.abs(yh) * (np.abs(yh * w) * sn).mean(1, keepdims=True))
    return g, s


# ------------------------------------------------------------------ optimiser
BLOCK = 256


def adamw(w, g, m, v, lr, beta1, beta2, eps, step, weight_decay=0.0, grad_scale=1.0):
    """New (w, m, v) of one tensor, fp64."""
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mean, var = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return w - lr * weight_decay * w - lr * mean / (np.sqrt(var) + eps), m, v


def grad_norm(gs, max_norm):
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in gs))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def decode_state(codes, scales):
    """Values of an 8-bit state: code times its block's scale."""
    return e4m3_to_f64(codes) * np.repeat(scales.astype(np.float64), BLOCK)[:codes.size]


def noise(seed, step, tensor, n):
    """The two 32-bit words of each of n values (integers only, so the GPU's are the same)."""
    M = (1 << 64) - 1
    z = ((seed ^ (step << 32) ^ tensor) + 0x9E3779B97F4A7C15) & M
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & M
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & M
    z ^= z >> 31
    k0, k1 = np.uint32(z & 0xFFFFFFFF), np.uint32(z >> 32)
    u = np.arange(n, dtype=np.uint32) ^ k0
    u = (u ^ (u >> np.uint32(16))) * np.uint32(0x32A0CD0B)
    u = (u ^ (u >> np.uint32(14)) ^ k1) * np.uint32(0x2F37D463)
    u = u ^ (u >> np.uint32(16))
    w = (u ^ k0) * np.uint32(0xBB67AE85)
    return u, w ^ (w >> np.uint32(15))


def e4m3_below(y):
    """The e4m3 value at or below y >= 0 and the step to the next code (448 has none: step 0)."""
    y = np.asarray(y, np.float64)
    e = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
    step = np.exp2(np.maximum(e, -6) - 3)
    low = np.floor(y / step) * step
    return np.minimum(low, 448.0), np.where(low >= 448, 0.0, step)
