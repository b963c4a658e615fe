"""Pins of oracle.block_ref: closed forms, central differences, torch's own AdamW, the rounding's
expectation and the random words' spread."""
import numpy as np
import pytest
import torch

from oracle import block_ref as R
from oracle import e4m3_to_f64


def _rng(seed):
    return np.random.default_rng(seed)


def _topk(logits, k):
    return np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)


def test_balance_is_one_for_an_even_load():
    # every expert takes the same share of slots and of probability
    E, k, T = 4, 1, 8
    logits = np.zeros((T, E), np.float32)
    ids = (np.arange(T) % E).astype(np.int32)[:, None]
    b = R.balance(logits, ids)
    assert abs(b["losses"][0] - 1) < 1e-12
    assert abs(b["losses"][1] - np.log(E) ** 2) < 1e-12
    # all tokens on one expert with certainty: the loss is E
    logits = np.full((T, E), -np.inf, np.float32)
    logits[:, 2] = 3.0
    b = R.balance(logits, np.full((T, 1), 2, np.int32))
    assert abs(b["losses"][0] - E) < 1e-12 and abs(b["losses"][1] - 9) < 1e-12


def test_balance_leaves_out_what_does_not_count():
    rng = _rng(1)
    T, E, k = 23, 6, 2
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids = _topk(logits, k)
    mask = (rng.random(T) > 0.3).astype(np.uint8)
    offsets = np.array([2, 9, 9, 20])
    logits[mask == 0] = np.nan
    logits[10] = -np.inf
    b = R.balance(logits, ids, mask, offsets)
    keep = [t for t in range(2, 20) if mask[t] and t != 10]
    assert b["tokens"].tolist() == [sum(t < 9 for t in keep), 0, sum(t >= 9 for t in keep), len(keep), 2]
    assert b["counts"].sum() == k * len(keep) and not b["counts"][1].any()
    assert np.all((b["lse"] > -np.inf) == np.isin(np.arange(T), keep))
    # each group on its own, as a batch of its own
    one = [R.balance(logits[[t for t in keep if lo <= t < hi]], ids[[t for t in keep if lo <= t < hi]])
           for lo, hi in ((2, 9), (9, 20))]
    assert abs(b["losses"][0] - np.mean([o["losses"][0] for o in one])) < 1e-12


def test_balance_gradient_by_differences():
    rng = _rng(2)
    T, E, k = 9, 5, 2
    logits = rng.standard_normal((T, E))
    ids = _topk(logits, k)
    mask = np.array([1, 1, 0, 1, 1, 1, 1, 1, 1], np.uint8)
    offsets = np.array([1, 5, 9])
    w = np.array([0.7, -0.3])
    d, size = R.balance_grad(R.balance(logits, ids, mask, offsets), k, w, d_in=np.ones((T, E)))
    h = 1e-5
    for t in range(T):
        for e in range(E):
            a, b = logits.copy(), logits.copy()
            a[t, e] += h
            b[t, e] -= h
            diff = w @ (R.balance(a, ids, mask, offsets)["losses"] - R.balance(b, ids, mask, offsets)["losses"]) / (2 * h)
            assert abs(d[t, e] - 1 - diff) < 1e-8
    assert np.all(np.abs(d) <= size * (1 + 1e-12))


GATES = [None, "channel", "token", "full"]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (None, True)])
def test_norm_gradients_by_differences(gate, post, pre):
    """post None: no block output at all (the norm before a block alone)."""
    if post is None and gate is not None:
        return
    rng = _rng(3)
    T, d = 4, 8
    v = {"h": rng.standard_normal((T, d))}
    if post is not None:
        v["y"] = rng.standard_normal((T, d))
        if post:
            v["w_post"] = rng.standard_normal(d)
        if gate:
            v["gate"] = rng.standard_normal({"channel": d, "token": T, "full": (T, d)}[gate])
    if pre:
        v["w_pre"] = rng.standard_normal(d)
    kw = dict(eps=0.1, res_scale=0.8, out_scale=1.3)
    ch, cx = rng.standard_normal((T, d)), rng.standard_normal((T, d))

    def value(v):
        out, x = R.norm_forward(v["h"], v.get("y"), v.get("w_post"), (gate, v["gate"]) if gate else None, v.get("w_pre"), **kw)
        out = v["h"] if out is None else out
        return (out * ch).sum() + (0 if x is None else (x * cx).sum())

    out, _ = R.norm_forward(v["h"], v.get("y"), v.get("w_post"), (gate, v["gate"]) if gate else None, v.get("w_pre"), **kw)
    g, s = R.norm_backward(ch, v["h"] if out is None else out, v.get("y"), v.get("w_post"),
                           (gate, v["gate"]) if gate else None, v.get("w_pre"), cx if pre else None, **kw)
    h = 1e-6
    for name, grad in (("h", "dh"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate"), ("w_pre", "dw_pre")):
        if name not in v:
            assert grad not in g
            continue
        for i in np.ndindex(v[name].shape):
            a, b = dict(v), dict(v)
            a[name], b[name] = v[name].copy(), v[name].copy()
            a[name][i] += h
            b[name][i] -= h
            assert abs(g[grad][i] - (value(a) - value(b)) / (2 * h)) < 2e-8 * max(1, s[grad][i])
        assert np.all(np.abs(g[grad]) <= s[grad] * (1 + 1e-12))


def test_adamw_is_torchs():
    rng = _rng(4)
    w = torch.tensor(rng.standard_normal(50))
    p = w.clone().requires_grad_()
    opt = torch.optim.AdamW([p], lr=0.02, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    x, m, v = w.numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 5):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        x, m, v = R.adamw(x, 2 * g, m, v, 0.02, 0.9, 0.95, 1e-6, step, weight_decay=0.1, grad_scale=0.5)
        assert np.abs(x - p.detach().numpy()).max() < 1e-14


def test_grad_norm_is_torchs():
    rng = _rng(5)
    gs = [rng.standard_normal(n) for n in (1, 7, 300)]
    ps = [torch.zeros(len(g), dtype=torch.float64, requires_grad=True) for g in gs]
    for p, g in zip(ps, gs):
        p.grad = torch.tensor(g)
    norm, scale = R.grad_norm(gs, 2.0)
    assert abs(float(torch.nn.utils.clip_grad_norm_(ps, 2.0)) - norm) < 1e-12
    assert abs(float(ps[2].grad[0]) / gs[2][0] - scale) < 1e-12
    assert R.grad_norm(gs, 1e6)[1] == 1.0


def test_e4m3_below_against_every_code():
    table = np.sort(e4m3_to_f64(np.arange(0x7F, dtype=np.uint8)))
    y = np.concatenate([table, (table[1:] + table[:-1]) / 2, table[1:] * (1 - 1e-9)])
    low, step = R.e4m3_below(y)
    i = np.searchsorted(table, y, side="right") - 1
    assert np.array_equal(low, table[i])
    inner = i < len(table) - 1
    assert np.array_equal(step[inner], (table[1:] - table[:-1])[i[inner]]) and np.all(step[~inner] == 0)


def test_noise_words_are_spread():
    """Sixteen bits at a time: even over 256 bins, no drift along neighbours, unlike for another step,
    seed or tensor."""
    n = 1 << 20
    a, b = R.noise(99, 7, 3, n)
    words = [a & 0xFFFF, a >> 16, b & 0xFFFF]
    for w in words:
        u = w / 65536.0
        assert abs(u.mean() - 0.5) < 5 / np.sqrt(12 * n)
        hist = np.histogram(u, 256, (0, 1))[0]
        chi = ((hist - n / 256) ** 2 / (n / 256)).sum()
        assert abs(chi - 255) < 6 * np.sqrt(2 * 255)
        for lag in (1, 2, 4, 64, 256, 4096):
            assert abs(np.corrcoef(u[:-lag], u[lag:])[0, 1]) < 0.01
    for other in (R.noise(99, 8, 3, n)[0], R.noise(98, 7, 3, n)[0], R.noise(99, 7, 4, n)[0]):
        assert abs(np.corrcoef(words[0], other & 0xFFFF)[0, 1]) < 0.01
    for x, y in ((0, 1), (0, 2), (1, 2)):
        assert abs(np.corrcoef(words[x], words[y])[0, 1]) < 0.01
