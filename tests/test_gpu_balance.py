"""Balance loss, z-loss, counts and their gradient against the fp64 oracle.

Bounds.  p = exp(l - lse): the exponent's argument carries at most |l - top| 2^-24 from the
subtraction and 1.45 |l - top| 2^-24 from the product inside exp, |l - top| <= 32 in these inputs, and
exp2 is within 2 units: a relative error of 82 2^-24, the same for the sum of the exponentials and
half a unit for its reciprocal: p is within 2^-16 of itself.  lse: 2^-17 from the sum, plus two
roundings of numbers up to its parts' size: 2^-16 (1 + |top|).  Sums of p have positive terms:
at most 512 fp32 additions in a piece, 2^-15 with the terms' own.  The gradient is a sum of terms,
whose sizes the oracle adds up: each within 2^-15, d_in and the final rounding within 2^-23."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from oracle import block_ref as R
from block_testlib import Guarded, assert_close, dev, f64, workspace

pytestmark = pytest.mark.gpu


def make(T, E, k, seed, S=1, mask=False, offsets=None, add=True, spread=1.0, ids_cut=False):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((T, E)) * spread + 0.5 * rng.standard_normal(E)).astype(np.float32)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    if ids_cut:   # slots that live on another GPU
        ids[rng.random(ids.shape) < 0.4] = -1
    m = (rng.random(T) > 0.25).astype(np.uint8) if mask else None
    if m is not None and T:
        logits[m == 0] = np.nan
    if offsets is None and S > 1:
        offsets = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    return dict(logits=logits, ids=ids, mask=m, offsets=offsets, S=S if offsets is None else len(offsets) - 1,
                d_in=(rng.standard_normal((T, E)) * 1e-3).astype(np.float32) if add else None,
                w=np.array([0.3, 0.05], np.float32), k=k)


def run(c, inplace=False, stream=None):
    T, E = c["logits"].shape
    S, k = c["S"], c["k"]
    dm = moe.dims(T, 128, 128, E, k)
    logits, ids = dev(c["logits"]), dev(c["ids"], torch.int32)
    mask = None if c["mask"] is None else dev(c["mask"], torch.uint8)
    goff = None if c["offsets"] is None else dev(c["offsets"], torch.int32)
    o = {"losses": Guarded((2,), torch.float32), "counts": Guarded((S, E), torch.int32, fill=7),
         "tokens": Guarded((S + 2,), torch.int32, fill=7), "lse": Guarded((T,), torch.float32),
         "d_logits": Guarded((T, E), torch.float32)}
    nb = moe.moe_balance_workspace_bytes(dm, S)
    ws = workspace(nb + 256)
    t = {n: g.t for n, g in o.items()}
    d_in = None if c["d_in"] is None else dev(c["d_in"])
    if inplace:
        t["d_logits"].copy_(d_in)
        d_in = t["d_logits"]
    moe.moe_balance_forward(dm, logits, ids, mask, goff, S, t["counts"], t["tokens"], t["losses"], t["lse"], ws, nb,
                            stream=stream)
    moe.moe_balance_backward(dm, logits, t["lse"], goff, S, t["counts"], t["tokens"], dev(c["w"]), d_in, t["d_logits"],
                             stream=stream)
    torch.cuda.synchronize()
    assert torch.all(ws[max(nb, 0):] == 0xA5), "written behind the workspace"
    return {n: g.check() for n, g in o.items()}


def check(c, o):
    b = R.balance(c["logits"], c["ids"], c["mask"], c["offsets"])
    d, size = R.balance_grad(b, c["k"], c["w"].astype(np.float64), c["d_in"])
    assert np.array_equal(f64(o["counts"]), b["counts"])
    assert np.array_equal(f64(o["tokens"]), b["tokens"])
    on = b["group"] >= 0
    top = np.where(on, np.abs(np.where(on[:, None], c["logits"], 0)).max(1, initial=0, where=np.isfinite(c["logits"])), 0)
    assert_close("lse", o["lse"], b["lse"], 2.0 ** -16 * (1 + top))
    zb = 2 * np.abs(b["lse"][on]).max(initial=0) * 2.0 ** -16 * (1 + top.max(initial=0)) + 2.0 ** -15 * b["losses"][1]
    assert_close("losses", o["losses"], b["losses"], [2.0 ** -15 * b["losses"][0], zb])
    assert_close("d_logits", o["d_logits"], d, 2.0 ** -15 * (size - (0 if c["d_in"] is None else np.abs(c["d_in"])))
                 + 2.0 ** -23 * (size + np.abs(d)))
    if c["d_in"] is not None:   # rows that do not count are left as they were
        assert np.array_equal(f64(o["d_logits"])[~on], c["d_in"].astype(np.float64)[~on])


CASES = {
    # every layout of a row over lanes: vectors of 4 for E % 4 == 0, single values otherwise
    "E1": dict(T=5, E=1, k=1), "E4": dict(T=70, E=4, k=2), "E8_k8": dict(T=64, E=8, k=8),
    "E32": dict(T=129, E=32, k=4), "E60": dict(T=77, E=60, k=3), "E128": dict(T=300, E=128, k=8),
    "E256": dict(T=65, E=256, k=8), "E500": dict(T=40, E=500, k=8), "E1024_k64": dict(T=33, E=1024, k=64),
    "E7": dict(T=200, E=7, k=2), "E65": dict(T=64, E=65, k=5), "E129": dict(T=130, E=129, k=8),
    "E509": dict(T=66, E=509, k=8), "E1023": dict(T=9, E=1023, k=3),
    "one_token": dict(T=1, E=128, k=8), "one_tile": dict(T=128, E=33, k=3), "two_tiles": dict(T=129, E=48, k=4),
    "tiles_of_64": dict(T=8193, E=24, k=2, S=3), "no_add": dict(T=100, E=64, k=4, add=False),
    "mask": dict(T=257, E=64, k=4, mask=True), "seqs": dict(T=400, E=96, k=4, S=9, mask=True),
    # tiles of more than 64 tokens: T > 1024 * 64
    "long": dict(T=70001, E=16, k=2, S=5, mask=True),
    # groups that begin late, end early, are empty, are of one token, end on a tile's edge
    "ragged": dict(T=300, E=128, k=8, offsets=np.array([3, 3, 64, 65, 65, 128, 191, 256, 290], np.int32), mask=True),
    "all_outside": dict(T=100, E=16, k=2, offsets=np.array([100, 100], np.int32)),
    "one_each": dict(T=70, E=12, k=2, offsets=np.arange(71, dtype=np.int32)),
    # as many groups as offsets that a wave loads at a time, one less and one more, and far more
    **{f"groups_{S}": dict(T=3 * S // 2, E=20, k=2, S=S, mask=S % 2 == 0) for S in (62, 63, 64, 127, 128, 255, 256, 1000)},
    "more_groups_than_tokens": dict(T=42, E=385, k=3, S=43), "groups_in_few_tiles": dict(T=900, E=200, k=6, S=400, mask=True),
    "most_groups": dict(T=3000, E=9, k=2, S=65535), "groups_in_long": dict(T=40000, E=12, k=2, S=300, mask=True),
    "local_slots": dict(T=150, E=32, k=8, ids_cut=True), "wide_logits": dict(T=90, E=40, k=4, spread=6.0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_balance_parity(name):
    print(f"[case] balance {name}", flush=True)
    c = make(seed=hash_of(name), **CASES[name])
    o = run(c)
    check(c, o)
    again = run(c, inplace=c["d_in"] is not None)
    for n in o:
        assert torch.equal(o[n].view(torch.int32), again[n].view(torch.int32)), f"{n} differs from run to run"


def hash_of(name):
    return sum(ord(ch) * 31 ** i for i, ch in enumerate(name)) % (1 << 31)


def test_rows_without_a_choice_and_forbidden_experts():
    """-inf logits: an expert that cannot be chosen, a token that has none left, the type's lowest value."""
    c = make(130, 24, 3, 5, mask=True)
    rng = np.random.default_rng(6)
    on = c["mask"] != 0
    c["logits"][on] = np.where(rng.random((on.sum(), 24)) < 0.3, -np.inf, c["logits"][on])
    c["mask"][7:12] = 1
    c["logits"][7] = -np.inf                                   # no expert left: does not count
    c["logits"][8] = np.where(np.arange(24) == 5, 2.0, -np.inf)   # one left
    c["logits"][9] = np.where(np.arange(24) == 5, 2.0, np.finfo(np.float32).min)   # masked by the lowest value
    c["logits"][10], c["logits"][11] = 0.25, 1.0
    print("[case] balance forbidden experts", flush=True)
    o = run(c)
    check(c, o)
    assert float(o["lse"][7]) == -np.inf and torch.equal(o["d_logits"][7].cpu(), torch.from_numpy(c["d_in"][7]))


def test_everything_masked_and_the_empty_batch():
    print("[case] balance nothing counts", flush=True)
    c = make(90, 16, 2, 7)
    c["mask"] = np.zeros(90, np.uint8)
    o = run(c)
    check(c, o)
    assert f64(o["losses"]).tolist() == [0, 0] and not o["counts"].any() and not o["tokens"].any()
    o = run(make(0, 16, 2, 8))
    assert f64(o["losses"]).tolist() == [0, 0] and not o["counts"].any() and not o["tokens"].any()
    o = run(make(0, 16, 2, 8, offsets=np.zeros(4, np.int32)))
    assert f64(o["losses"]).tolist() == [0, 0] and not o["counts"].any() and not o["tokens"].any()


def test_gradient_against_differences():
    """The whole pass on the GPU, differentiated by central differences of the losses it returns
    (steps of 2^-4: the losses' fp32 rounding, 2^-24 relative, over a step is 2^-19; the third
    derivative of a softmax term is at most itself, times step^2 / 6 = 2^-10.6)."""
    print("[case] balance differences", flush=True)
    c = make(6, 8, 2, 9, add=False)
    c["w"][:] = 1.0
    d = f64(run(c)["d_logits"])
    h = 2.0 ** -4
    for t, e in ((0, 0), (2, 3), (5, 7)):
        up, down = dict(c, logits=c["logits"].copy()), dict(c, logits=c["logits"].copy())
        up["logits"][t, e] += h
        down["logits"][t, e] -= h
        diff = (f64(run(up)["losses"]).sum() - f64(run(down)["losses"]).sum()) / (2 * h)
        total = f64(run(c)["losses"]).sum()
        assert abs(diff - d[t, e]) <= 2.0 ** -10 * max(1.0, total) + 2.0 ** -18 * total


def test_joint_counts_of_two_shards():
    """Two GPUs' halves of a batch with counts and tokens added between the directions: the gradient is
    that of the joint batch."""
    print("[case] balance shards", flush=True)
    T, E, k = 160, 32, 4
    c = make(T, E, k, 10, add=False)
    dm, half = moe.dims(T, 128, 128, E, k), moe.dims(T // 2, 128, 128, E, k)
    whole = run(c)
    w = dev(c["w"])
    parts = []
    for i in range(2):
        rows = slice(i * T // 2, (i + 1) * T // 2)
        x, ids = dev(c["logits"][rows]), dev(c["ids"][rows], torch.int32)
        counts, tokens = torch.empty((1, E), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
        losses, lse = torch.empty(2, device="cuda"), torch.empty(T // 2, device="cuda")
        moe.moe_balance_forward(half, x, ids, None, None, 1, counts, tokens, losses, lse,
                                workspace(moe.moe_balance_workspace_bytes(half, 1)))
        parts.append((x, counts, tokens, lse))
    counts = parts[0][1] + parts[1][1]
    tokens = parts[0][2] + parts[1][2]
    tokens[-1] = 1
    assert torch.equal(counts, whole["counts"])
    got = []
    for x, _, _, lse in parts:
        d = torch.empty((T // 2, E), device="cuda")
        moe.moe_balance_backward(half, x, lse, None, 1, counts, tokens, w, None, d)
        got.append(d)
    assert torch.equal(torch.cat(got), whole["d_logits"])


def test_two_streams_with_workspaces_of_their_own():
    print("[case] balance two streams", flush=True)
    cs = [make(5000, 64, 4, 11, S=3), make(5000, 64, 4, 12, S=3)]
    ref = [run(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, s, r in zip(cs, streams, ref):
        with torch.cuda.stream(s):
            o = run(c)
        for n in r:
            assert torch.equal(o[n], r[n])
