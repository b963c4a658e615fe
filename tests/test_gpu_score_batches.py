"""Routing by scores and its gradient over whole batches, against 64-bit references computed by torch: the launches that
short batches do not take (a gradient of more than 4096 tokens, a choice whose plan does not fit the blocks of the
choice), and choices that leave few or no experts over.

Bounds: test_gpu_score's.  The choice and the plan are equal; a weight within 2^-18 (logits within +-8); a gradient
within 2^-16 of its terms' magnitudes."""
import pytest
import torch

import grouped_gemm_expert_router_amd as moe
from block_testlib import Guarded, workspace
from test_gpu_score import desc, run_backward, run_route

pytestmark = pytest.mark.gpu
I32 = torch.int32


# -------------------------------------------------------------------------------- gradient
def gradient(x, ids, g, sigmoid, renorm, scale):
    """d_logits and the sum of each element's terms' magnitudes; ids out of range have no part."""
    E = x.shape[1]
    there = (ids >= 0) & (ids < E)
    at = torch.where(there, ids, 0).long()
    x = torch.where(there.any(1, keepdim=True), x.double(), 0.0)
    g = torch.where(there, g.double(), 0.0) * scale
    s = torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)
    q = torch.where(there, s.gather(1, at), 0.0)
    if renorm:
        q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
        dlog, size = q * (g - (g * q).sum(1, keepdim=True)), q * (g.abs() + (g * q).abs().sum(1, keepdim=True))
    else:
        dlog, size = g * q, (g * q).abs()
    if sigmoid:
        f = torch.sigmoid(-x).gather(1, at)
        dlog, size = dlog * f, size * f
    zero = torch.zeros_like(x)
    d, total = zero.scatter_add(1, at, torch.where(there, dlog, 0.0)), zero.scatter_add(1, at, torch.where(there, size, 0.0))
    if not sigmoid and not renorm:
        d, total = d - s * dlog.sum(1, keepdim=True), total + s * size.sum(1, keepdim=True)
    return d, total


@pytest.mark.parametrize("T,E,k", [(4097, 256, 8), (4111, 1024, 16), (5003, 63, 4), (8190, 128, 1), (21805, 256, 8), (5001, 96, 20)])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
def test_gradient_of_a_batch(T, E, k, sigmoid, renorm):
    print(f"[case] gradient {T}x{E} k={k}", flush=True)
    gen = torch.Generator("cuda").manual_seed(T + E)
    x = torch.randn(T, E, generator=gen, device="cuda").mul_(1.5).clamp_(-8, 8)
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, 1).indices.to(I32)
    g = torch.randn(T, k, generator=gen, device="cuda")
    if k > 1:
        ids[::5, 1] = ids[::5, 0]                                   # an expert twice
        ids[torch.rand(T, k, generator=gen, device="cuda") < 0.1] = -1
        ids[3::11, 0] = E
    ids[2::7] = -1                                                  # no expert at all: neither row is read
    x[2::7] = float("nan")
    g[ids < 0] = float("nan")
    got = run_backward(desc(T, E, k, sigmoid, renorm, 2.5), x, ids, g).double()
    ref, size = gradient(x, ids, g, sigmoid, renorm, 2.5)
    assert (got[2::7] == 0).all()
    over = (got - ref).abs() - size * 2.0 ** -16 - 1e-37
    assert (over <= 0).all(), (float(over.max()), int((~(over <= 0)).sum()))   # a NaN fails


# ---------------------------------------------------------------------------------- choice
def choice(x, k, sigmoid, bias, mask, groups, keep, best):
    """ids, their scores and whether there is an expert, by sorting in 64 bits."""
    T, E = x.shape
    live = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    y = torch.where(live[:, None], x, 0.0).double()
    s = torch.sigmoid(y) if sigmoid else torch.softmax(y, 1)
    c = s if bias is None else s + bias.double()
    c = torch.where(live[:, None] & (y > -torch.inf), c, -torch.inf)
    if groups > 1:
        top = c.view(T, groups, -1).sort(2, descending=True).values[:, :, :best]
        value = torch.where(top > -torch.inf, top, 0.0).sum(2).masked_fill(top[:, :, 0] == -torch.inf, -torch.inf)
        stay = torch.zeros(T, groups, dtype=torch.bool, device="cuda")
        stay.scatter_(1, torch.sort(value, dim=1, descending=True, stable=True).indices[:, :keep], True)
        c = torch.where(stay[:, :, None], c.view(T, groups, -1), -torch.inf).view(T, E)
    c, ids = torch.sort(c, dim=1, descending=True, stable=True)
    there = c[:, :k] > -torch.inf
    return torch.where(there, ids[:, :k], -1).to(I32), torch.where(there, s.gather(1, ids[:, :k]), 0.0)


def check_batch(x, k, sigmoid, renorm, bias=None, mask=None, groups=1, keep=1, best=1):
    T, E = x.shape
    got = run_route(desc(T, E, k, sigmoid, renorm, 1.0, groups, keep, best), x, bias, mask)
    got = {n: torch.from_numpy(v).cuda() for n, v in got.items()}
    ids, w = choice(x, k, sigmoid, bias, mask, groups, keep, best)
    assert torch.equal(got["ids"], ids)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    assert ((got["w"].double() - w).abs() <= w * 2.0 ** -18).all()
    flat = ids.view(-1).long()
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    order = torch.sort(torch.where(flat >= 0, flat, E), stable=True).indices
    n = int(counts.sum())
    inv = torch.full_like(flat, -1)
    inv[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(got["counts"].long(), counts)
    assert torch.equal(got["offsets"].long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    assert torch.equal(got["perm"][:n].long(), order[:n]) and (got["perm"][n:] == 77).all()   # behind the last: as it was
    assert torch.equal(got["inv_perm"].long(), inv)


@pytest.mark.parametrize("T,E,k,groups", [(131072, 32, 16, 1), (131073, 32, 16, 4), (262150, 16, 8, 2), (200001, 40, 11, 8), (1100000, 8, 2, 1)])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_choice_of_a_batch_whose_plan_is_made_apart(T, E, k, groups, sigmoid):
    """The last batch whose pairs the choice's blocks hold, and batches past it."""
    print(f"[case] route {T}x{E} k={k}", flush=True)
    gen = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, E, generator=gen, device="cuda").mul_(1.5).clamp_(-8, 8)
    bias = torch.randn(E, generator=gen, device="cuda") * 0.02
    mask = torch.rand(T, generator=gen, device="cuda") < 0.9
    x[~mask] = float("nan")
    keep = max(groups // 2, -(-k * groups // E))
    check_batch(x, k, sigmoid, True, bias, mask.to(torch.uint8), groups, keep, 2)


@pytest.mark.parametrize("E,k,groups,keep", [(8, 8, 1, 1), (8, 7, 1, 1), (8, 6, 1, 1), (64, 8, 8, 1), (64, 7, 8, 1), (16, 16, 1, 1), (17, 16, 1, 1),
                                             (128, 16, 8, 1), (1, 1, 1, 1), (3, 2, 1, 1), (24, 6, 4, 1), (300, 16, 2, 1)])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_as_many_experts_as_are_chosen(E, k, groups, keep, sigmoid):
    """All of the experts that stay are chosen, or all but one or two; with barred ones there are fewer than slots."""
    gen = torch.Generator("cuda").manual_seed(E + k)
    for T in (3, 2000):
        x = torch.randn(T, E, generator=gen, device="cuda").mul_(1.5).clamp_(-8, 8)
        bias = torch.randn(E, generator=gen, device="cuda") * 0.02
        check_batch(x, k, sigmoid, True, None, None, groups, keep, 2)
        check_batch(x, k, sigmoid, False, bias, None, groups, keep, 1)
        x[torch.rand(T, E, generator=gen, device="cuda") < 0.1] = -torch.inf
        x[:, 0] = 0.5                                               # no token without an expert: its softmax would be NaN here
        check_batch(x, k, sigmoid, True, None, None, groups, keep, 2)
        check_batch(x, k, sigmoid, False, bias, None, groups, keep, 2)


# ------------------------------------------------------------------------- as many tokens as there may be
def chunks(n, step=1 << 27):
    for i in range(0, n, step):
        yield i, min(n, i + step)


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def test_the_largest_batch():
    """2^31 - 1 pairs: every third token goes to expert 0, the others to expert 1; the plan, the weights and the gradient in
    closed form.  Plain scores of sigmoids: w = s, d_l = s (1 - s)."""
    room(120)
    T = (1 << 31) - 1
    x = torch.zeros(T, 2, device="cuda")
    x[:, 1] = 1
    x[::3, 1] = -1
    sd = desc(T, 2, 1, True, False)
    o = {"ids": Guarded((T, 1), I32, fill=77), "w": Guarded((T, 1), torch.float32), "counts": Guarded((2,), I32, fill=77),
         "offsets": Guarded((3,), I32, fill=77), "perm": Guarded((T,), I32, fill=77), "inv_perm": Guarded((T,), I32, fill=77)}
    moe.moe_score_route(sd, x, None, None, *[o[n].t for n in ("ids", "w", "counts", "offsets", "perm", "inv_perm")],
                        workspace(moe.moe_score_workspace_bytes(sd)))
    torch.cuda.synchronize()
    o = {n: g.check().view(-1) for n, g in o.items()}
    n0 = (T + 2) // 3
    assert o["counts"].tolist() == [n0, T - n0] and o["offsets"].tolist() == [0, n0, T]
    s0, s1 = 0.5, 1 / (1 + 2.718281828459045 ** -1)
    for a, b in chunks(T):
        t = torch.arange(a, b, device="cuda")
        third = t % 3 == 0
        pos = torch.where(third, t // 3, n0 + t - (t + 2) // 3)
        assert torch.equal(o["ids"][a:b], (~third).to(I32)) and torch.equal(o["inv_perm"][a:b].long(), pos)
        assert torch.equal(o["perm"][pos].long(), t)
        want = torch.where(third, s0, s1)
        assert ((o["w"][a:b] - want).abs() <= want * 2.0 ** -18).all()
        del t, third, pos, want
    ids = o["ids"].view(T, 1)
    del o
    g = torch.ones(T, 1, device="cuda")
    d = Guarded((T, 2), torch.float32)
    moe.moe_score_backward(sd, x, ids, g, d.t)
    torch.cuda.synchronize()
    d = d.check()
    for a, b in chunks(T):
        third = torch.arange(a, b, device="cuda") % 3 == 0
        want = torch.stack([torch.where(third, s0 * (1 - s0), 0.0), torch.where(third, 0.0, s1 * (1 - s1))], 1)
        assert ((d[a:b] - want).abs() <= want * 2.0 ** -18).all()
        del third, want


@pytest.mark.parametrize("k,sigmoid", [(2, True), (2, False), (17, False)])
def test_logits_past_32_bit_offsets(k, sigmoid):
    """More than 2^31 logits of more than 2^24 tokens, whose rows repeat: choice, weights and gradient repeat with them."""
    room(100)
    T, E, period = (1 << 24) + 77, 136, 1009
    gen = torch.Generator("cuda").manual_seed(1)
    base = torch.randn(period, E, generator=gen, device="cuda").mul_(1.5).clamp_(-8, 8)
    g0 = torch.randn(period, k, generator=gen, device="cuda")
    times = -(-T // period)
    x, g = base.repeat(times, 1)[:T], g0.repeat(times, 1)[:T]
    sd, small = desc(T, E, k, sigmoid, False), desc(period, E, k, sigmoid, False)
    ids, w = torch.empty(T, k, dtype=I32, device="cuda"), torch.empty(T, k, device="cuda")
    rest = [torch.empty(n, dtype=I32, device="cuda") for n in (E, E + 1, T * k, T * k)]
    moe.moe_score_route(sd, x, None, None, ids, w, *rest, workspace(moe.moe_score_workspace_bytes(sd)))
    d = torch.empty(T, E, device="cuda")
    moe.moe_score_backward(sd, x, ids, g, d)
    one = run_route(small, base, None, None)
    ids0, w0 = torch.from_numpy(one["ids"]).cuda(), torch.from_numpy(one["w"]).cuda()
    d0 = run_backward(small, base, ids0, g0)
    for got, want in ((ids, ids0), (w, w0), (d, d0)):
        whole = T // period * period
        assert torch.equal(got[:whole].view(-1, period, got.shape[1]), want.expand(whole // period, -1, -1))
        assert torch.equal(got[whole:], want[:T - whole])
    want, score = choice(base, k, sigmoid, None, None, 1, 1, 1)
    assert torch.equal(ids0, want) and ((w0.double() - score).abs() <= score * 2.0 ** -18).all()
    flat = ids.view(-1)
    assert torch.equal(rest[0].long(), torch.bincount(flat, minlength=E))
    assert (flat[rest[2].long()].diff() >= 0).all()                 # pairs by expert
    assert torch.equal(rest[2][rest[3].long()], torch.arange(T * k, dtype=I32, device="cuda"))
