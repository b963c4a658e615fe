"""Cases of scored routing (sigmoid or softmax scores, balance bias, groups) with its gradient, and of
the 8-bit quantiser and matrix product with one scale for each block of 128, each in plain torch
operations and as the library's calls (``own``)."""
import math

import torch

own = False
device = "cuda" if torch.cuda.is_available() else "cpu"

BF16, F32, F64, F8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn, torch.int32
TYPES = {"bf16": BF16, "f32": F32}
BLOCK = 128
INF = math.inf


# ------------------------------------------------------------------ cases
def _route(name, T, E, k, score, groups=1, keep=1, best=1, bias=False, renorm=True, scale=1.0, mask=False, ban=False):
    case = {"op": "route", "T": T, "E": E, "k": k, "score": score, "groups": groups, "keep": keep, "best": best,
            "bias": bias, "renorm": renorm, "scale": scale, "mask": mask, "ban": ban}
    return {"name": name, **case} if name else case


def _backward(name, T, E, k, score, renorm, scale, mask):
    case = {"op": "backward", "T": T, "E": E, "k": k, "score": score, "renorm": renorm, "scale": scale, "mask": mask}
    return {"name": name, **case} if name else case


def _quantize(name, form, rows, cols, src):
    case = {"op": "quantize", "form": form, "rows": rows, "cols": cols, "src": src}
    return {"name": name, **case} if name else case


def _matmul(name, form, M, N, K, out, add):
    case = {"op": "matmul", "form": form, "M": M, "N": N, "K": K, "out": out, "add": add}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one new token through a 256-expert gate with groups and bias: latency
        _route("route_1x256_groups", 1, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5),
        # a training micro-batch through a 128-expert softmax gate whose weights are its probabilities
        _route("route_16384x128_softmax", 16384, 128, 8, "softmax", renorm=False),
        # the tokens of a large batch over 256 experts in groups, padded rows among them, some experts barred for
        # some tokens, and the bias moved by the counts
        _route("route_21804x256_groups", 21804, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5, mask=True, ban=True),
        # gradient of a small softmax gate whose weights are probabilities: every logit has one
        _backward("backward_1000x64_softmax", 1000, 64, 6, "softmax", False, 1.0, False),
        # gradient of the large batch's sigmoid gate
        _backward("backward_21804x256_sigmoid", 21804, 256, 8, "sigmoid", True, 2.5, True),
        # a decode batch's rows, in front of a product
        _quantize("quantize_rows_17x7168", "rows", 17, 7168, "bf16"),
        # a batch's output gradients along the tokens, for the weights' gradient
        _quantize("quantize_tokens_21804x4096", "tokens", 21804, 4096, "bf16"),
        # one token times a weight matrix [K, N]: the weights' bytes count
        _matmul("matmul_1x4096x7168_kn", "kn", 1, 4096, 7168, "bf16", False),
        # a decode batch times a weight matrix stored [N, K]
        _matmul("matmul_48x7168x2048_nk", "nk", 48, 7168, 2048, "bf16", False),
        # a short batch's input gradient: dy times the transposed weights
        _matmul("matmul_1023x7168x4096_nk", "nk", 1023, 7168, 4096, "bf16", False),
        # the large batch through the first product of a dense layer
        _matmul("matmul_21804x4096x7168_kn", "kn", 21804, 4096, 7168, "bf16", False),
        # that product's weight gradient, added to the gradient of the micro-batches before
        _matmul("matmul_7168x4096x21808_rows", "rows", 7168, 4096, 21808, "f32", True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["route", "route", "backward", "quantize", "matmul", "matmul", "matmul"])
    if op in ("route", "backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        each = _log_int(rng, 3, 512 // groups)
        E = groups * each
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * each))
        T = _log_int(rng, 1, min(65536, 21804 * 256 // E))
        score, renorm, scale = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, rng.choice([1.0, 2.5])
        mask = rng.random() < 0.5
        if op == "backward":
            return _backward(None, T, E, k, score, renorm, scale, mask)
        return _route(None, T, E, k, score, groups, keep, rng.randint(1, 2), rng.random() < 0.6, renorm, scale, mask, rng.random() < 0.3)
    if op == "quantize":
        cols = 16 * _log_int(rng, 1, 1024)
        rows = _log_int(rng, 1, min(65536, 21804 * 4096 // cols))
        return _quantize(None, rng.choice(["rows", "tokens", "tiles"]), rows, cols, rng.choice(["bf16", "f32"]))
    form = rng.choice(["kn", "nk", "rows"])
    N, K = 16 * _log_int(rng, 4, 512), 16 * _log_int(rng, 8, 1024)
    M = _log_int(rng, 1, min(32768, 21804 * 4096 * 7168 // (N * K)))
    return _matmul(None, form, M, N, K, rng.choice(["bf16", "f32"]), rng.random() < 0.3)


# ------------------------------------------------------------------ inputs
def _rand(shape, gen, dtype=F32, scale=1.0):
    return torch.randn(shape, generator=gen, device=device).mul_(scale).to(dtype)


def _up(n, m):
    return -(-n // m) * m


def _spread(rows, cols, gen, scale=1.0):
    """Activations: columns of unlike size, as a residual stream has them."""
    return _rand((rows, cols), gen, scale=scale) * torch.exp(_rand((cols,), gen, scale=0.5))


def _coded(x, block):
    """e4m3 codes of x and the scales of its blocks (rows x columns of a block): a stand-in for stored data."""
    R, C = x.shape
    r, c = block
    p = torch.nn.functional.pad(x, (0, -C % c, 0, -R % r)).view(_up(R, r) // r, r, _up(C, c) // c, c)
    scale = (p.abs().amax((1, 3)) / 448).clamp(min=2.0 ** -126)
    codes = (p / scale[:, None, :, None]).to(F8).view(torch.uint8)
    return codes.view(_up(R, r), _up(C, c))[:R, :C].contiguous().view(F8), scale


def _inputs(case, seed):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("route", "backward"):
        T, E, k = (case[n] for n in "TEk")
        # a gate that prefers some experts
        logits = _rand((T, E), gen) + _rand((E,), gen, scale=0.5)
        s = {"logits": logits, "mask": None}
        if op == "route":
            s["bias"] = _rand((E,), gen, scale=0.02) if case["bias"] else None
            if case["ban"]:  # experts that a token must not go to
                logits.masked_fill_(torch.rand((T, E), generator=gen, device=device) < 1 / 64, -INF)
        else:
            s["ids"] = torch.topk(logits + _rand((T, E), gen, scale=0.1), k, dim=1).indices.to(I32)
            s["d_w"] = _rand((T, k), gen, scale=1e-2)
        if case["mask"]:  # padding: about a sixteenth of the tokens; their logits are whatever was there
            drop = torch.rand(T, generator=gen, device=device) < 1 / 16
            logits[drop] = math.nan
            if op == "route":
                s["mask"] = (~drop).to(torch.uint8)
            else:
                s["ids"][drop] = -1
        return s
    if op == "quantize":
        return {"src": _spread(case["rows"], case["cols"], gen).to(TYPES[case["src"]])}
    M, N, K, form = (case[n] for n in ("M", "N", "K", "form"))
    s = {}
    s["a"], s["a_scale"] = _coded(_spread(M, K, gen), (1, BLOCK))
    shape = (K, N) if form == "kn" else (N, K)
    b = _spread(N, K, gen, 0.1) if form == "rows" else _rand(shape, gen, scale=K ** -0.5)
    s["b"], s["b_scale"] = _coded(b, (1, BLOCK) if form == "rows" else (BLOCK, BLOCK))
    s["add"] = _rand((M, N), gen, TYPES[case["out"]]) if case["add"] else None
    return s


RATE = 1e-3   # of the bias


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _handles(case, s)
    return s


def _handles(case, s):
    """What a program keeps beside its inputs: output buffers, workspaces and descriptors."""
    import grouped_gemm_expert_router_amd as moe

    def new(*shape, dtype=F32):
        return torch.empty(shape, dtype=dtype, device=device)

    def ws(n):
        return torch.empty(max(n, 256), dtype=torch.uint8, device=device)

    op = case["op"]
    if op in ("route", "backward"):
        T, E, k = (case[n] for n in "TEk")
        kinds = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}
        more = {"groups": case["groups"], "group_topk": case["keep"], "group_best": case["best"]} if op == "route" else {}
        sd = s["sd"] = moe.score_desc(T, E, k, kinds[case["score"]], renormalise=case["renorm"], scale=case["scale"], **more)
        if op == "backward":
            s["d_logits"] = new(T, E)
            return
        s["out"] = {"ids": new(T, k, dtype=I32), "w": new(T, k), "counts": new(E, dtype=I32), "offsets": new(E + 1, dtype=I32),
                    "perm": torch.full((T * k,), -1, dtype=I32, device=device), "inv_perm": new(T * k, dtype=I32)}
        s["new_bias"] = new(E) if case["bias"] else None
        s["ws"] = ws(moe.moe_score_workspace_bytes(sd))
    elif op == "quantize":
        R, C = case["rows"], case["cols"]
        blocks = lambda n: _up(n, BLOCK) // BLOCK  # noqa: E731
        codes, scales = {"rows": ((R, C), (R, blocks(C))), "tokens": ((C, _up(R, 16)), (C, blocks(R))),
                         "tiles": ((R, C), (blocks(R), blocks(C)))}[case["form"]]
        s.update(codes=new(*codes, dtype=F8), scales=new(*scales))
    else:
        forms = {"kn": moe.MOE_B_KN, "nk": moe.MOE_B_NK, "rows": moe.MOE_B_NK_ROWS}
        outs = {"bf16": moe.MOE_BF16, "f32": moe.MOE_F32}
        s["md"] = moe.matmul_desc(case["M"], case["N"], case["K"], forms[case["form"]], outs[case["out"]])
        s["c"] = new(case["M"], case["N"], dtype=TYPES[case["out"]])
        s["ws"] = ws(moe.moe_fp8_matmul_workspace_bytes(s["md"]))


# ------------------------------------------------------------------ one pass
def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _own_route(s):
    import grouped_gemm_expert_router_amd as moe
    o = s["out"]
    moe.moe_score_route(s["sd"], s["logits"], s["bias"], s["mask"], o["ids"], o["w"], o["counts"], o["offsets"], o["perm"], o["inv_perm"], s["ws"])
    if s["bias"] is None:
        return o
    moe.moe_bias_update(o["counts"], RATE, s["bias"], s["new_bias"])
    return {**o, "bias": s["new_bias"]}


def _own_backward(s):
    import grouped_gemm_expert_router_amd as moe
    moe.moe_score_backward(s["sd"], s["logits"], s["ids"], s["d_w"], s["d_logits"])
    return s["d_logits"]


def _own_quantize(s):
    import grouped_gemm_expert_router_amd as moe
    case = s["case"]
    forms = {"rows": moe.MOE_BLOCK_ROWS, "tokens": moe.MOE_BLOCK_TOKENS, "tiles": moe.MOE_BLOCK_TILES}
    moe.moe_fp8_quantize(s["src"], case["rows"], case["cols"], forms[case["form"]], s["codes"], s["scales"])
    return {"codes": s["codes"], "scales": s["scales"]}


def _own_matmul(s):
    import grouped_gemm_expert_router_amd as moe
    moe.moe_fp8_matmul(s["md"], s["a"], s["a_scale"], s["b"], s["b_scale"], s["add"], s["c"], s["ws"])
    return s["c"]


def _ordered(c):
    """Values in descending order and where they stood; ties to the lower place."""
    return torch.sort(c, dim=-1, descending=True, stable=True)


def _plain_route(s):
    case = s["case"]
    T, E, k = (case[n] for n in "TEk")
    x = s["logits"].double()   # the choice is between values next to each other: 64 bits
    ok = x > -INF
    if s["mask"] is not None:
        ok &= (s["mask"] != 0)[:, None]
        x = torch.where(ok, x, -INF)
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top > -INF, top, 0.0))
        score = e / e.sum(1, keepdim=True)
    c = score if s["bias"] is None else score + s["bias"].double()
    c = torch.where(ok, c, -INF)
    if case["groups"] > 1:
        each = E // case["groups"]
        best = _ordered(c.view(T, case["groups"], each)).values[:, :, :case["best"]]
        value = torch.where(best > -INF, best, 0.0).sum(2)
        value = torch.where(best[:, :, 0] > -INF, value, -INF)
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, _ordered(value).indices[:, :case["keep"]], True)
        c = torch.where(kept[:, :, None], c.view(T, case["groups"], each), -INF).view(T, E)
    best, ids = _ordered(c)
    best, ids = best[:, :k], ids[:, :k]
    there = best > -INF
    w = torch.where(there, score.gather(1, ids), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    ids = torch.where(there, ids, -1)
    # the plan: pairs by expert, in their order
    key = torch.where(there, ids, E).view(-1)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    ends = torch.cumsum(counts, 0)
    order = torch.sort(key, stable=True).indices
    place = torch.arange(T * k, device=device)
    inv = torch.empty_like(place).scatter_(0, order, place)
    out = {"ids": ids.int(), "w": (w * case["scale"]).float(), "counts": counts.int(),
           "offsets": torch.cat([ends.new_zeros(1), ends]).int(), "perm": torch.where(place < ends[-1], order, -1).int(),
           "inv_perm": torch.where(key < E, inv, -1).int()}
    if s["bias"] is not None:
        out["bias"] = s["bias"] + RATE * torch.sign(counts.sum() - E * counts)
    return out


def _plain_backward(s):
    case, x = s["case"], s["logits"]
    ids = s["ids"].long()
    there = ids >= 0
    at = ids.clamp(min=0)
    x = torch.where(there.any(1, keepdim=True), x, 0.0)
    score = 1 / (1 + torch.exp(-x)) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    chosen = torch.where(there, score.gather(1, at), 0.0)
    g = torch.where(there, s["d_w"], 0.0) * case["scale"]
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        w = chosen / total
        g = torch.where(there, (g - (g * w).sum(1, keepdim=True)) / total, 0.0)
    d = torch.zeros_like(x).scatter_add_(1, at, g)
    if case["score"] == "sigmoid":
        return d * score * (1 - score)
    return score * (d - (d * score).sum(1, keepdim=True))


def _plain_quantize(s):
    case, x = s["case"], s["src"].float()
    R, C = x.shape
    if case["form"] == "tokens":
        x, R, C = x.t(), C, R
    r = BLOCK if case["form"] == "tiles" else 1
    p = torch.nn.functional.pad(x, (0, -C % BLOCK, 0, -R % r)).view(_up(R, r) // r, r, _up(C, BLOCK) // BLOCK, BLOCK)
    top = p.abs().amax((1, 3))
    scale = torch.where(top > 0, top.clamp(min=448 * 2.0 ** -126) / 448, 1.0)
    factor = torch.where(top > 0, 448 / top.clamp(min=448 * 2.0 ** -126), 1.0)
    codes = (p * factor[:, None, :, None]).clamp(-448, 448).to(F8).view(torch.uint8)
    codes = codes.view(_up(R, r), _up(C, BLOCK))[:R, :_up(C, 16)].contiguous().view(F8)
    return {"codes": codes, "scales": scale}


def _valued(codes, scale, block, dtype):
    """The values that codes and scales stand for."""
    scale = scale.to(dtype).repeat_interleave(block, 1)[:, :codes.shape[1]]
    if scale.shape[0] != codes.shape[0]:
        scale = scale.repeat_interleave(block, 0)[:codes.shape[0]]
    return codes.to(dtype) * scale


def _plain_matmul(s):
    a, b = _valued(s["a"], s["a_scale"], BLOCK, F32), _valued(s["b"], s["b_scale"], BLOCK, F32)
    c = torch.matmul(a, b if s["case"]["form"] == "kn" else b.t())
    if s["add"] is not None:
        c = c + s["add"].float()
    return c.to(TYPES[s["case"]["out"]])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    if op == "route":
        T, E, k = (case[n] for n in "TEk")
        # logits, bias, mask; ids, weights, perm and inv_perm; counts, offsets, the new bias
        return {"bytes": T * E * 4 + T * case["mask"] + T * k * 16 + E * (8 + 8 * case["bias"]), "flops": T * E * 12}
    if op == "backward":
        T, E, k = (case[n] for n in "TEk")
        # the gradient; ids and their gradients; the chosen logits, or all of them where all have a part in the sum
        every = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * 4 + T * k * 8 + (T * E * 4 if every else T * k * 4), "flops": T * (E * 8 if every else k * 12)}
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        scales = {"rows": R * _up(C, BLOCK), "tokens": C * _up(R, BLOCK), "tiles": _up(R, BLOCK) * _up(C, BLOCK) // BLOCK}[case["form"]] // BLOCK
        return {"bytes": R * C * (size[case["src"]] + 1) + 4 * scales, "flops": 3 * R * C}
    M, N, K = case["M"], case["N"], case["K"]
    blocks = _up(K, BLOCK) // BLOCK
    b_scales = N * blocks if case["form"] == "rows" else blocks * _up(N, BLOCK) // BLOCK
    return {"bytes": M * K + N * K + 4 * (M * blocks + b_scales) + M * N * size[case["out"]] * (1 + case["add"]), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, _inputs(case, seed))


def _first_best(c):
    """Where each row's largest value stands first, and that value."""
    top = c.max(-1, keepdim=True).values
    place = torch.arange(c.shape[-1], device=device).expand_as(c)
    return torch.where(c == top, place, c.shape[-1]).min(-1).values, top[..., 0]


def _exact_route(case, s):
    """One choice after the other from the definition, with the chosen struck out."""
    T, E, k, G = (case[n] for n in ("T", "E", "k", "groups"))
    live = torch.ones(T, dtype=torch.bool, device=device) if s["mask"] is None else s["mask"].bool()
    x = torch.where(live[:, None], s["logits"].double(), -INF)
    free = ~torch.isinf(x)
    if case["score"] == "sigmoid":
        score = torch.sigmoid(x)
    else:
        score = torch.nan_to_num(torch.exp(x - torch.logsumexp(x, 1, keepdim=True)), nan=0.0)
    c = score + (0 if s["bias"] is None else s["bias"].double())
    c = c.masked_fill(~free, -INF)
    if G > 1:
        left, value = c.reshape(T, G, E // G).clone(), torch.zeros((T, G), dtype=F64, device=device)
        some = torch.isfinite(left).any(2)
        for _ in range(min(case["best"], E // G)):
            at, top = _first_best(left)
            value += torch.nan_to_num(top, neginf=0.0)
            left.scatter_(2, at[..., None], -INF)
        value = value.masked_fill(~some, -INF)
        kept = torch.zeros((T, G), dtype=torch.bool, device=device)
        for _ in range(case["keep"]):
            at, _ = _first_best(value)
            kept.scatter_(1, at[:, None], True)
            value = value.masked_fill(kept, -INF)
            value[kept.all(1)] = 0
        c = c.masked_fill(~kept.repeat_interleave(E // G, 1), -INF)
    ids = torch.full((T, k), -1, dtype=torch.int64, device=device)
    for j in range(k):
        at, top = _first_best(c)
        ids[:, j] = torch.where(torch.isfinite(top), at, -1)
        c = c.scatter(1, at[:, None], -INF)
    there = ids >= 0
    w = score.gather(1, ids.clamp(min=0)) * there
    if case["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    flat = ids.view(-1)
    perm = torch.full((T * k,), -1, dtype=I32, device=device)
    inv = torch.full((T * k,), -1, dtype=I32, device=device)
    counts = torch.zeros(E, dtype=torch.int64, device=device)
    begin = 0
    for e in range(E):
        pairs = torch.nonzero(flat == e)[:, 0]
        counts[e] = pairs.numel()
        perm[begin:begin + pairs.numel()] = pairs.int()
        inv[pairs] = torch.arange(begin, begin + pairs.numel(), device=device, dtype=I32)
        begin += pairs.numel()
    out = {"ids": ids.int(), "w": w * case["scale"], "counts": counts.int(),
           "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(), "perm": perm, "inv_perm": inv}
    if s["bias"] is not None:
        over = (counts.double() - counts.double().mean()).sign()
        out["bias"] = s["bias"].double() - RATE * over
    return out


def _exact_backward(case, s):
    """The weights from the definition, differentiated."""
    x = torch.where((s["ids"] >= 0).any(1)[:, None], s["logits"].double(), 0.0).requires_grad_()
    score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    there = s["ids"] >= 0
    w = score.gather(1, s["ids"].long().clamp(min=0)) * there
    if case["renorm"]:
        w = w / torch.where(there.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    return torch.autograd.grad((w * case["scale"] * torch.where(there, s["d_w"].double(), 0.0)).sum(), x)[0]


def _exact_quantize(case, s):
    x = s["src"].double()
    if case["form"] == "tokens":
        x = x.transpose(0, 1)
    R, C = x.shape
    r = BLOCK if case["form"] == "tiles" else 1
    full = x.new_zeros((_up(R, r), _up(C, BLOCK)))
    full[:R, :C] = x
    top = torch.nn.functional.max_pool2d(full.abs()[None, None], (r, BLOCK))[0, 0]
    scale = torch.where(top == 0, 1.0, top / 448)
    v = full / scale.repeat_interleave(r, 0).repeat_interleave(BLOCK, 1)
    # nearest e4m3 value, ties to even: three bits behind the leading one, steps of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    v = torch.round(v / step) * step
    return {"codes": v[:R, :_up(C, 16)].contiguous(), "scales": scale}


def _exact_matmul(case, s):
    a, b = _valued(s["a"], s["a_scale"], BLOCK, F64), _valued(s["b"], s["b_scale"], BLOCK, F64)
    if case["form"] == "kn":
        b = b.t().contiguous()
    c = torch.nn.functional.linear(a, b)
    return c if s["add"] is None else c + s["add"].double()
