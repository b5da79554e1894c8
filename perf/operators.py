"""Workloads of the mixture-of-experts operators: what each measures, its
inputs, its plain form in elementary torch operations, and its values from
the definition in 64 bits.

Three operators, in both directions where a model trains through them:

  route        expert scores of every token (softmax or sigmoid) -> the top-k
               experts and their weights, with a balance bias, expert groups
               and renormalisation; and the gradient of the logits
  combine      the experts' output rows of every token, weighted and summed
               in token order; and the gradients of the rows and the weights
  w4_matvec    a few rows times a matrix held in 4 bits with group scales,
               alone or as the products of the experts each token is routed to

``own`` selects the side that ``run`` takes: False computes the plain form,
True calls the library.  All inputs come from the seed alone.
"""
import math

import torch

own = False

E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


# ---- cases --------------------------------------------------------------------
def _route(T, E, topk, dtype, score, bias=False, groups=1, topk_groups=1, group_score="max", renorm=False, scale=1.0,
           pad=0, masked=False, op="route"):
    return {"op": op, "T": T, "E": E, "topk": topk, "dtype": dtype, "score": score, "bias": bias, "groups": groups,
            "topk_groups": topk_groups, "group_score": group_score, "renorm": renorm, "scale": scale, "pad": pad,
            "masked": masked}


def _combine(T, topk, n, experts, laid_out, op="combine"):
    return {"op": op, "T": T, "topk": topk, "n": n, "experts": experts, "laid_out": laid_out}


def _w4(m, n, k, group, fmt, scales, zeros=False, out="bf16"):
    return {"op": "w4", "m": m, "n": n, "k": k, "group": group, "fmt": fmt, "scales": scales, "zeros": zeros,
            "out": out}


def _w4_experts(T, topk, E, n, k, group, fmt, scales, zeros=False, out="bf16", per_pair=False):
    return {"op": "w4_experts", "T": T, "topk": topk, "E": E, "n": n, "k": k, "group": group, "fmt": fmt,
            "scales": scales, "zeros": zeros, "out": out, "per_pair": per_pair}


def listed():
    return [
        # one decoding step of a small batch: every microsecond is latency
        dict(_route(8, 256, 8, "bf16", "sigmoid", bias=True, groups=8, topk_groups=4, group_score="top2",
                    renorm=True, scale=2.5), name="route_decode"),
        # a long prefill batch through the same router, FP32 logits
        dict(_route(32768, 256, 8, "f32", "sigmoid", bias=True, groups=8, topk_groups=4, group_score="top2",
                    renorm=True, scale=2.5), name="route_prefill"),
        # an odd expert count in a padded logits buffer, some experts masked off, some rows without any
        dict(_route(5003, 60, 4, "f32", "softmax", pad=4, masked=True), name="route_softmax_odd"),
        # training: the gradient of the router's logits (the softmax runs over all experts, so it is dense)
        dict(_route(16384, 128, 8, "bf16", "softmax", op="route_bwd"), name="route_backward"),
        # decode: 32 tokens' expert rows, one after another
        dict(_combine(32, 8, 7168, 16, False), name="combine_decode"),
        # prefill: rows in the grouped GEMM's layout, 128-row blocks per expert
        dict(_combine(4096, 8, 7168, 16, True), name="combine_prefill"),
        # training: the gradients of the experts' rows and of the routing weights, an odd row count
        dict(_combine(4001, 4, 4096, 8, True, op="combine_bwd"), name="combine_backward"),
        # one token, a projection of the benchmark's dense sweep
        dict(_w4(1, 4096, 7168, 128, "int4", "bf16"), name="w4_one_token"),
        # a short batch with the finest groups and an output width that fills no tile
        dict(_w4(5, 2111, 7168, 32, "e2m1", "bf16"), name="w4_fine_groups"),
        # 16 tokens against the longest reduction of the dense sweep, zero points, FP32 output
        dict(_w4(16, 7168, 16384, 128, "int4", "f32", zeros=True, out="f32"), name="w4_sixteen_tokens"),
        # one token's chosen experts, out of 64
        dict(_w4_experts(1, 8, 64, 4096, 2048, 64, "int4", "bf16", zeros=True), name="w4_experts_one_token"),
        # a decoding batch that reaches nearly every expert, one input row per pair (a second projection)
        dict(_w4_experts(64, 8, 128, 7168, 2048, 128, "e2m1", "f32", per_pair=True), name="w4_experts_batch"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("route", "route_bwd", "combine", "combine_bwd", "w4", "w4", "w4_experts", "w4_experts"))
    if kind.startswith("route"):
        groups = rng.choice((1, 1, 2, 4, 8, 5))
        per = _log(rng, max(4, 8 // groups), 256 // groups)
        topk_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(16, per * topk_groups))
        score = rng.choice(("softmax", "sigmoid"))
        bias = rng.random() < 0.5
        return _route(_log(rng, 1, 16384), groups * per, topk, rng.choice(("f32", "bf16")), score, bias, groups,
                      topk_groups, rng.choice(("max", "top2")), rng.random() < 0.5, rng.choice((1.0, 2.5)),
                      rng.choice((0, 0, 3, 8)), rng.random() < 0.25, kind)
    if kind.startswith("combine"):
        n = 8 * _log(rng, 8, 896)
        n += 8 if n == 3072 else 0
        return _combine(_log(rng, 1, 4096), rng.randint(1, 8), n, rng.choice((8, 16, 40)), rng.random() < 0.7, kind)
    group = rng.choice((32, 64, 128))
    fmt = rng.choice(("int4", "e2m1"))
    more = {"zeros": fmt == "int4" and rng.random() < 0.5, "out": rng.choice(("bf16", "bf16", "f32"))}
    if kind == "w4":
        n = _log(rng, 16, 8192)
        n += 1 if n == 3072 else 0
        k = group * _log(rng, max(1, 256 // group), 8192 // group)
        k += group if k == 3072 else 0
        return _w4(_log(rng, 1, 64), n, k, group, fmt, rng.choice(("f32", "bf16")), **more)
    n = 8 * _log(rng, 8, 512)
    n += 8 if n == 3072 else 0
    k = group * _log(rng, max(1, 256 // group), 4096 // group)
    k += group if k == 3072 else 0
    E = rng.choice((8, 16, 40, 64))
    return _w4_experts(_log(rng, 1, 64), rng.randint(1, 8), E, n, k, group, fmt, rng.choice(("f32", "bf16")), **more,
                       per_pair=rng.random() < 0.5)


def work(case):
    c = case
    if c["op"].startswith("route"):
        T, E, k, b = c["T"], c["E"], c["topk"], _BYTES[c["dtype"]]
        if c["op"] == "route":
            return {"bytes": T * E * b + (4 * E if c["bias"] else 0) + T * k * 8, "flops": 4 * T * E}
        dense = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": T * E * b + (T * E * b if dense else T * k * b) + T * k * 8,
                "flops": 6 * T * E if dense else 10 * T * k}
    if c["op"].startswith("combine"):
        T, k, n = c["T"], c["topk"], c["n"]
        index = 4 * T * k if c["laid_out"] else 0
        if c["op"] == "combine":
            return {"bytes": T * k * n * 2 + T * n * 2 + index + 4 * T * k, "flops": 2 * T * k * n}
        return {"bytes": 2 * T * k * n * 2 + T * n * 2 + index + 8 * T * k, "flops": 3 * T * k * n}
    n, k, g = c["n"], c["k"], c["group"]
    matrix = n * k // 2 + n * (k // g) * (_BYTES[c["scales"]] + (1 if c["zeros"] else 0))
    if c["op"] == "w4":
        return {"bytes": matrix + c["m"] * k * 2 + c["m"] * n * _BYTES[c["out"]], "flops": 2 * c["m"] * n * k}
    P = c["T"] * min(c["topk"], c["E"])
    reached = c["E"] * (1 - (1 - min(c["topk"], c["E"]) / c["E"]) ** c["T"])  # experts with a token, on average
    rows = P if c["per_pair"] else c["T"]
    return {"bytes": int(reached * matrix) + rows * k * 2 + P * n * _BYTES[c["out"]] + 4 * P, "flops": 2 * P * n * k}


# ---- inputs -------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logits(case, g, rows):
    """Logits as a router's projection gives them: a spread over the experts, some of them hotter; with `masked`,
    an eighth of the entries masked off, and one row in 64 without any expert (a padding token)."""
    E = case["E"]
    x = (1.5 * _randn(g, rows, E) + 0.5 * _randn(g, 1, E)).to(_DTYPES[case["dtype"]])
    if case["masked"]:
        x.masked_fill_(torch.rand(rows, E, generator=g, device="cuda") < 0.125, -math.inf)
        x.masked_fill_(torch.rand(rows, 1, generator=g, device="cuda") < 1 / 64, -math.inf)
    return x


def _undecided(case, logits, bias):
    """Rows in which two candidates lie so close (without being equal) that the rounding of exp decides between them."""
    E, G = case["E"], case["groups"]
    l = logits.double()
    off = torch.isneginf(l)
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, -1).nan_to_num(0.0)
    b = torch.zeros(E, dtype=torch.float64, device="cuda") if bias is None else bias.double()
    pick = (s + b).masked_fill(off, -math.inf)
    room = (4e-6 * (s + b.abs())).masked_fill(off, 0.0)

    def close(values, rooms, count):
        v, at = values.sort(-1, descending=True)
        r = rooms.gather(-1, at)
        gap = (v[:, :-1] - v[:, 1:])[:, :count]
        return ((gap > 0) & (gap < (r[:, :-1] + r[:, 1:])[:, :count])).any(-1)

    bad = close(pick, room, case["topk"])
    if G > 1:
        grouped = pick.view(-1, G, E // G)
        two, at = grouped.topk(min(2 if case["group_score"] == "top2" else 1, E // G), -1)
        score = two[..., 0] + torch.where(torch.isneginf(two[..., 1]), 0.0, two[..., 1]) if two.shape[-1] == 2 else two[..., 0]
        score_room = room.view(-1, G, E // G).gather(-1, at).sum(-1)
        bad |= close(score, score_room, case["topk_groups"])
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(-1, score.sort(dim=-1, descending=True, stable=True)[1][:, :case["topk_groups"]], True)
        bad |= close(grouped.masked_fill(~keep[..., None], -math.inf).view(-1, E), room, case["topk"])
    return bad


def _distinct_experts(g, T, topk, E):
    """topk different experts per token, hotter ones more often."""
    heat = 0.7 * _randn(g, 1, E)
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    return (heat + noise).topk(min(topk, E), -1)[1].to(torch.int32)


def _laid_out(expert, E):
    """Row of every pair when each expert's pairs follow one another from a multiple of 128, and the rows that always
    suffice for that."""
    flat = expert.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    starts, before = ends - (counts + 127) // 128 * 128, torch.cumsum(counts, 0) - counts
    order = torch.argsort(flat, stable=True)
    dst = torch.empty_like(flat)
    dst[order] = starts[flat[order]] + torch.arange(flat.numel(), device="cuda") - before[flat[order]]
    return dst.view(expert.shape).to(torch.int32), (flat.numel() + E * 127 + 127) // 128 * 128


def _matrix(case, g, experts):
    """4-bit codes, scales and zero points of `experts` matrices (codes spread as rounded weights are)."""
    n, k, G = case["n"], case["k"], case["k"] // case["group"]
    codes = torch.empty(experts, n, k // 2, dtype=torch.uint8, device="cuda")
    for e in range(experts):
        if case["fmt"] == "int4":
            c = (8.0 + 2.6 * _randn(g, n, k)).round_().clamp_(0, 15).to(torch.uint8)
        else:
            c = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
        codes[e] = c[:, 0::2] | (c[:, 1::2] << 4)
    scales = (0.004 * torch.exp(0.4 * _randn(g, experts, n, G))).to(_DTYPES[case["scales"]])
    zeros = None
    if case["zeros"]:
        zeros = (8.0 + 1.2 * _randn(g, experts, n, G)).round_().clamp_(0, 15).to(torch.uint8)
    return codes, scales, zeros


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op.startswith("route"):
        T, E, k = case["T"], case["E"], case["topk"]
        # a balance bias, moved in steps of 0.001
        s["bias"] = (30 * _randn(g, E)).round().mul(0.001) if case["bias"] else None
        x = _logits(case, g, T)
        for _ in range(50):  # which of two nearly equal experts wins is no property of the operator: draw such rows again
            bad = _undecided(case, x, s["bias"]).nonzero().view(-1)
            if not bad.numel():
                break
            x[bad] = _logits(case, g, bad.numel())
        wide = torch.empty(T, E + case["pad"], dtype=x.dtype, device="cuda").fill_(7.0)
        wide[:, :E] = x
        s["logits"] = wide[:, :E]
        if op == "route":
            s["expert_idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty(T, k, device="cuda")
        else:
            s["expert_idx"] = _plain_route(case, s["logits"], s["bias"])[0]
            s["grad_weights"] = _randn(g, T, k)
            s["grad_logits"] = torch.empty(T, E, dtype=x.dtype, device="cuda")
    elif op.startswith("combine"):
        T, k, n = case["T"], case["topk"], case["n"]
        s["dst_row"], rows = None, T * k
        if case["laid_out"]:
            s["dst_row"], rows = _laid_out(_distinct_experts(g, T, k, case["experts"]), case["experts"])
            s["dst_row"].masked_fill_(torch.rand(T, k, generator=g, device="cuda") < 0.01, -1)  # dropped pairs
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        s["weights"] = 2.5 * w / w.sum(-1, keepdim=True)
        s["y"] = _randn(g, rows, n).to(torch.bfloat16)
        if op == "combine":
            s["out"] = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
        else:
            s["grad_out"] = _randn(g, T, n).to(torch.bfloat16)
            s["grad_y"] = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")  # padding rows stay zero
            s["grad_weights"] = torch.empty(T, k, device="cuda")
    else:
        k, n = case["k"], case["n"]
        rows = case["m"] if op == "w4" else case["T"]
        if op == "w4":
            s["w"], s["scales"], s["zeros"] = (None if v is None else v[0] for v in _matrix(case, g, 1))
        else:
            s["w"], s["scales"], s["zeros"] = _matrix(case, g, case["E"])
            s["expert_idx"] = _distinct_experts(g, rows, case["topk"], case["E"])
            rows = s["expert_idx"].numel()
        s["x"] = _randn(g, case["T"] if op != "w4" and not case["per_pair"] else rows, k).to(torch.bfloat16)
        s["out"] = torch.empty(rows, n, dtype=_DTYPES[case["out"]], device="cuda")
    return s


# ---- the plain form -------------------------------------------------------------
def _plain_scores(case, logits):
    """(scores, experts that may be picked), FP32."""
    l = logits.float()
    able = l > -math.inf
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l)), able
    e = torch.exp(l - l.amax(-1, keepdim=True).clamp_min(-3.0e38)) * able
    return e / e.sum(-1, keepdim=True).clamp_min(1e-37), able


def _plain_weights(case, picked, valid):
    w = picked * valid
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-37)
    return w * case["scale"]


def _first(values, count):
    """Indices of the `count` largest per row, in order, ties to the lowest index."""
    return values.sort(dim=-1, descending=True, stable=True)[1][..., :count]


def _plain_route(case, logits, bias):
    T, E, G = case["T"], case["E"], case["groups"]
    s, able = _plain_scores(case, logits)
    pick = (s if bias is None else s + bias).masked_fill(~able, -math.inf)
    if G > 1:
        best = pick.view(T, G, E // G).sort(-1, descending=True)[0][..., :2]
        score = best[..., 0]
        if case["group_score"] == "top2" and E // G > 1:
            score = score + best[..., 1].masked_fill(best[..., 1] == -math.inf, 0.0)
        keep = torch.zeros(T, G, dtype=torch.bool, device=pick.device).scatter_(1, _first(score, case["topk_groups"]), True)
        pick = pick.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    at = _first(pick, case["topk"])
    valid = pick.gather(1, at) > -math.inf
    return at.masked_fill(~valid, -1).to(torch.int32), _plain_weights(case, s.gather(1, at), valid)


def _plain_route_backward(case, logits, expert_idx, grad_weights):
    s, _ = _plain_scores(case, logits)
    valid = expert_idx >= 0
    at = expert_idx.long().clamp_min(0)
    p = s.gather(1, at) * valid
    gw = grad_weights * valid * case["scale"]
    if case["renorm"]:  # weights p / sum(p)
        total = p.sum(-1, keepdim=True).clamp_min(1e-37)
        gp = (gw - (gw * p).sum(-1, keepdim=True) / total) / total * valid
    else:
        gp = gw
    gs = torch.zeros_like(s).scatter_add_(1, at, gp)
    if case["score"] == "sigmoid":
        gl = gs * s * (1.0 - s)
    else:
        gl = s * (gs - (gs * s).sum(-1, keepdim=True))
    return gl.to(logits.dtype)


def _plain_matrix(case, codes, scales, zeros):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    c = c.unflatten(-1, (-1, case["group"]))
    if case["fmt"] == "e2m1":
        v = torch.tensor(E2M1_VALUES, device="cuda")[c.int()]
    else:
        v = c.float() - (8.0 if zeros is None else zeros.float()[..., None])
    return (v * scales.float()[..., None]).flatten(-2)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "route":
        return _plain_route(c, s["logits"], s["bias"])
    if op == "route_bwd":
        return _plain_route_backward(c, s["logits"], s["expert_idx"], s["grad_weights"])
    if op.startswith("combine"):
        T, k = c["T"], c["topk"]
        dst = s["dst_row"] if s["dst_row"] is not None else torch.arange(T * k, device="cuda").view(T, k)
        valid, at = (dst >= 0)[..., None], dst.long().clamp_min(0)
        rows = s["y"][at].float() * valid
        if op == "combine":
            return (rows * s["weights"][..., None]).sum(1).to(torch.bfloat16)
        go = s["grad_out"].float()[:, None]
        gy = torch.zeros(s["y"].shape[0] + 1, c["n"], dtype=torch.bfloat16, device="cuda")
        gy[dst.long().masked_fill(dst < 0, s["y"].shape[0])] = (s["weights"][..., None] * go).to(torch.bfloat16)
        return gy[:-1], (go * rows).sum(-1)
    x, out = s["x"].float(), _DTYPES[c["out"]]
    if op == "w4":
        return (x @ _plain_matrix(c, s["w"], s["scales"], s["zeros"]).t()).to(out)
    e = s["expert_idx"].long().view(-1)
    pair = torch.arange(e.numel(), device="cuda")
    row = pair if c["per_pair"] else pair // s["expert_idx"].shape[1]
    if e.numel() < c["E"]:  # each pair's own matrix
        w = _plain_matrix(c, s["w"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e])
        return (w @ x[row][..., None]).squeeze(-1).to(out)
    w = _plain_matrix(c, s["w"], s["scales"], s["zeros"])  # every token times every matrix, then the routed ones
    token = pair // s["expert_idx"].shape[1]
    if c["per_pair"]:
        x = torch.zeros(c["E"], c["T"], c["k"], device="cuda").index_put_((e, token), x)
    return (x @ w.transpose(1, 2))[e, token].to(out)


def _own(s):
    import fp8_block_scaled_04_amd as fp8
    c, op = s["case"], s["case"]["op"]
    if op.startswith("route"):
        score = fp8.FP8G_SIGMOID if c["score"] == "sigmoid" else fp8.FP8G_SOFTMAX
        if op == "route":
            return fp8.fp8_moe_route(s["logits"], c["topk"], score, s["bias"], c["groups"], c["topk_groups"],
                                     fp8.FP8G_GROUP_TOP2 if c["group_score"] == "top2" else fp8.FP8G_GROUP_MAX,
                                     c["renorm"], c["scale"], s["expert_idx"], s["weights"])
        return fp8.fp8_moe_route_backward(s["logits"], s["expert_idx"], s["grad_weights"], s["grad_logits"], score,
                                          c["renorm"], c["scale"])
    if op == "combine":
        return fp8.fp8_moe_combine(s["y"], s["dst_row"], s["weights"], s["out"])
    if op == "combine_bwd":
        return fp8.fp8_moe_combine_backward(s["grad_out"], s["y"], s["dst_row"], s["weights"], s["grad_y"],
                                            s["grad_weights"])
    fmt = fp8.FP8G_E2M1 if c["fmt"] == "e2m1" else fp8.FP8G_INT4
    if op == "w4":
        return fp8.fp8_w4_matvec(s["x"], s["w"], s["scales"], s["out"], fmt, s["zeros"])
    return fp8.fp8_w4_matvec_experts(s["x"], s["expert_idx"], s["w"], s["scales"], s["out"], fmt, s["zeros"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ----------------------------------------------------
def _exact_picks(case, sel, able):
    """Picked experts of every row, best first: repeated maxima of the selection scores, the lowest index first."""
    T, E, G = case["T"], case["E"], case["groups"]
    sel = torch.where(able, sel, -math.inf)
    if G > 1:
        left, gscore = sel.view(T, G, -1).clone(), None
        for _ in range(2 if case["group_score"] == "top2" else 1):
            top, at = left.max(-1)
            gscore = top if gscore is None else gscore + torch.where(top == -math.inf, 0.0, top)
            left.scatter_(-1, at[..., None], -math.inf)
        kept = torch.zeros(T, G, dtype=torch.bool, device=sel.device)
        for _ in range(case["topk_groups"]):
            at = gscore.argmax(-1, keepdim=True)
            first = (gscore == gscore.gather(1, at)).int().argmax(-1, keepdim=True)
            kept.scatter_(1, first, gscore.gather(1, first) > -math.inf)
            gscore.scatter_(1, first, -math.inf)
        sel = torch.where(kept[..., None].expand(T, G, E // G).reshape(T, E), sel, -math.inf)
    sel, picks = sel.clone(), []
    for _ in range(case["topk"]):
        top = sel.max(-1, keepdim=True)[0]
        first = (sel == top).int().argmax(-1, keepdim=True)
        picks.append(torch.where(top == -math.inf, -1, first))
        sel.scatter_(1, first, -math.inf)
    return torch.cat(picks, 1)


def _exact_values(case, logits):
    """log of every expert's score, and which experts there are."""
    l = logits.double()
    able = ~torch.isneginf(l)
    if case["score"] == "sigmoid":
        return -torch.logaddexp(torch.zeros_like(l), -l), able
    return l - torch.logsumexp(l, -1, keepdim=True), able


def _exact_weights(case, logs, picks):
    """Weights of the picked experts (zero where there is none) before the scale."""
    lp = torch.where(picks >= 0, logs.gather(1, picks.clamp_min(0)), -math.inf)
    if case["renorm"]:
        lp = lp - torch.logsumexp(lp, -1, keepdim=True)
    return torch.where(picks >= 0, lp.exp(), 0.0)


def _exact_matrix(case, s, e=None):
    """One matrix in 64 bits."""
    codes, scales, zeros = ((t if e is None or t is None else t[e]) for t in (s["w"], s["scales"], s["zeros"]))
    w = torch.empty(case["n"], case["k"], dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = codes.remainder(16).double(), codes.div(16, rounding_mode="floor").double()
    if case["fmt"] == "e2m1":  # sign, two exponent bits, one mantissa bit
        code = w.clone()
        mag = code.remainder(8)
        step = torch.div(mag, 2, rounding_mode="floor")
        val = torch.where(mag < 2, mag * 0.5, (1 + 0.5 * mag.remainder(2)) * torch.exp2(step - 1))
        w = torch.where(code >= 8, -val, val)
    else:
        w -= 8.0 if zeros is None else zeros.double().repeat_interleave(case["group"], 1)
    return w * scales.double().repeat_interleave(case["group"], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("route"):
        logs, able = _exact_values(case, s["logits"])
        logs = torch.where(able, logs, -math.inf)
        sel = logs.exp() + (0.0 if s["bias"] is None else s["bias"].double())
        if op == "route":
            picks = _exact_picks(case, sel, able)
            return picks.to(torch.int32), _exact_weights(case, logs, picks) * case["scale"]
        # d(weight j)/d(logit e) = scale * weight_j * (d log score_j / d logit_e, less its weighted mean when renormalised)
        picks = s["expert_idx"].long()
        w = _exact_weights(case, logs, picks) * case["scale"]
        gw = s["grad_weights"].double() * w
        if case["renorm"]:
            gw = gw - w / case["scale"] * gw.sum(-1, keepdim=True)
        grad = torch.zeros_like(logs)
        for j in range(case["topk"]):
            at = picks[:, j:j + 1]
            slope = 1.0 - logs.gather(1, at.clamp_min(0)).exp() if case["score"] == "sigmoid" else 1.0
            grad.scatter_add_(1, at.clamp_min(0), torch.where(at >= 0, gw[:, j:j + 1] * slope, 0.0))
        if case["score"] == "softmax":
            grad -= logs.exp().nan_to_num(0.0) * gw.sum(-1, keepdim=True)
        return grad
    if op.startswith("combine"):
        T, k, n = case["T"], case["topk"], case["n"]
        y, w = s["y"], s["weights"].double()
        out = torch.zeros(T, n, dtype=torch.float64, device="cuda")
        gy = torch.zeros(y.shape, dtype=torch.float64, device="cuda") if op != "combine" else None
        gw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            d = s["dst_row"][:, j].long() if s["dst_row"] is not None else torch.arange(T, device="cuda") * k + j
            t = (d >= 0).nonzero().view(-1)
            rows = y[d[t]].double()
            if op == "combine":
                out[t] += w[t, j, None] * rows
            else:
                go = s["grad_out"][t].double()
                gy[d[t]] = w[t, j, None] * go
                gw[t, j] = (go * rows).sum(-1)
        return out if op == "combine" else (gy, gw)
    if op == "w4":
        return s["x"].double() @ _exact_matrix(case, s).t()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    e = s["expert_idx"].view(-1)
    for expert in torch.unique(e).tolist():
        p = (e == expert).nonzero().view(-1)
        rows = s["x"][p if case["per_pair"] else p // s["expert_idx"].shape[1]]
        out[p] = rows.double() @ _exact_matrix(case, s, expert).t()
    return out
