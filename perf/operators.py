"""Cases of the routing and 8-bit integer operators: their inputs, their plain forms in elementary
torch operations, the calls that a program makes of the framework, and their values in 64 bits.

Operators:
  route    hidden states -> experts: sigmoid or softmax scores, a bias that is added for the
           selection only, expert groups of which the best stay, top-k, weights
  logits   the same selection from router logits that the caller already has
  product  bf16 rows quantized to int8 with a scale for each token, times int8 weights with a
           scale for each output channel
  layer    the routed-MoE layer (route, SwiGLU experts, weighted sum, residual, RMSNorm) on int8
           expert weights
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------
def _router(score, bias, n_group, topk_group, group_top, renorm, scale):
    return {"score": score, "bias": bias, "n_group": n_group, "topk_group": topk_group,
            "group_top": group_top, "renorm": renorm, "scale": scale}


# balance bias, 8 groups of which 4 stay by the sum of their two best, weights to sum 1, times 2.5
GROUPED = _router("sigmoid", True, 8, 4, 2, True, 2.5)


def listed():
    return [
        # a decode step of 8 sequences at the layer's real shape: latency
        {"name": "route_decode", "op": "route", "M": 8, "H": 7168, "E": 256, "k": 16, **GROUPED},
        # a prefill chunk at the same shape
        {"name": "route_prefill", "op": "route", "M": 2048, "H": 7168, "E": 256, "k": 16, **GROUPED},
        # softmax scores, groups by their best expert, plain weights; a ragged batch, E not a power of two
        {"name": "route_softmax", "op": "route", "M": 333, "H": 4096, "E": 160, "k": 6,
         **_router("softmax", False, 8, 3, 1, False, 1.0)},
        # one token whose logits another kernel made
        {"name": "logits_token", "op": "logits", "M": 1, "E": 256, "k": 8, "masked": 0.0, **GROUPED},
        # a long prefill whose caller masks experts that are not served
        {"name": "logits_masked", "op": "logits", "M": 8192, "E": 384, "k": 8, "masked": 0.1,
         **_router("softmax", True, 1, 1, 1, True, 1.0)},
        # a shared expert's gate and up projection at decode
        {"name": "product_decode", "op": "product", "M": 8, "N": 4096, "K": 7168, "f32": False},
        # ragged sizes, fp32 results
        {"name": "product_odd", "op": "product", "M": 77, "N": 1537, "K": 2064, "f32": True},
        # the same projection over a long prefill
        {"name": "product_prefill", "op": "product", "M": 8192, "N": 4096, "K": 7168, "f32": False},
        # the layer at decode: bound by the touched experts' weights
        {"name": "layer_decode", "op": "layer", "M": 8, "H": 7168, "E": 256, "I": 2048, "k": 16,
         "block": 16, **GROUPED},
        # a small layer and a ragged batch
        {"name": "layer_small", "op": "layer", "M": 203, "H": 2048, "E": 60, "I": 1408, "k": 4,
         "block": 32, **_router("softmax", False, 1, 1, 1, True, 1.0)},
        # the layer over a prefill chunk: every expert's weights and many rows for each
        {"name": "layer_prefill", "op": "layer", "M": 2048, "H": 7168, "E": 256, "I": 2048, "k": 16,
         "block": 64, **GROUPED},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_router(rng, most_experts):
    n_group = rng.choice([1, 1, 2, 4, 8])
    per = max(2, _log(rng, 8, most_experts) // n_group)
    topk_group = rng.randint(1, n_group)
    r = _router(rng.choice(["sigmoid", "softmax"]), rng.random() < 0.6, n_group, topk_group,
                rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]))
    return n_group * per, min(rng.randint(1, 16), topk_group * per), r


def draw(rng):
    op = rng.choice(["route", "logits", "product", "layer"])
    if op == "route":
        E, k, r = _draw_router(rng, 512)
        return {"op": op, "M": _log(rng, 1, 8192), "H": 8 * _log(rng, 32, 1024), "E": E, "k": k, **r}
    if op == "logits":
        E, k, r = _draw_router(rng, 1024)
        return {"op": op, "M": _log(rng, 1, 16384), "E": E, "k": k,
                "masked": rng.choice([0.0, 0.0, 0.1, 0.5]), **r}
    if op == "product":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, 8192),
                "K": 16 * _log(rng, 16, 512), "f32": rng.random() < 0.3}
    E, k, r = _draw_router(rng, 64)
    return {"op": op, "M": _log(rng, 1, 2048), "H": 64 * _log(rng, 4, 64), "E": E,
            "I": 64 * _log(rng, 4, 32), "k": k, "block": rng.choice([16, 32, 64, 128]), **r}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _normal(g, shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    return t.mul_(std).add_(mean).to(dtype)


def _int8_weights(g, stacks, rows, cols):
    """Normal weights, each row (output channel) as int8 codes and the scale max / 127."""
    codes = torch.empty((stacks, rows, cols), dtype=torch.int8, device=DEV)
    scales = torch.empty((stacks, rows), dtype=torch.float32, device=DEV)
    for e in range(stacks):
        w = torch.randn((rows, cols), generator=g, device=DEV).mul_(0.02)
        top = w.abs().amax(dim=1, keepdim=True)
        codes[e].copy_(w.mul_(127.0 / top).round_())
        scales[e].copy_(top[:, 0] / 127.0)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1_000_003 + 17)
    op, M = case["op"], case["M"]
    s = {"case": case}
    if op in ("route", "layer"):
        # hidden states after a norm, a gate whose logits have a standard deviation of about 1.7
        H, E = case["H"], case["E"]
        s["x"] = _normal(g, (M, H))
        s["gate"] = _normal(g, (E, H), 1.7 / math.sqrt(H))
    if op == "logits":
        E = case["E"]
        s["logits"] = _normal(g, (M, E), 1.7, 0.0, torch.float32)
        if case["masked"]:
            # experts that no token may take, and as many more for each token by itself
            gone = torch.rand((1, E), generator=g, device=DEV) < case["masked"] / 2
            each = torch.rand((M, E), generator=g, device=DEV) < case["masked"] / 2
            s["logits"].masked_fill_(gone | each, -math.inf)
    if op != "product":
        # the bias that a balancing rule has built up
        s["bias"] = _normal(g, (case["E"],), 0.05, 0.0, torch.float32) if case["bias"] else None
    if op == "product":
        s["x"] = _normal(g, (M, case["K"]))
        codes, scales = _int8_weights(g, 1, case["N"], case["K"])
        s["w"], s["w_scale"] = codes[0], scales[0]
    if op == "layer":
        H, I, E = case["H"], case["I"], case["E"]
        s["w13"], s["w13_scale"] = _int8_weights(g, E, 2 * I, H)
        s["w2"], s["w2_scale"] = _int8_weights(g, E, H, I)
        s["residual"] = _normal(g, (M, H))
        s["norm"] = _normal(g, (H,), 0.05, 1.0)
    return s


# ---------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------
def _plain_select(logits, bias, c):
    """Experts and weights from logits in 64 bits (a choice between near scores needs them)."""
    M, E = logits.shape
    k, G = c["k"], c["n_group"]
    off = ~(logits > -math.inf)                       # masked, or not a number: no score
    l = torch.where(off, -math.inf, logits)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(dim=1, keepdim=True)
        p = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        total = p.sum(dim=1, keepdim=True)
        score = p / torch.where(total > 0, total, 1.0)
    choice = score if bias is None else score + bias.double()
    order = l if bias is None else choice             # without a bias the logits have the scores' order
    best = torch.where(off, -math.inf, choice).view(M, G, E // G).topk(c["group_top"], dim=2).values
    some = best[:, :, 0] > -math.inf
    group = torch.where(some, torch.where(best > -math.inf, best, 0.0).sum(dim=2), -math.inf)
    stay = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
    kept = torch.zeros((M, G), dtype=torch.bool, device=l.device).scatter_(1, stay, True)
    kept = kept.repeat_interleave(E // G, dim=1)
    order = torch.where(kept, torch.where(off, -1e300, order), -math.inf)
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_quantize(v):
    """Rows in 32 bits -> codes (as whole float numbers) and the scale of each row."""
    top = v.abs().amax(dim=1, keepdim=True)
    codes = torch.round(v * 127.0 / torch.where(top > 0, top, 1.0))
    return codes, top / 127.0


def _plain_layer(s, c):
    M, I, k = c["M"], c["I"], c["k"]
    ids, w = _plain_select(s["x"].double() @ s["gate"].double().T, s["bias"], c)
    xq, xs = _plain_quantize(s["x"].float())
    m = torch.zeros((M, c["H"]), dtype=torch.float32, device=DEV)
    for e in torch.unique(ids).tolist():              # one product for each expert that has tokens
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = (xq[t] @ s["w13"][e].float().T) * (xs[t] * s["w13_scale"][e])
        act = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
        aq, a_scale = _plain_quantize(act)
        y = (aq @ s["w2"][e].float().T) * (a_scale * s["w2_scale"][e])
        m.index_add_(0, t, y * w[t, j].unsqueeze(1))
    z = m + s["residual"].float()
    out = z * torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS) * s["norm"].float()
    return {"out": out.bfloat16(), "residual": z.bfloat16(), "ids": ids, "weights": w}


def _plain(s, c):
    if c["op"] == "route":
        ids, w = _plain_select(s["x"].double() @ s["gate"].double().T, s["bias"], c)
        return {"ids": ids, "weights": w}
    if c["op"] == "logits":
        ids, w = _plain_select(s["logits"].double(), s["bias"], c)
        return {"ids": ids, "weights": w}
    if c["op"] == "product":
        codes, scale = _plain_quantize(s["x"].float())
        out = (codes @ s["w"].float().T) * (scale * s["w_scale"])
        return {"out": out if c["f32"] else out.bfloat16()}
    return _plain_layer(s, c)


# ---------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------
def _room(s, nbytes):
    """The workspace that a program keeps beside its weights."""
    if "room" not in s:
        s["room"] = torch.empty(max(1, nbytes), dtype=torch.uint8, device=DEV)
    return s["room"]


def _own(s, c):
    from prefill_sigmoid_router_amd import binding as B
    M, op = c["M"], c["op"]
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if op == "product":
        codes, scale = new((M, c["K"]), torch.int8), new((M,), torch.float32)
        out = new((M, c["N"]), torch.float32 if c["f32"] else torch.bfloat16)
        B.moe_i8_quantize(s["x"], codes, scale)
        B.moe_i8_matmul(codes, scale, s["w"], s["w_scale"], out,
                        _room(s, B.moe_i8_matmul_workspace_bytes(M, c["N"], c["K"])))
        return {"out": out}
    k = c["k"]
    ids, w = new((M, k), torch.int32), new((M, k), torch.float32)
    rule = {"score": B.SCORE_SIGMOID if c["score"] == "sigmoid" else B.SCORE_SOFTMAX,
            "n_group": c["n_group"], "topk_group": c["topk_group"], "group_top": c["group_top"],
            "renormalize": c["renorm"], "scale": c["scale"]}
    if op == "route":
        B.moe_route_groups(s["x"], s["gate"], s["bias"], k, ids, w,
                           _room(s, B.moe_route_groups_workspace_bytes(M, c["E"])), **rule)
        return {"ids": ids, "weights": w}
    if op == "logits":
        B.moe_route_logits(s["logits"], s["bias"], k, ids, w, **rule)
        return {"ids": ids, "weights": w}
    H, E, I = c["H"], c["E"], c["I"]
    out, z = new((M, H), torch.bfloat16), new((M, H), torch.bfloat16)
    B.moe_forward_i8(s["x"], s["gate"], s["bias"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"],
                     s["residual"], s["norm"], EPS, k, c["block"], out,
                     _room(s, B.moe_i8_workspace_bytes(M, H, E, I, k, c["block"])),
                     residual_out=z, topk_ids_out=ids, topk_w_out=w, **rule)
    return {"out": out, "residual": z, "ids": ids, "weights": w}


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    M, op = case["M"], case["op"]
    if op == "product":
        N, K = case["N"], case["K"]
        return {"bytes": M * K * 2 + N * K + N * 4 + M * N * (4 if case["f32"] else 2),
                "flops": 2 * M * N * K}
    E, k = case["E"], case["k"]
    picks = M * k * 8 + (E * 4 if case["bias"] else 0)
    if op == "logits":
        return {"bytes": M * E * 4 + picks, "flops": 8 * M * E}
    H = case["H"]
    route = {"bytes": M * H * 2 + E * H * 2 + picks, "flops": 2 * M * E * H}
    if op == "route":
        return route
    I = case["I"]
    touched = E * (1.0 - (1.0 - k / E) ** M)          # experts that the picks are expected to touch
    weights = touched * (3 * H * I + (2 * I + H) * 4)
    return {"bytes": route["bytes"] + weights + 3 * M * H * 2 + H * 2,
            "flops": route["flops"] + 6 * M * k * H * I}


# ---------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_select(logits, bias, c):
    """Token by token: numpy, lexicographic sorts."""
    l = np.asarray(logits, dtype=np.float64)
    M, E = l.shape
    k, G = c["k"], c["n_group"]
    per = E // G
    b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
    ids, w = np.empty((M, k), dtype=np.int64), np.zeros((M, k))
    index = np.arange(E)
    for t in range(M):
        live = l[t] > -np.inf
        score = np.zeros(E)
        if live.any():
            v = l[t][live]
            if c["score"] == "sigmoid":
                score[live] = 1.0 / (1.0 + np.exp(-v))
            else:
                p = np.exp(v - v.max())
                score[live] = p / p.sum()
        choice = score + b
        totals = np.full(G, -np.inf)
        for grp in range(G):
            mine = choice[grp * per:(grp + 1) * per][live[grp * per:(grp + 1) * per]]
            if mine.size:
                totals[grp] = np.sort(mine)[::-1][:c["group_top"]].sum()
        chosen = np.lexsort((np.arange(G), -totals))[:c["topk_group"]]
        inside = np.isin(index // per, chosen)
        key = choice if bias is not None else np.where(live, l[t], 0.0)
        ranked = np.lexsort((index, -np.where(live, key, 0.0), ~live, ~inside))
        ids[t] = ranked[:k]
        got = score[ids[t]]
        if c["renorm"] and got.sum() > 0:
            got = got / got.sum()
        w[t] = got * c["scale"]
    return ids, w


def _exact_quantize(v):
    top = v.abs().max(dim=1).values
    safe = torch.where(top == 0, torch.ones_like(top), top)
    return (127.0 * v / safe[:, None]).round(), top / 127.0


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "product":
        codes, scale = _exact_quantize(s["x"].double())
        total = torch.matmul(codes, s["w"].double().T.contiguous())
        return {"out": total * scale[:, None] * s["w_scale"].double()[None, :]}
    logits = s["logits"] if op == "logits" else torch.matmul(s["x"].double(), s["gate"].double().T.contiguous())
    ids, w = _exact_select(logits.double().cpu().numpy(), s["bias"], c)
    ids, w = torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
    if op != "layer":
        return {"ids": ids, "weights": w}
    M, I, k = c["M"], c["I"], c["k"]
    codes, scale = _exact_quantize(s["x"].double())
    flat = ids.reshape(-1)
    y = torch.zeros((M * k, c["H"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        rows = torch.nonzero(flat == e)[:, 0]
        if rows.numel() == 0:
            continue
        t = torch.div(rows, k, rounding_mode="floor")
        h = torch.matmul(codes[t], s["w13"][e].double().T.contiguous())
        h = h * scale[t][:, None] * s["w13_scale"][e].double()[None, :]
        gate, up = h[:, :I], h[:, I:]
        a_codes, a_scale = _exact_quantize(gate * torch.sigmoid(gate) * up)
        part = torch.matmul(a_codes, s["w2"][e].double().T.contiguous())
        y[rows] = part * a_scale[:, None] * s["w2_scale"][e].double()[None, :]
    z = (y.view(M, k, c["H"]) * w[:, :, None]).sum(dim=1) + s["residual"].double()
    out = z / torch.sqrt((z * z).mean(dim=1, keepdim=True) + EPS) * s["norm"].double()
    return {"out": out, "residual": z, "ids": ids, "weights": w}
