"""Cases of the operators around and inside a routed-MoE block: their inputs, their plain forms in
elementary torch operations, the calls that a program makes of the framework, and their values in
64 bits.

Operators:
  norm     the norm after a block, its gate and scale, the residual, and the next block's norm
  product  bf16 tokens times bf16 weights with bias, activation (gated or not) and residual in
           the epilogue
  layer    the whole routed-MoE layer (route, SwiGLU experts, weighted sum, residual, RMSNorm)
           for a few tokens
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
def _router(score, select_bias, router_bias, n_group, topk_group, group_top, renorm, scale):
    return {"score": score, "select_bias": select_bias, "router_bias": router_bias,
            "n_group": n_group, "topk_group": topk_group, "group_top": group_top,
            "renorm": renorm, "scale": scale}


# the layer's own router: sigmoid scores renormalised over the picks
PLAIN = _router("sigmoid", False, False, 1, 1, 1, True, 1.0)
# balance bias, 8 groups of which 4 stay by the sum of their two best, weights to sum 1, times 2.5
GROUPED = _router("sigmoid", True, False, 8, 4, 2, True, 2.5)


def listed():
    return [
        # between two blocks at decode, one token: latency
        {"name": "norm_token", "op": "norm", "M": 1, "H": 7168, "post": "rms", "pre": "rms",
         "gate": "none", "y_f32": False, "r_f32": False, "bias": False, "offset": 0.0, "a": 1.0,
         "b": 1.0, "pad": 0},
        # a ragged batch with layer norms, a gate for each token and channel, a residual stream in
        # fp32, rows that are slices of wider ones
        {"name": "norm_odd", "op": "norm", "M": 333, "H": 2056, "post": "layer", "pre": "layer",
         "gate": "full", "y_f32": True, "r_f32": True, "bias": True, "offset": 0.0, "a": 0.5,
         "b": 1.5, "pad": 24},
        # between two blocks over a long prefill: a channel gate, weights around 0 (1 + w)
        {"name": "norm_prefill", "op": "norm", "M": 8192, "H": 7168, "post": "rms", "pre": "rms",
         "gate": "channel", "y_f32": False, "r_f32": False, "bias": False, "offset": 1.0, "a": 1.0,
         "b": 0.25, "pad": 0},
        # a shared expert at decode: gate and up projection with SwiGLU
        {"name": "product_decode", "op": "product", "M": 8, "N": 2048, "K": 7168, "act": "silu",
         "gated": True, "bias": False, "res": "none", "f32": False, "pad": 0},
        # its down projection onto the residual stream
        {"name": "product_down", "op": "product", "M": 8, "N": 7168, "K": 2048, "act": "none",
         "gated": False, "bias": False, "res": "bf16", "f32": False, "pad": 0},
        # ragged sizes, a column count without alignment, rows that are slices of wider ones
        {"name": "product_odd", "op": "product", "M": 77, "N": 1537, "K": 2072, "act": "gelu",
         "gated": False, "bias": True, "res": "f32", "f32": True, "pad": 8},
        # a down projection over a prefill chunk, bias and residual
        {"name": "product_chunk", "op": "product", "M": 2048, "N": 7168, "K": 2048, "act": "none",
         "gated": False, "bias": True, "res": "bf16", "f32": False, "pad": 0},
        # the shared expert's gate and up projection over a long prefill
        {"name": "product_prefill", "op": "product", "M": 8192, "N": 2048, "K": 7168, "act": "silu",
         "gated": True, "bias": False, "res": "none", "f32": False, "pad": 0},
        # a tiny layer: launches and hand-overs only
        {"name": "layer_tiny", "op": "layer", "M": 4, "H": 256, "E": 8, "I": 512, "k": 2, **PLAIN},
        # one token through a small layer with softmax scores
        {"name": "layer_token", "op": "layer", "M": 1, "H": 2048, "E": 60, "I": 1408, "k": 4,
         **_router("softmax", False, True, 1, 1, 1, True, 1.0)},
        # one token at the real shape
        {"name": "layer_single", "op": "layer", "M": 1, "H": 7168, "E": 256, "I": 2048, "k": 16,
         **PLAIN},
        # a decode step of 8 sequences at the real shape, with expert groups
        {"name": "layer_decode", "op": "layer", "M": 8, "H": 7168, "E": 256, "I": 2048, "k": 16,
         **GROUPED},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "product", "layer"])
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 8192), "H": 8 * _log(rng, 8, 896),
                "post": rng.choice(["none", "rms", "rms", "layer"]),
                "pre": rng.choice(["none", "rms", "rms", "layer"]),
                "gate": rng.choice(["none", "channel", "full", "token"]),
                "y_f32": rng.random() < 0.3, "r_f32": rng.random() < 0.4,
                "bias": rng.random() < 0.4, "offset": rng.choice([0.0, 1.0]),
                "a": rng.choice([1.0, 0.5]), "b": rng.choice([1.0, 0.25]),
                "pad": rng.choice([0, 0, 8, 40])}
    if op == "product":
        gated = rng.random() < 0.4
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 33, 4096),
                "K": 8 * _log(rng, 8, 896), "gated": gated,
                "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"] if gated else
                                  ["none", "none", "silu", "gelu", "gelu_tanh", "relu"]),
                "bias": rng.random() < 0.5, "res": rng.choice(["none", "bf16", "f32"]),
                "f32": rng.random() < 0.3, "pad": rng.choice([0, 0, 8, 40])}
    n_group = rng.choice([1, 1, 2, 4, 8])
    per = max(2, _log(rng, 8, 96) // n_group)
    topk_group = rng.randint(1, n_group)
    return {"op": op, "M": rng.randint(1, 16), "H": 8 * _log(rng, 32, 896), "E": n_group * per,
            "I": 16 * _log(rng, 8, 128), "k": min(rng.randint(1, 16), topk_group * per),
            **_router(rng.choice(["sigmoid", "softmax"]), rng.random() < 0.5, rng.random() < 0.3,
                      n_group, topk_group, rng.choice([1, 2]), rng.random() < 0.7,
                      rng.choice([1.0, 2.5]))}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _normal(g, shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    return t.mul_(std).add_(mean).to(dtype)


def _rows(g, M, n, pad, std, dtype):
    """[M, n], a slice of rows that are `pad` values longer."""
    return _normal(g, (M, n + pad), std, 0.0, dtype)[:, :n]


def _dtype(f32):
    return torch.float32 if f32 else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1_000_003 + 29)
    op, M = case["op"], case["M"]
    s = {"case": case}
    if op == "norm":
        # a residual stream that has grown over the layers, with a few channels far above the rest
        H, pad = case["H"], case["pad"]
        s["y"] = _rows(g, M, H, pad, 1.0, _dtype(case["y_f32"]))
        s["residual"] = _rows(g, M, H, pad, 3.0, _dtype(case["r_f32"]))
        s["residual"][:, ::max(1, H // 4)] *= 24.0
        around = 1.0 - case["offset"]
        for n in ("post", "pre"):
            s[n + "_w"] = _normal(g, (H,), 0.05, around) if case[n] != "none" else None
            with_bias = case[n] != "none" and case["bias"]
            s[n + "_b"] = _normal(g, (H,), 0.1) if with_bias else None
        shape = {"none": None, "channel": (1, H), "full": (M, H), "token": (M, 1)}[case["gate"]]
        s["gate"] = None if shape is None else _normal(g, shape, 0.3, 0.7)
    if op == "product":
        # tokens after a norm, weights of a trained model's size
        N, K = case["N"], case["K"]
        rows = 2 * N if case["gated"] else N
        s["x"] = _rows(g, M, K, case["pad"], 1.0, torch.bfloat16)
        s["w"] = _normal(g, (rows, K), 0.02)
        s["bias"] = _normal(g, (rows,), 0.2) if case["bias"] else None
        s["residual"] = None
        if case["res"] != "none":
            s["residual"] = _rows(g, M, N, case["pad"], 2.0, _dtype(case["res"] == "f32"))
    if op == "layer":
        # hidden states after a norm, a gate whose logits have a standard deviation of about 1.7
        H, E, I = case["H"], case["E"], case["I"]
        s["x"] = _normal(g, (M, H))
        s["router"] = _normal(g, (E, H), 1.7 / math.sqrt(H))
        s["router_bias"] = _normal(g, (E,), 0.5, 0.0, torch.float32) if case["router_bias"] else None
        s["select_bias"] = _normal(g, (E,), 0.05, 0.0, torch.float32) if case["select_bias"] else None
        s["w13"] = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
        s["w2"] = torch.empty((E, H, I), dtype=torch.bfloat16, device=DEV)
        for e in range(E):
            s["w13"][e].copy_(_normal(g, (2 * I, H), 0.02))
            s["w2"][e].copy_(_normal(g, (H, I), 0.02))
        s["residual"] = _normal(g, (M, H))
        s["norm"] = _normal(g, (H,), 0.05, 1.0)
    return s


# ---------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------
def _plain_norm(v, kind, w, b, offset):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    v = v * (w.float() + offset)
    return v if b is None else v + b.float()


def _plain_act(h, act):
    if act == "relu":
        return torch.where(h > 0, h, torch.zeros_like(h))
    if act == "silu":
        return h / (1.0 + torch.exp(-h))
    if act == "gelu":
        return 0.5 * h * (1.0 + torch.erf(h * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return h / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (h + 0.044715 * h * h * h)))
    return h


def _plain_select(logits, bias, c):
    """Experts and weights from logits in 64 bits (a choice between near scores needs them)."""
    M, E = logits.shape
    k, G = c["k"], c["n_group"]
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = p / p.sum(dim=1, keepdim=True)
    choice = score if bias is None else score + bias.double()
    order = logits if bias is None else choice        # without a bias the logits have the scores' order
    group = choice.view(M, G, E // G).topk(c["group_top"], dim=2).values.sum(dim=2)
    stay = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
    kept = torch.zeros((M, G), dtype=torch.bool, device=DEV).scatter_(1, stay, True)
    order = torch.where(kept.repeat_interleave(E // G, dim=1), order, -math.inf)
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_layer(s, c):
    M, I, k = c["M"], c["I"], c["k"]
    logits = s["x"].double() @ s["router"].double().T
    if s["router_bias"] is not None:
        logits = logits + s["router_bias"].double()
    ids, w = _plain_select(logits, s["select_bias"], c)
    x = s["x"].float()
    m = torch.zeros((M, c["H"]), dtype=torch.float32, device=DEV)
    for e in torch.unique(ids).tolist():              # one product for each expert that has tokens
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = x[t] @ s["w13"][e].float().T
        y = _plain_act(h[:, :I], "silu") * h[:, I:] @ s["w2"][e].float().T
        m.index_add_(0, t, y * w[t, j].unsqueeze(1))
    z = m + s["residual"].float()
    out = z * torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS) * s["norm"].float()
    return {"out": out.bfloat16(), "residual": z.bfloat16(), "ids": ids, "weights": w}


def _plain(s, c):
    if c["op"] == "norm":
        u = _plain_norm(s["y"].float(), c["post"], s["post_w"], s["post_b"], c["offset"])
        if s["gate"] is not None:
            u = u * s["gate"].float()
        z = c["a"] * s["residual"].float() + c["b"] * u
        out = _plain_norm(z, c["pre"], s["pre_w"], s["pre_b"], c["offset"])
        return {"out": out.bfloat16(), "z": z.to(s["residual"].dtype)}
    if c["op"] == "product":
        h = s["x"].float() @ s["w"].float().T
        if s["bias"] is not None:
            h = h + s["bias"].float()
        if c["gated"]:
            h = _plain_act(h[:, :c["N"]], c["act"]) * h[:, c["N"]:]
        else:
            h = _plain_act(h, c["act"])
        if s["residual"] is not None:
            h = h + s["residual"].float()
        return {"out": h.to(_dtype(c["f32"]))}
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
    if op == "norm":
        kinds = {"none": B.NORM_NONE, "rms": B.NORM_RMS, "layer": B.NORM_LAYER}
        out, z = new((M, c["H"]), torch.bfloat16), new((M, c["H"]), s["residual"].dtype)
        B.moe_block_norm(s["y"], s["residual"], out, z_out=z, gate=s["gate"],
                         post=kinds[c["post"]], post_w=s["post_w"], post_b=s["post_b"],
                         pre=kinds[c["pre"]], pre_w=s["pre_w"], pre_b=s["pre_b"], eps=EPS,
                         weight_offset=c["offset"], residual_scale=c["a"], block_scale=c["b"])
        return {"out": out, "z": z}
    if op == "product":
        acts = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "silu": B.ACT_SILU, "gelu": B.ACT_GELU,
                "gelu_tanh": B.ACT_GELU_TANH}
        out = new((M, c["N"]), _dtype(c["f32"]))
        B.moe_matmul(s["x"], s["w"], out, bias=s["bias"], act=acts[c["act"]], gated=c["gated"],
                     residual=s["residual"],
                     workspace=_room(s, B.moe_matmul_workspace_bytes(M, c["N"], c["K"], c["gated"])))
        return {"out": out}
    H, E, I, k = c["H"], c["E"], c["I"], c["k"]
    ids, w = new((M, k), torch.int32), new((M, k), torch.float32)
    out, z = new((M, H), torch.bfloat16), new((M, H), torch.bfloat16)
    B.moe_forward_few(s["x"], s["router"], s["router_bias"], s["w13"], s["w2"], s["residual"],
                      s["norm"], EPS, k, out, _room(s, B.moe_few_workspace_bytes(M, H, E, I, k)),
                      residual_out=z, topk_ids_out=ids, topk_w_out=w, select_bias=s["select_bias"],
                      score=B.SCORE_SIGMOID if c["score"] == "sigmoid" else B.SCORE_SOFTMAX,
                      n_group=c["n_group"], topk_group=c["topk_group"], group_top=c["group_top"],
                      renormalize=c["renorm"], scale=c["scale"])
    return {"out": out, "residual": z, "ids": ids, "weights": w}


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    M, op = case["M"], case["op"]
    if op == "norm":
        H = case["H"]
        gate = {"none": 0, "channel": H, "full": M * H, "token": M}[case["gate"]]
        weights = sum(H * (2 if case["bias"] else 1) for n in ("post", "pre") if case[n] != "none")
        value = (4 if case["y_f32"] else 2) + 2 * (4 if case["r_f32"] else 2) + 2
        return {"bytes": M * H * value + 2 * (gate + weights), "flops": 12 * M * H}
    if op == "product":
        N, K = case["N"], case["K"]
        rows = 2 * N if case["gated"] else N
        res = {"none": 0, "bf16": 2, "f32": 4}[case["res"]]
        return {"bytes": 2 * (M * K + rows * K) + (2 * rows if case["bias"] else 0) +
                M * N * (res + (4 if case["f32"] else 2)), "flops": 2 * M * rows * K}
    H, E, I, k = case["H"], case["E"], case["I"], case["k"]
    touched = E * (1.0 - (1.0 - k / E) ** M)          # experts that the picks are expected to touch
    biases = 4 * E * (int(case["select_bias"]) + int(case["router_bias"]))
    return {"bytes": 2 * (touched * 3 * H * I + E * H + 4 * M * H + H) + M * k * 8 + biases,
            "flops": 2 * M * E * H + 6 * M * k * H * I}


# ---------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_norm(v, kind, w, b, offset):
    if kind == "none":
        return v
    H = v.shape[1]
    if kind == "layer":
        v = v - v.sum(dim=1)[:, None] / H
    root = torch.sqrt(torch.linalg.vector_norm(v, dim=1) ** 2 / H + EPS)
    v = v / root[:, None] * (offset + w.double())[None, :]
    return v + b.double()[None, :] if b is not None else v


def _exact_act(h, act):
    if act == "relu":
        return torch.clamp(h, min=0.0)
    if act == "silu":
        return h * torch.sigmoid(h)
    if act == "gelu":
        return h * torch.special.ndtr(h)
    if act == "gelu_tanh":
        return h * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (h + 0.044715 * h ** 3))) / 2.0
    return h


def _exact_select(logits, bias, c):
    """Token by token: numpy, lexicographic sorts."""
    M, E = logits.shape
    k, G = c["k"], c["n_group"]
    per = E // G
    ids, w = np.empty((M, k), dtype=np.int64), np.zeros((M, k))
    index = np.arange(E)
    for t in range(M):
        v = logits[t]
        if c["score"] == "sigmoid":
            score = 1.0 / (1.0 + np.exp(-v))
        else:
            score = np.exp(v - v.max())
            score = score / score.sum()
        choice = score + bias if bias is not None else score
        totals = [np.sort(choice[n * per:(n + 1) * per])[::-1][:c["group_top"]].sum() for n in range(G)]
        chosen = np.lexsort((np.arange(G), -np.array(totals)))[:c["topk_group"]]
        key = choice if bias is not None else v
        ids[t] = np.lexsort((index, -key, ~np.isin(index // per, chosen)))[:k]
        got = score[ids[t]]
        w[t] = (got / got.sum() if c["renorm"] else got) * c["scale"]
    return ids, w


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "norm":
        u = _exact_norm(s["y"].double(), c["post"], s["post_w"], s["post_b"], c["offset"])
        if c["gate"] != "none":
            u = s["gate"].double() * u
        z = s["residual"].double() * c["a"] + u * c["b"]
        return {"out": _exact_norm(z, c["pre"], s["pre_w"], s["pre_b"], c["offset"]), "z": z}
    if op == "product":
        parts = s["w"].double().split(c["N"])          # gate and up rows, or all
        h = [torch.matmul(s["x"].double(), p.T.contiguous()) for p in parts]
        if c["bias"]:
            h = [a + b[None, :] for a, b in zip(h, s["bias"].double().split(c["N"]))]
        v = _exact_act(h[0], c["act"])
        if c["gated"]:
            v = v * h[1]
        return {"out": v + s["residual"].double() if c["res"] != "none" else v}
    logits = torch.matmul(s["x"].double(), s["router"].double().T.contiguous())
    if c["router_bias"]:
        logits = logits + s["router_bias"].double()[None, :]
    bias = s["select_bias"].double().cpu().numpy() if c["select_bias"] else None
    ids, w = _exact_select(logits.cpu().numpy(), bias, c)
    ids, w = torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
    z = s["residual"].double().clone()
    for t in range(c["M"]):
        for j in range(c["k"]):
            e = int(ids[t, j])
            h = s["w13"][e].double() @ s["x"][t].double()
            act = _exact_act(h[:c["I"]], "silu") * h[c["I"]:]
            z[t] += w[t, j] * (s["w2"][e].double() @ act)
    out = z / torch.sqrt((z * z).mean(dim=1, keepdim=True) + EPS) * s["norm"].double()
    return {"out": out, "residual": z, "ids": ids, "weights": w}
