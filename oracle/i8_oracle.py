"""CPU oracle of grouped expert routing and of the 8-bit integer rows, products and layer.

TEST INFRASTRUCTURE ONLY, like moe_oracle: plain float64 numpy, no code of the library.

Routing: l = x Wr^T (or given logits); s = sigmoid(l) or softmax(l); c = s + b; a group's
score is the sum of its group_top largest c; topk_group groups stay (ties to the lower
group); the top_k largest c in them are picked (ties to the lower id; without a bias the
logits are compared); weights are s of the picks, divided by their sum if renormalize, times
scale.  Experts with a logit of -inf or NaN have no score: weight 0, last in their groups.

int8 rows: a = max |v|, scale a / 127, code = 127 v / a rounded to nearest even (Fractions:
exact).  A product is the exact integer sum times both scales.  The layer quantizes x and act row by row.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .moe_oracle import bf16_to_f64, finalize

__all__ = ["route_logits", "route", "quantize", "quantize_exact", "matmul", "round_bf16", "layer"]


def route_logits(logits, bias, top_k, softmax=False, n_group=1, topk_group=1, group_top=1,
                 renormalize=True, scale=1.0):
    """ids [M, k] int32, weights [M, k] float64."""
    l = np.asarray(logits, dtype=np.float64)
    M, E = l.shape
    per = E // n_group
    b = None if bias is None else np.asarray(bias, dtype=np.float32).astype(np.float64)
    ids = np.empty((M, top_k), dtype=np.int32)
    w = np.zeros((M, top_k))
    for t in range(M):
        has = l[t] > -np.inf                     # False for NaN too
        s = np.zeros(E)
        if has.any():
            v = np.minimum(l[t][has], np.finfo(np.float64).max)
            if softmax:
                p = np.exp(v - v.max())
                s[has] = p / p.sum()
            else:
                s[has] = 1.0 / (1.0 + np.exp(-v))
        c = s if b is None else s + b
        group = np.full(n_group, -np.inf)
        for g in range(n_group):
            mine = np.sort(c[g * per:(g + 1) * per][has[g * per:(g + 1) * per]])[::-1]
            if mine.size:
                group[g] = mine[:group_top].sum()
        stay = sorted(range(n_group), key=lambda g: (-group[g], g))[:topk_group]
        inside = [e for g in sorted(stay) for e in range(g * per, (g + 1) * per)]
        key = l[t] if b is None else c
        scored = sorted((e for e in inside if has[e]), key=lambda e: (-key[e], e))
        picks = (scored + [e for e in inside if not has[e]])[:top_k]
        ids[t] = picks
        w[t] = s[picks]
        if renormalize:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
    return ids, w * float(scale)


def route(x_bits, router_w_bits, bias, top_k, **rule):
    return route_logits(bf16_to_f64(x_bits) @ bf16_to_f64(router_w_bits).T, bias, top_k, **rule)


def quantize_exact(row):
    """One row of floats -> (codes, scale as a Fraction), in exact arithmetic."""
    f = [Fraction(float(v)) for v in row]
    a = max(abs(v) for v in f)
    if a == 0:
        return [0] * len(f), Fraction(0)
    return [round(127 * v / a) for v in f], a / 127     # Fraction rounds half to even


def quantize(v):
    """Rows of float64 values -> codes int8 and scales float64.  For values with at most 8
    significant bits this equals quantize_exact: 127 v is exact, and so far from a tie when
    it is none that float64 division rounds to the same side."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v).max(axis=-1, keepdims=True)
    return np.rint(127.0 * v / np.where(a > 0, a, 1.0)).astype(np.int8), a[..., 0] / 127.0


def matmul(a, a_scale, w, w_scale):
    total = np.asarray(a, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T   # exact integers
    return total * np.asarray(a_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]


def round_bf16(v):
    """float64 -> the nearest bf16 (ties to even), as float64."""
    u = np.asarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def layer(x_bits, ids, weights, w13, w13_scale, w2, w2_scale, residual_bits, norm_w_bits, eps):
    """The layer after routing; w13 / w2 int8 codes [E, 2I, H] / [E, H, I] with their scales.
    Returns (out, z, y [M*k, H])."""
    xq, xs = quantize(bf16_to_f64(x_bits))
    M, k = ids.shape
    I = w13.shape[1] // 2
    y = np.zeros((M * k, xq.shape[1]))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        h = matmul(xq[t], xs[t], w13[e], w13_scale[e])
        act = h[:, :I] / (1.0 + np.exp(-h[:, :I])) * h[:, I:]
        aq, a_s = quantize(act)
        y[t * k + j] = matmul(aq, a_s, w2[e], w2_scale[e])
    out, z = finalize(y, weights, residual_bits, norm_w_bits, eps)
    return out, z, y
