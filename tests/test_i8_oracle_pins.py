"""Pins of oracle/i8_oracle.py that do not reuse its code, and the host checks of the new
entry points (no launch happens on these paths)."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import i8_oracle as o


@pytest.fixture(scope="module")
def lib():
    from prefill_sigmoid_router_amd import binding, build
    if not os.path.exists(binding.library_path()):
        build.build()
    return binding.load_library()


def test_quantize_equals_exact_arithmetic_for_bf16_values():
    rng = np.random.default_rng(3)
    for scale in (1.0, 1e-20, 1e20):
        v = o.round_bf16(rng.normal(0, scale, (40, 64)))
        v[0, :] = np.arange(-32, 32) * scale               # many exact ties
        v[1, :] = 0.0
        v[2, 1:] = np.repeat([254, 1, 3, 5, 253, 251, 127], 9) / 2 * scale
        v = o.round_bf16(v)
        codes, scales = o.quantize(v)
        for r in range(v.shape[0]):
            want, s = o.quantize_exact(v[r])
            assert codes[r].tolist() == want
            assert abs(float(s) - scales[r]) <= 2 ** -52 * float(s)


def test_route_by_hand():
    # four groups of two; sums of both scores; the bias decides between the groups
    l = np.array([[0.0, 0.0, 1.0, -1.0, 2.0, -9.0, 0.5, 0.5]])
    ids, w = o.route_logits(l, None, 2, n_group=4, topk_group=2, group_top=2, renormalize=False)
    # sums: 1.0, 1.0, 0.8809, 1.2449: groups 3 and 0 (the tie with 1 goes to the lower group)
    assert ids.tolist() == [[6, 7]]
    assert np.allclose(w, 1 / (1 + np.exp(-0.5)))
    ids, w = o.route_logits(l, np.array([0, 0, 0, 0, 5, 0, 0, 0.0]), 2, n_group=4, topk_group=1,
                            group_top=1, renormalize=True, scale=2.0)
    s = 1 / (1 + np.exp(-np.array([2.0, -9.0])))
    assert ids.tolist() == [[4, 5]] and np.allclose(w, 2.0 * s / s.sum())


def test_route_without_scores():
    inf = np.inf
    l = np.array([[-inf] * 4, [np.nan, 1.0, -inf, -inf], [-inf, -inf, 3.0, 3.0]])
    ids, w = o.route_logits(l, np.zeros(4), 2, softmax=True, n_group=2, topk_group=1, group_top=2)
    assert ids.tolist() == [[0, 1], [1, 0], [2, 3]]
    assert w.tolist() == [[0.0, 0.0], [1.0, 0.0], [0.5, 0.5]]


def test_softmax_weights_sum_to_one_over_all_experts():
    l = np.random.default_rng(0).normal(0, 3, (5, 12))
    ids, w = o.route_logits(l, None, 12, softmax=True, renormalize=False)
    assert np.allclose(w.sum(1), 1.0) and (np.diff(w, axis=1) <= 0).all()
    assert (np.sort(ids, axis=1) == np.arange(12)).all()


# ---------------------------------------------------------------------------------------
# Host checks of the entry points
# ---------------------------------------------------------------------------------------
P = ctypes.c_void_p


def _rule(kw):
    r = dict(E=8, k=2, score=0, G=2, kg=1, gt=2, renorm=1, scale=1.0)
    r.update({k: v for k, v in kw.items() if k in r})
    return r


RULE_REFUSALS = [dict(E=0), dict(E=1025), dict(k=0), dict(k=5), dict(score=2), dict(score=-1),
                 dict(G=0), dict(G=3), dict(G=65, E=65), dict(kg=0), dict(kg=3), dict(gt=0),
                 dict(gt=3), dict(gt=2, G=8), dict(scale=float("nan")), dict(scale=float("inf"))]


def _groups(lib, **kw):
    r = _rule(kw)
    a = dict(x=256, rw=256, bias=None, M=4, H=256, ids=256, w=256, ws=256, wsb=1 << 40)
    a.update({k: v for k, v in kw.items() if k in a})
    return lib.moe_route_groups(P(a["x"]), P(a["rw"]), P(a["bias"]), a["M"], a["H"], r["E"], r["k"],
                                r["score"], r["G"], r["kg"], r["gt"], r["renorm"], r["scale"],
                                P(a["ids"]), P(a["w"]), P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("bad,code", [(b, -1) for b in RULE_REFUSALS] + [
    (dict(M=-1), -1), (dict(H=4), -1), (dict(H=12), -1), (dict(H=16392), -1),
    (dict(M=1 << 30), -1), (dict(x=None), -1), (dict(x=8), -1), (dict(rw=None), -1),
    (dict(ids=None), -1), (dict(w=2), -1), (dict(bias=1), -1), (dict(ws=None), -3),
    (dict(ws=8), -3), (dict(wsb=64), -3)])
def test_route_groups_refuses_on_the_host(lib, bad, code):
    assert _groups(lib, **bad) == code


def _logits(lib, **kw):
    r = _rule(kw)
    a = dict(l=256, ld=8, bias=None, M=4, ids=256, w=256)
    a.update({k: v for k, v in kw.items() if k in a})
    return lib.moe_route_logits(P(a["l"]), a["ld"], P(a["bias"]), a["M"], r["E"], r["k"],
                                r["score"], r["G"], r["kg"], r["gt"], r["renorm"], r["scale"],
                                P(a["ids"]), P(a["w"]), None)


@pytest.mark.parametrize("bad", RULE_REFUSALS + [
    dict(M=-1), dict(ld=7), dict(ld=(1 << 32) + 1), dict(M=1 << 30), dict(l=None), dict(l=2),
    dict(ids=None), dict(ids=2), dict(w=None), dict(w=6), dict(bias=3)])
def test_route_logits_refuses_on_the_host(lib, bad):
    if "E" in bad:
        bad = dict(bad, ld=max(8, bad["E"]))
    assert _logits(lib, **bad) == -1


@pytest.mark.parametrize("a", [
    (256, -1, 32, 256, 256), (256, 4, 24, 256, 256), (256, 4, 0, 256, 256),
    (256, 4, 131088, 256, 256), (256, 1 << 40, 32, 256, 256), (None, 4, 32, 256, 256),
    (8, 4, 32, 256, 256), (256, 4, 32, 8, 256), (256, 4, 32, None, 256), (256, 4, 32, 256, None),
    (256, 4, 32, 256, 2)])
def test_i8_quantize_refuses_on_the_host(lib, a):
    assert lib.moe_i8_quantize(P(a[0]), a[1], a[2], P(a[3]), P(a[4]), None) == -1


def _matmul(lib, **kw):
    a = dict(a=256, sa=256, w=256, sw=256, M=4, N=8, K=32, out=256, f32=0, ws=256, wsb=1 << 40)
    a.update(kw)
    return lib.moe_i8_matmul(P(a["a"]), P(a["sa"]), P(a["w"]), P(a["sw"]), a["M"], a["N"], a["K"],
                             P(a["out"]), a["f32"], P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(K=0), dict(K=40), dict(K=131088), dict(f32=2), dict(a=None),
    dict(a=8), dict(sa=None), dict(sa=2), dict(w=8), dict(sw=4), dict(out=None), dict(out=8)])
def test_i8_matmul_refuses_on_the_host(lib, bad):
    assert _matmul(lib, **bad) == -1


def _forward(lib, **kw):
    r = _rule(kw)
    a = dict(x=256, rw=256, bias=None, c13=256, s13=256, c2=256, s2=256, res=256, g=256, eps=1e-5,
             M=4, H=256, I=512, block=16, out=256, rout=None, ws=256, wsb=1 << 40)
    a.update({k: v for k, v in kw.items() if k in a})
    return lib.moe_forward_i8(
        P(a["x"]), P(a["rw"]), P(a["bias"]), P(a["c13"]), P(a["s13"]), P(a["c2"]), P(a["s2"]),
        P(a["res"]), P(a["g"]), a["eps"], a["M"], a["H"], r["E"], a["I"], r["k"], a["block"],
        r["score"], r["G"], r["kg"], r["gt"], r["renorm"], r["scale"], P(a["out"]), P(a["rout"]),
        None, None, None, None, None, P(a["ws"]), a["wsb"], None, None)


@pytest.mark.parametrize("bad,code", [(b, -1) for b in RULE_REFUSALS] + [
    (dict(M=-1), -1), (dict(H=264), -1), (dict(I=24), -1), (dict(eps=0.0), -1),
    (dict(eps=float("nan")), -1), (dict(block=48), -2), (dict(x=None), -1), (dict(c13=8), -1),
    (dict(s13=4), -1), (dict(c2=None), -1), (dict(s2=8), -1), (dict(rout=8), -1), (dict(ws=64), -3),
    (dict(ws=None), -3), (dict(wsb=4096), -3)])
def test_forward_i8_refuses_on_the_host(lib, bad, code):
    assert _forward(lib, **bad) == code


@pytest.mark.parametrize("sizes", [dict(M=1 << 22, H=16, I=16), dict(M=1 << 19, H=8192, I=16),
                                   dict(M=1 << 21, H=16, I=16, E=64, k=32)])
def test_forward_i8_refuses_more_than_its_grids_hold(lib, sizes):
    a = dict(E=8, k=2)
    a.update(sizes)
    assert _forward(lib, **sizes) == -2
    assert lib.moe_i8_workspace_bytes(a["M"], a["H"], a["E"], a["I"], a["k"], 16) == 0


@pytest.mark.parametrize("bad", [dict(M=(1 << 30) + 1), dict(N=(1 << 26) + 1)])
def test_i8_matmul_refuses_more_than_its_grids_hold(lib, bad):
    assert _matmul(lib, **bad) == -1


def test_no_rows_is_a_success(lib):
    assert _groups(lib, M=0, x=None, ids=None, ws=None, wsb=0) == 0
    assert _logits(lib, M=0, l=None, ids=None) == 0
    assert lib.moe_i8_quantize(None, 0, 32, None, None, None) == 0
    assert _matmul(lib, M=0, a=None, out=None, ws=None) == 0
    assert _forward(lib, M=0, x=None, out=None, ws=None, wsb=0) == 0


def test_workspace_sizes(lib):
    M, H, E, I, k, blk = 2048, 7168, 256, 2048, 16, 64
    cap = lib.moe_align_capacity(M, k, E, blk)
    assert lib.moe_i8_workspace_bytes(M, H, E, I, k, blk) >= \
        lib.moe_workspace_bytes(M, H, E, I, k, blk) + M * H + cap * I + 4 * (M + cap)
    assert lib.moe_i8_workspace_bytes(M, H + 8, E, I, k, blk) == 0     # H % 16
    assert lib.moe_i8_workspace_bytes(M, H, E, I, k, 48) == 0
    assert lib.moe_route_groups_workspace_bytes(M, E) >= 8 * M * E
    assert lib.moe_route_groups_workspace_bytes(M, 2000) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    from prefill_sigmoid_router_amd import binding as B
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.moe_i8_quantize(x, torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(TypeError):
        B.moe_route_logits(x, None, 2, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        B.moe_route_logits(x.float(), None, 2, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
