"""Grouped expert routing on the GPU against the 64-bit oracle: ids bit for bit, weights.

Weights: a logit from fp32 sums carries at most n 2^-23 A (A = sum |x| |w|, n = 41 roundings
of a 256-wide part of the sum and of joining the parts), which moves a sigmoid, and a
softmax over its sum, by at most twice that much relative to itself, and the quotient over
the picks' sum by as much again; the result is rounded to fp32 (2^-24).  From given logits
the computation is fp64, so only the last rounding counts, doubled for fp64's own.
"""
import numpy as np
import pytest
import torch

import moe_inputs as mi
from oracle import i8_oracle as orc
from oracle.moe_oracle import bf16_to_f64

pytestmark = pytest.mark.gpu
bits = mi.bf16_bits


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def B(dev):
    from prefill_sigmoid_router_amd import binding
    binding.load_library()
    return binding


def _rule(rule):
    r = dict(softmax=False, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0)
    r.update(rule)
    api = {k: v for k, v in r.items() if k != "softmax"}
    api["score"] = 1 if r["softmax"] else 0
    return r, api


def _buffers(M, k, dev):
    return (torch.full((M, k), -7, dtype=torch.int32, device=dev),
            torch.full((M, k), float("nan"), dtype=torch.float32, device=dev))


def _run_logits(B, l, bias, k, rule, dev):
    r, api = _rule(rule)
    ids, w = _buffers(l.shape[0], k, dev)
    B.moe_route_logits(l, bias, k, ids, w, **api)
    torch.cuda.synchronize()
    return ids, w


def _check_logits(B, l, bias, k, rule, dev):
    ids, w = _run_logits(B, l, bias, k, rule, dev)
    r, _ = _rule(rule)
    rid, rw = orc.route_logits(l.cpu().numpy(), None if bias is None else bias.cpu().numpy(), k, **r)
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = w.cpu().numpy().astype(np.float64)
    assert (np.abs(got - rw) <= 2 ** -23 * np.abs(rw) + 1e-44).all()


RULES = [
    dict(), dict(softmax=True), dict(renormalize=False, scale=2.5),
    dict(n_group=4, topk_group=2, group_top=2), dict(n_group=4, topk_group=3, softmax=True),
    dict(n_group=2, topk_group=1, group_top=2, softmax=True, renormalize=False, scale=16.0),
    dict(n_group=4, topk_group=4),
]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("M,E,k", [(1, 8, 2), (5, 60, 4), (67, 64, 7), (33, 160, 6), (130, 256, 16),
                                   (9, 384, 8), (3, 512, 40), (4, 1024, 70)])
@pytest.mark.parametrize("biased", [False, True])
def test_logits(B, dev, M, E, k, rule, biased):
    g = torch.Generator().manual_seed(E * 31 + k)
    l = (torch.randn(M, E, generator=g) * 2).to(dev)
    bias = (torch.randn(E, generator=g) * 0.1).to(dev) if biased else None
    _check_logits(B, l, bias, k, rule, dev)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("share", [0.3, 0.95, 1.0])
def test_masked_logits(B, dev, rule, share):
    M, E, k = 50, 96, 8
    g = torch.Generator().manual_seed(11)
    l = torch.randn(M, E, generator=g) * 2
    l[torch.rand(M, E, generator=g) < share] = -float("inf")
    l[0] = -float("inf")
    l[1, :50] = float("nan")
    l[2, 7] = float("inf")
    bias = (torch.randn(E, generator=g) * 0.5).to(dev)
    for b in (None, bias):
        _check_logits(B, l.to(dev), b, k, rule, dev)


@pytest.mark.parametrize("rule", RULES)
def test_ties_go_to_the_lower_index(B, dev, rule):
    g = torch.Generator().manual_seed(5)
    l = torch.randint(-2, 3, (40, 128), generator=g).float()
    l[3] = 0.0
    l[4] = -0.0
    l[5, ::2] = -0.0
    l[5, 1::2] = 0.0
    bias = (torch.randint(0, 2, (128,), generator=g).float()).to(dev)
    for b in (None, bias):
        _check_logits(B, l.to(dev), b, 9, rule, dev)


def test_every_expert_picked_and_one_expert(B, dev):
    l = torch.randn(7, 48, generator=torch.Generator().manual_seed(1)).to(dev)
    _check_logits(B, l, None, 48, dict(softmax=True, renormalize=False), dev)
    _check_logits(B, l, None, 12, dict(n_group=4, topk_group=1, group_top=2), dev)
    _check_logits(B, l[:, :1].contiguous(), None, 1, dict(), dev)
    _check_logits(B, l, None, 16, dict(n_group=48, topk_group=16), dev)
    big = torch.randn(2, 1024, generator=torch.Generator().manual_seed(2)).to(dev)
    _check_logits(B, big, None, 1024, dict(softmax=True), dev)
    _check_logits(B, big, None, 100, dict(n_group=64, topk_group=30, group_top=2), dev)


def test_rows_of_a_wider_tensor(B, dev):
    wide = torch.randn(21, 200, generator=torch.Generator().manual_seed(4)).to(dev)
    part = wide[:, 33:97]
    ids, w = _run_logits(B, part, None, 6, {}, dev)
    ids2, w2 = _run_logits(B, part.contiguous(), None, 6, {}, dev)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    with pytest.raises(ValueError):
        B.moe_route_logits(wide.t(), None, 3, *_buffers(200, 3, dev))


def _run_x(B, x, wr, bias, k, rule, dev, stream=None, ws=None):
    M, E = x.shape[0], wr.shape[0]
    _, api = _rule(rule)
    ids, w = _buffers(M, k, dev)
    if ws is None:
        ws = torch.full((B.moe_route_groups_workspace_bytes(M, E),), 0xFF, dtype=torch.uint8, device=dev)
    B.moe_route_groups(x, wr, bias, k, ids, w, ws, stream=stream, **api)
    torch.cuda.synchronize()
    return ids, w


def _check_x(B, x, wr, bias, k, rule, dev):
    ids, w = _run_x(B, x, wr, bias, k, rule, dev)
    r, _ = _rule(rule)
    rid, rw = orc.route(bits(x), bits(wr), None if bias is None else bias.cpu().numpy(), k, **r)
    assert np.array_equal(ids.cpu().numpy(), rid)
    A = np.abs(bf16_to_f64(bits(x))) @ np.abs(bf16_to_f64(bits(wr))).T
    tol = (4 * 41 * 2 ** -23 * A.max(axis=1) + 2 ** -24)[:, None] * np.abs(rw)
    assert (np.abs(w.cpu().numpy() - rw) <= tol + 1e-44).all()


def _inputs(M, H, E, dev, seed=0, std=1.7):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(M, H, generator=g, device=dev).bfloat16()
    wr = (torch.randn(E, H, generator=g, device=dev) * (std / H ** 0.5)).bfloat16()
    bias = torch.randn(E, generator=g, device=dev) * 0.05
    return x, wr, bias


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("M,H,E,k", [(1, 256, 8, 2), (7, 1032, 60, 4), (8, 7168, 256, 16),
                                     (300, 520, 64, 7), (515, 1024, 160, 6), (1025, 2048, 256, 16),
                                     (260, 264, 512, 16), (257, 8, 1024, 8), (701, 520, 64, 7),
                                     (130, 7168, 320, 8), (1300, 1032, 36, 5)])
@pytest.mark.parametrize("biased", [False, True])
def test_hidden_states(B, dev, M, H, E, k, rule, biased):
    x, wr, bias = _inputs(M, H, E, dev)
    _check_x(B, x, wr, bias if biased else None, k, rule, dev)


@pytest.mark.parametrize("M", [9, 400, 900])
@pytest.mark.parametrize("rule", RULES)
def test_equal_and_nearly_equal_router_rows(B, dev, M, rule):
    """Exact ties, rows one bf16 step apart in one value, zero tokens."""
    x, wr, bias = _inputs(M, 512, 96, dev, seed=3)
    wr[48:] = wr[:48]
    wr[60:72] = wr[:12]
    near = wr[72:80].view(torch.int16)
    near[:, 5] += 1
    x[2] = 0.0
    bias = bias.clone()
    bias[48:] = bias[:48]
    for b in (None, bias):
        _check_x(B, x, wr, b, 8, rule, dev)


@pytest.mark.parametrize("M", [6, 300, 1300])
def test_all_router_rows_equal(B, dev, M):
    x, wr, bias = _inputs(M, 256, 64, dev, seed=8)
    wr[:] = wr[0]
    for rule in RULES:
        _check_x(B, x, wr, None, 4, rule, dev)


@pytest.mark.parametrize("M", [5, 300, 2600])
def test_tokens_that_are_not_finite_get_valid_ids(B, dev, M):
    x, wr, bias = _inputs(M, 256, 32, dev, seed=9)
    x[1, 3] = float("nan")
    x[2, :] = float("inf")
    x[3, 7] = -float("inf")
    for rule in RULES:
        ids, w = _run_x(B, x, wr, bias, 5, rule, dev)
        i = ids.cpu().numpy()
        assert ((i >= 0) & (i < 32)).all()
        assert all(len(set(row)) == 5 for row in i)
        clean = [t for t in range(M) if t not in (1, 2, 3)]
        ids2, w2 = _run_x(B, x[clean].contiguous(), wr, bias, 5, rule, dev)
        if M < 256:     # (the many-token path ends at 256)
            assert torch.equal(ids[clean], ids2) and torch.equal(w[clean], w2)


@pytest.mark.parametrize("M", [300, 1300])
def test_large_values(B, dev, M):
    """Logits in the hundreds: sigmoids at 1, softmax with one expert at 1."""
    x, wr, bias = _inputs(M, 1024, 64, dev, seed=10, std=150.0)
    for rule in (dict(softmax=True), dict(), dict(n_group=4, topk_group=2)):
        _check_x(B, x, wr, None, 4, rule, dev)


@pytest.mark.parametrize("rule", [dict(), dict(renormalize=False), dict(softmax=True),
                                  dict(softmax=True, renormalize=False),
                                  dict(n_group=4, topk_group=2, group_top=2)])
@pytest.mark.parametrize("size", [100.0, 20000.0])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("M", [300, 1300])
def test_weights_where_large_terms_cancel(B, dev, M, rule, size, biased):
    """Two halves of the row whose products cancel but for ordinary logits: the fp32 sums are
    off by parts of the terms' size.  A weight may be off by twice 2^-9 of itself: 2^-9 from
    its own logit, 2^-9 from those of what it is divided by."""
    x, wr, bias = _inputs(M, 1024, 64, dev, seed=12)
    x[:, 256:512] = size / 256
    x[:, 768:] = -size / 256
    wr[:, 256:512] = wr[:, 768:] = 1.0
    b = bias if biased else None
    ids, w = _run_x(B, x, wr, b, 6, rule, dev)
    r, _ = _rule(rule)
    rid, rw = orc.route(bits(x), bits(wr), None if b is None else b.cpu().numpy(), 6, **r)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(w.cpu().numpy() - rw) <= 2 * 2 ** -9 * np.abs(rw) * (1 + 2 ** -6)).all()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("M", [8, 512, 1300])
def test_graph_replays_equal_eager_calls(B, dev, M, softmax):
    rule = dict(n_group=4, topk_group=2, group_top=2, scale=2.5, softmax=softmax)
    _, api = _rule(rule)
    x, wr, bias = _inputs(M, 512, 64, dev, seed=1)
    k = 6
    ids, w = _buffers(M, k, dev)
    ws = torch.empty(B.moe_route_groups_workspace_bytes(M, 64), dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.moe_route_groups(x, wr, bias, k, ids, w, ws, **api)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_route_groups(x, wr, bias, k, ids, w, ws, **api)
    for seed in range(4):
        fresh, _, _ = _inputs(M, 512, 64, dev, seed=20 + seed)
        x.copy_(fresh)
        ids.fill_(-7)
        w.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = _run_x(B, fresh, wr, bias, k, rule, dev)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])


@pytest.mark.parametrize("more", [0, 1000])
@pytest.mark.parametrize("softmax", [False, True])
def test_two_streams_at_once(B, dev, more, softmax):
    rule = dict(n_group=4, topk_group=2, group_top=2, softmax=softmax)
    a, b = _inputs(700 + more, 1024, 64, dev, seed=1), _inputs(300 + more, 1024, 64, dev, seed=2)
    want = [_run_x(B, v[0], v[1], v[2], 6, rule, dev) for v in (a, b)]
    torch.cuda.synchronize()
    _, api = _rule(rule)
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for v, s in zip((a, b), streams):
        M = v[0].shape[0]
        o = _buffers(M, 6, dev) + (torch.empty(B.moe_route_groups_workspace_bytes(M, 64),
                                               dtype=torch.uint8, device=dev),)
        outs.append(o)
    torch.cuda.synchronize()
    for _ in range(5):
        for v, s, o in zip((a, b), streams, outs):
            B.moe_route_groups(v[0], v[1], v[2], 6, o[0], o[1], o[2], stream=s, **api)
    torch.cuda.synchronize()
    for o, wv in zip(outs, want):
        assert torch.equal(o[0], wv[0]) and torch.equal(o[1], wv[1])


@pytest.mark.parametrize("rule", [dict(softmax=True), dict(softmax=True, n_group=4, topk_group=1)])
@pytest.mark.parametrize("same", [1400, 60])
def test_softmax_divisor_decides(B, dev, rule, same):
    """A bias that makes up for the difference of two experts' scores to fp32's last bit: their
    order hangs on every logit of the token, in few tokens and in nearly all."""
    x, wr, _ = _inputs(1400, 1024, 64, dev, seed=14)
    x[:same] = x[0]
    l = bf16_to_f64(bits(x[:1])) @ bf16_to_f64(bits(wr)).T
    p = np.exp(l[0] - l.max())
    p /= p.sum()
    bias = torch.zeros(64, device=dev)
    bias[int(p.argmin())] = float(p.max() - p.min())
    _check_x(B, x, wr, bias, 8, rule, dev)
