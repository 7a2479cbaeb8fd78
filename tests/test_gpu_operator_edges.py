"""Grouped routing, int8 products and the int8 layer where they can go wrong by little: tighter
bounds than the shape grids', sums and scores at the ends of their types, kernels that only large
sizes reach.  Against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import _bars as bars
import moe_inputs as mi
from oracle import i8_oracle as orc
from oracle import moe_oracle
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


# ---------------------------------------------------------------------------------------
# The layer, code by code
# ---------------------------------------------------------------------------------------
def _quantize(B, v):
    codes = torch.full(tuple(v.shape), 99, dtype=torch.int8, device=v.device)
    scales = torch.full(tuple(v.shape[:-1]), float("nan"), dtype=torch.float32, device=v.device)
    B.moe_i8_quantize(v, codes, scales)
    return codes, scales


def _layer_reference(xq, xs, ids, weights, w13, s13, w2, s2):
    """m = sum of the weighted picks, and how far it may be off, for the rows given.

    Relative errors in units of u = 2^-24.  gate and up: the sum, the token's scale, the scales'
    product and the product of both round once each: 4.  silu(g) = g / (1 + exp(-g)) changes by
    at most 1 + |g| times what g does; exp is exp2 of a rounded product (log2 e rounded too: 1.5
    |g|, and 2 of its own), 1 + exp and the product with g round once, the reciprocal is good
    to 2: 4 (1 + |g|) + 1.5 |g| + 2 + 1 + 1 + 2 = 5.5 |g| + 10.  times up (4, and 1 for the
    product): act 5.5 |g| + 15.  127 act / a, a an act itself: both, and 2 for the product and
    the division (the scale a / 127 one more).  A code may be the next one where its quotient is
    that near to a border.  A result: the sum, the scales' product, and both's product round: 3,
    the scale's own error, and the code's; the weighted sum rounds 2 k times more, the weight
    once (and once in the division that made it)."""
    u = 2.0 ** -24
    n, k = ids.shape
    H = xq.shape[1]
    I = w13.shape[1] // 2
    m, tol, terms = np.zeros((n, H)), np.zeros((n, H)), np.zeros((n, H))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        h = orc.matmul(xq[t], xs[t], w13[e], s13[e])
        g = h[:, :I]
        act = g / (1.0 + np.exp(-g)) * h[:, I:]
        off = 5.5 * np.abs(g) + 15.0
        at = np.abs(act).argmax(axis=1)[:, None]
        top_off = np.take_along_axis(off, at, 1)
        q = 127.0 * act / np.abs(np.take_along_axis(act, at, 1))
        off = np.abs(q) * (off + top_off + 2.0) * u
        near = np.abs(np.abs(q - np.rint(q)) - 0.5) <= off
        codes, scale = orc.quantize(act)
        wt = weights[t, j][:, None]
        y = orc.matmul(codes, scale, w2[e], s2[e])
        moved = (near.astype(np.float64) @ np.abs(w2[e].astype(np.float64)).T) * scale[:, None] * s2[e][None, :]
        np.add.at(m, t, wt * y)
        np.add.at(terms, t, np.abs(wt * y))
        np.add.at(tol, t, np.abs(wt) * (np.abs(y) * (top_off + 1 + 3) * u + moved))
    return m, tol + terms * (2 * k + 3) * u


def _check_z(got, m, tol, residual):
    """z = m + residual, rounded to bf16: half a unit of the last place, at the largest it may be."""
    z = m + residual
    tol = tol + 2.0 ** -24 * (np.abs(z) + tol)
    err = np.abs(got.double().cpu().numpy() - z)
    bound = tol + 0.5 * bars.bf16_ulp(np.abs(z) + tol)
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.size} off, {err[worst]:.3e} at {worst}, bound {bound[worst]:.3e}"


@pytest.mark.parametrize("M,H,E,I,k,block", [(3, 256, 8, 2048, 4, 16), (40, 656, 4, 768, 2, 16),
                                             (64, 272, 12, 48, 3, 32), (205, 768, 4, 1408, 1, 16),
                                             (450, 784, 4, 784, 2, 16), (300, 400, 8, 256, 3, 64),
                                             (9, 512, 3, 8208, 2, 16),
                                             # more than 2^24 results of the down product
                                             (1100, 4096, 4, 640, 4, 64), (200, 16384, 8, 16, 8, 16)])
def test_layer_is_off_only_by_codes_at_a_border(B, dev, M, H, E, I, k, block):
    """No residual, so that sums near 0 show what the bf16 rounding of others hides.  Of many
    tokens the first, the last and some between are compared."""
    g = torch.Generator(device=dev).manual_seed(M + I)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=dev) * std  # noqa: E731
    x, wr = n(M, H).bfloat16(), n(E, H, std=1.7 / H ** 0.5).bfloat16()
    w13, s13 = _quantize(B, n(E, 2 * I, H, std=1.0 / H ** 0.5).bfloat16())
    w2, s2 = _quantize(B, n(E, H, I, std=1.0 / I ** 0.5).bfloat16())
    zero, one = torch.zeros(M, H, dtype=torch.bfloat16, device=dev), torch.ones(H, dtype=torch.bfloat16, device=dev)
    out, z = torch.empty_like(zero), torch.full_like(zero, float("nan"))
    ids = torch.full((M, k), -7, dtype=torch.int32, device=dev)
    w = torch.full((M, k), float("nan"), device=dev)
    ws = torch.full((B.moe_i8_workspace_bytes(M, H, E, I, k, block),), 0xFF, dtype=torch.uint8, device=dev)
    B.moe_forward_i8(x, wr, None, w13, s13, w2, s2, zero, one, 1e-5, k, block, out, ws, residual_out=z,
                     topk_ids_out=ids, topk_w_out=w)
    torch.cuda.synchronize()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    rid, rw = orc.route(bits(x), bits(wr), None, k)
    assert np.array_equal(ids.cpu().numpy(), rid)
    at = np.unique(np.linspace(0, M - 1, 60).astype(int)) if M * H > 1 << 20 else np.arange(M)
    xq, xs = orc.quantize(bf16_to_f64(bits(x))[at])
    m, tol = _layer_reference(xq, xs, rid[at], f64(w)[at], w13.cpu().numpy(), f64(s13), w2.cpu().numpy(), f64(s2))
    _check_z(z[torch.from_numpy(at).to(dev)], m, tol, 0.0)


# ---------------------------------------------------------------------------------------
# Routing: scores and sums at the ends of their types
# ---------------------------------------------------------------------------------------
def _rule(rule):
    r = dict(softmax=False, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0)
    r.update(rule)
    return r, dict({n: v for n, v in r.items() if n != "softmax"}, score=1 if r["softmax"] else 0)


def _picks(M, k, dev):
    return (torch.full((M, k), -7, dtype=torch.int32, device=dev),
            torch.full((M, k), float("nan"), dtype=torch.float32, device=dev))


def _from_logits(B, l, bias, k, rule):
    ids, w = _picks(l.shape[0], k, l.device)
    B.moe_route_logits(l, bias, k, ids, w, **_rule(rule)[1])
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.double().cpu().numpy()


def _from_hidden(B, x, wr, bias, k, rule):
    M, E = x.shape[0], wr.shape[0]
    ids, w = _picks(M, k, x.device)
    ws = torch.full((B.moe_route_groups_workspace_bytes(M, E),), 0xFF, dtype=torch.uint8, device=x.device)
    B.moe_route_groups(x, wr, bias, k, ids, w, ws, **_rule(rule)[1])
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.double().cpu().numpy()


def test_softmax_groups_far_below_the_top_by_hand(B, dev):
    """exp(-87.5) is no normal number in fp32 any more, but a fifth of group 2's sum, which
    makes it the larger one: exp(-86) (1 + exp(-1.5)) against exp(-85.95) (1 + exp(-9.05))."""
    l = torch.tensor([[0.0, -300.0, -300.0, -301.0, -86.0, -87.5, -85.95, -95.0]], device=dev) + 3.0
    ids, _ = _from_logits(B, l, None, 4, dict(softmax=True, n_group=4, topk_group=2, group_top=2))
    assert ids.tolist() == [[0, 4, 5, 1]]


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("renormalize", [False, True])
def test_softmax_groups_far_below_the_top(B, dev, group_top, renormalize):
    rule = dict(softmax=True, n_group=8, topk_group=3, group_top=group_top, renormalize=renormalize)
    g = torch.Generator().manual_seed(5 + group_top)
    l = torch.rand(400, 64, generator=g) * 3.0 + (3.0 - 88.8)
    l[:, 9] = 3.0
    ids, w = _from_logits(B, l.to(dev), None, 20, rule)
    rid, rw = orc.route_logits(l.numpy(), None, 20, **_rule(rule)[0])
    assert np.array_equal(ids, rid)
    assert (np.abs(w - rw) <= 2.0 ** -23 * rw + 2.0 ** -149).all()


@pytest.mark.parametrize("M", [200, 1300])
def test_softmax_groups_far_below_the_top_from_hidden_states(B, dev, M):
    """The first values of x raise expert 9's logit to about 87 above the others' at M from fp64
    sums and from bounded ones."""
    rule = dict(softmax=True, n_group=8, topk_group=3, group_top=2)
    g = torch.Generator(device=dev).manual_seed(M)
    x = torch.randn(M, 264, generator=g, device=dev)
    x[:, :8] = 1.0
    wr = torch.randn(64, 264, generator=g, device=dev) * (0.7 / 16)
    wr[:, :8] = 0.0
    wr[9, :8] = 87.0 / 8
    x, wr = x.bfloat16(), wr.bfloat16()
    ids, _ = _from_hidden(B, x, wr, None, 20, rule)
    rid, _ = orc.route(bits(x), bits(wr), None, 20, **_rule(rule)[0])
    assert np.array_equal(ids, rid)


@pytest.mark.parametrize("E,masked", [(8, 0), (96, 0), (96, 90), (512, 0)])
@pytest.mark.parametrize("scale", [1.0, 2.5, -3.0])
def test_weights_of_scores_next_to_zero(B, dev, E, masked, scale):
    """Scores of e^-709 to e^-716 are numbers in 64 bits, but 1 over their sum is none: sigmoid
    scores, and softmax scores of picks that a bias prefers to the token's best expert."""
    g = torch.Generator().manual_seed(E)
    k = min(E - masked, 4)
    l = torch.full((50, E), -float("inf"))
    l[:, masked:] = torch.rand(50, E - masked, generator=g) * 0.5 - 709.4
    rule = dict(scale=scale)
    for kk in {1, k, k + (1 if masked else 0)}:
        ids, w = _from_logits(B, l.to(dev), None, kk, rule)
        rid, rw = orc.route_logits(l.numpy(), None, kk, **_rule(rule)[0])
        assert np.array_equal(ids, rid)
        assert (np.abs(w - rw) <= 2.0 ** -23 * np.abs(rw)).all()
    l[:, masked:] = torch.rand(50, E - masked, generator=g) * 5.0 - 716.0
    l[:, E - 1] = 0.0
    bias = torch.zeros(E)
    bias[E - 1] = -2.0
    bias[:E - 1] = torch.rand(E - 1, generator=g)
    rule = dict(softmax=True, scale=scale)
    ids, w = _from_logits(B, l.to(dev), bias.to(dev), k - 1, rule)
    rid, rw = orc.route_logits(l.numpy(), bias.numpy(), k - 1, **_rule(rule)[0])
    assert np.array_equal(ids, rid)
    assert (np.abs(w - rw) <= 2.0 ** -23 * np.abs(rw)).all()


@pytest.mark.parametrize("rule", [dict(), dict(renormalize=False, scale=2.5), dict(softmax=True),
                                  dict(softmax=True, renormalize=False),
                                  dict(n_group=8, topk_group=4, group_top=2, scale=2.5),
                                  dict(n_group=8, topk_group=3, softmax=True, renormalize=False)])
@pytest.mark.parametrize("M,H,E,k", [(8, 7168, 256, 16), (300, 7168, 256, 16), (1300, 264, 64, 6), (170, 1032, 480, 8)])
@pytest.mark.parametrize("biased", [False, True])
def test_weights_of_logits_that_fp32_holds(B, dev, M, H, E, k, rule, biased):
    """Whole numbers times 2^-7 whose sums stay below 2^24 of it: fp32 sums are exact in any
    order, so the weights may be off by their own rounding only (2^-24, doubled for the 64-bit
    arithmetic before it), from fp64 logits and from bounded ones.  Many logits tie."""
    g = torch.Generator(device=dev).manual_seed(M + E)
    n = lambda *s: torch.randint(-4, 5, s, generator=g, device=dev).float()  # noqa: E731
    x, wr = n(M, H).bfloat16(), (n(E, H) * 2.0 ** -7).bfloat16()
    bias = torch.randn(E, generator=g, device=dev) * 0.05 if biased else None
    ids, w = _from_hidden(B, x, wr, bias, k, rule)
    rid, rw = orc.route(bits(x), bits(wr), None if bias is None else bias.cpu().numpy(), k, **_rule(rule)[0])
    assert np.array_equal(ids, rid)
    assert (np.abs(w - rw) <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149).all()


@pytest.mark.parametrize("M", [5, 300, 1300, 2600])
@pytest.mark.parametrize("rule", [dict(), dict(softmax=True), dict(n_group=4, topk_group=2, group_top=2),
                                  dict(n_group=4, topk_group=2, softmax=True, renormalize=False)])
@pytest.mark.parametrize("biased", [False, True])
def test_tokens_that_are_not_finite_stay_by_themselves(B, dev, M, rule, biased):
    """The other tokens get what they get beside finite ones, bit by bit, and the exact ids (M * 32
    logits: from 64-bit sums and, of 1,300 and 2,600 tokens, from bounded ones)."""
    g = torch.Generator(device=dev).manual_seed(M)
    x = torch.randn(M, 256, generator=g, device=dev).bfloat16()
    wr = (torch.randn(32, 256, generator=g, device=dev) * (1.7 / 16)).bfloat16()
    bias = torch.randn(32, generator=g, device=dev) * 0.05 if biased else None
    ids, w = _from_hidden(B, x, wr, bias, 5, rule)
    rid, _ = orc.route(bits(x), bits(wr), None if bias is None else bias.cpu().numpy(), 5, **_rule(rule)[0])
    assert np.array_equal(ids, rid)
    odd = [t for t in (1, 2, 3, 65, 66, 129, 1290) if t < M]
    for i, t in enumerate(odd):
        if i % 3 == 0:
            x[t, 3] = float("nan")
        elif i % 3 == 1:
            x[t, :] = float("inf")
        else:
            x[t, 7] = -float("inf")
    ids2, w2 = _from_hidden(B, x, wr, bias, 5, rule)
    keep = np.setdiff1d(np.arange(M), odd)
    assert np.array_equal(ids2[keep], ids[keep]) and np.array_equal(w2[keep], w[keep])
    assert all(len(set(ids2[t])) == 5 and (0 <= ids2[t]).all() and (ids2[t] < 32).all() for t in odd)


@pytest.mark.parametrize("M", [200, 1300])
@pytest.mark.parametrize("power", [-130, -126, 100])
def test_hidden_states_next_to_zero(B, dev, M, power):
    """Subnormal bf16 values times large weights make ordinary logits; so do large ones.  From
    bounded logits a weight is within 2^-9 of itself by its own logit and by its divisor's each."""
    g = torch.Generator(device=dev).manual_seed(M)
    x = (torch.randn(M, 264, generator=g, device=dev) * 2.0 ** power).bfloat16()
    wr = ((torch.randn(64, 264, generator=g, device=dev) / 16).double() * 2.0 ** -power).bfloat16()
    if power == -130:
        wr = (torch.randn(64, 264, generator=g, device=dev) * 2.0 ** 124).bfloat16()
    for rule in (dict(), dict(softmax=True), dict(n_group=4, topk_group=2)):
        ids, w = _from_hidden(B, x, wr, None, 6, rule)
        rid, rw = orc.route(bits(x), bits(wr), None, 6, **_rule(rule)[0])
        assert np.array_equal(ids, rid)
        assert (np.abs(w - rw) <= 2 * 2.0 ** -9 * np.abs(rw) * (1 + 2.0 ** -6)).all()


# ---------------------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N", [(3, 40), (20, 40), (70, 300), (300, 300), (2112, 1024)])
def test_matmul_sums_of_the_lowest_codes(B, dev, M, N, f32):
    """Rows of one code each, -128 among them, at the largest K: 128^2 K is 2^31.  (2112 x 1024
    takes the step stream.)  Roundings as in the other products: three of 2^-24, and the result's."""
    K = 131072
    av = (torch.arange(M, device=dev) % 3 - 1) * 127 - (torch.arange(M, device=dev) % 3 == 0).long()
    wv = (torch.arange(N, device=dev) % 5 - 2) * 63
    wv[::2] = -128
    wv[1::4] = 127
    a = av.to(torch.int8)[:, None].expand(M, K).contiguous()
    w = wv.to(torch.int8)[:, None].expand(N, K).contiguous()
    sa, sw = torch.rand(M, device=dev) + 0.5, torch.rand(N, device=dev) * 1e-4 + 1e-4
    out = torch.full((M, N), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    B.moe_i8_matmul(a, sa, w, sw, out)
    torch.cuda.synchronize()
    want = av.double()[:, None] * wv.double()[None, :] * K * sa.double()[:, None] * sw.double()[None, :]
    assert (want > 2.0 ** 31 * 0.5e-4).any()
    tol = (3.01 * 2.0 ** -24 + (0 if f32 else 2.0 ** -8)) * want.abs()
    assert ((out.double() - want).abs() <= tol).all()


def _codes(M, N, K, dev, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device=dev, dtype=torch.int8)  # noqa: E731
    return (code(M, K), torch.rand(M, generator=g, device=dev) + 0.01, code(N, K),
            torch.rand(N, generator=g, device=dev) * 1e-4 + 1e-6)


# step streams of 64, 128 and 256 token rows, whole last chunks of K and partial ones
STREAMS = [(4100, 513, 640), (900, 4097, 2048), (3000, 2300, 1024), (5000, 1537, 2048), (3500, 2500, 768),
           (2500, 1300, 656), (3000, 2300, 1040), (5000, 1537, 2064)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", STREAMS)
def test_matmul_step_streams(B, dev, M, N, K, f32):
    """Exact sums (in float64), three roundings of 2^-24 and the result's; nothing written
    around the result."""
    a, sa, w, sw = _codes(M, N, K, dev, M + K)
    guard = 64
    flat = torch.full((M * N + 2 * guard,), 77.0, dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    out = flat[guard:guard + M * N].view(M, N)
    B.moe_i8_matmul(a, sa, w, sw, out)
    torch.cuda.synchronize()
    want = (a.double() @ w.double().T.contiguous()) * sa.double()[:, None] * sw.double()[None, :]
    tol = (3.01 * 2.0 ** -24 + (0 if f32 else 2.0 ** -8)) * want.abs()
    assert ((out.double() - want).abs() <= tol).all()
    assert (flat[:guard] == 77.0).all() and (flat[-guard:] == 77.0).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", [(2500, 1300, 640), (3000, 2300, 1024), (3500, 2500, 768), (3000, 2300, 1040)])
def test_matmul_step_streams_in_a_graph(B, dev, M, N, K, f32):
    a, sa, w, sw = _codes(M, N, K, dev, 1)
    out = torch.zeros(M, N, dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    other = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.moe_i8_matmul(a, sa, w, sw, out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_i8_matmul(a, sa, w, sw, out)
    for seed in range(4):
        fresh = _codes(M, N, K, dev, 30 + seed)
        a.copy_(fresh[0])
        sa.copy_(fresh[1])
        out.zero_()
        B.moe_i8_matmul(fresh[0], fresh[1], w, sw, other)     # eager work between replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, other)


# ---------------------------------------------------------------------------------------
# Offsets that pass 32 bits
# ---------------------------------------------------------------------------------------
def test_quantize_more_than_four_billion_values(B, dev):
    K, part = 65536, 4097
    v = torch.randn(part, K, generator=torch.Generator(device=dev).manual_seed(1), device=dev).bfloat16()
    want = _quantize(B, v)
    codes, scales = _quantize(B, v.repeat(17, 1))
    for i in range(17):
        at = slice(i * part, (i + 1) * part)
        assert torch.equal(codes[at], want[0]) and torch.equal(scales[at], want[1])


@pytest.mark.parametrize("M,N,K", [(70000, 256, 65536), (40, 70000, 65536), (70000, 65536, 64)])
def test_matmul_past_32_bits(B, dev, M, N, K):
    """More than 2^32 codes of tokens, of weights, and results: rows that repeat give the results
    of the rows that they repeat."""
    a, sa, w, sw = _codes(min(M, 7000), min(N, 7000), K, dev, 5)
    want = (a.double() @ w.double().T.contiguous()) * sa.double()[:, None] * sw.double()[None, :]
    ra, rw = -(-M // a.shape[0]), -(-N // w.shape[0])
    big = (a.repeat(ra, 1)[:M].contiguous(), sa.repeat(ra)[:M].contiguous(), w.repeat(rw, 1)[:N].contiguous(),
           sw.repeat(rw)[:N].contiguous())
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev)
    B.moe_i8_matmul(*big, out)
    torch.cuda.synchronize()
    tol = (3.01 * 2.0 ** -24 + 2.0 ** -8) * want.abs()
    for m in range(0, M, a.shape[0]):
        for n in range(0, N, w.shape[0]):
            got = out[m:m + a.shape[0], n:n + w.shape[0]].double()
            i, j = got.shape
            assert ((got - want[:i, :j]).abs() <= tol[:i, :j]).all()


def test_layer_next_to_its_most_values(B, dev):
    """M * H just below 2^32, and more than that many bytes of everything between."""
    part, times, H, E, I, k, block = 65535, 16, 4096, 4, 16, 1, 64
    g = torch.Generator(device=dev).manual_seed(3)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=dev) * std  # noqa: E731
    x, wr = n(part, H).bfloat16(), n(E, H, std=1.7 / H ** 0.5).bfloat16()
    w13, s13 = _quantize(B, n(E, 2 * I, H, std=1.0 / H ** 0.5).bfloat16())
    w2, s2 = _quantize(B, n(E, H, I, std=1.0 / I ** 0.5).bfloat16())
    one = torch.ones(H, dtype=torch.bfloat16, device=dev)

    def run(x):
        M = x.shape[0]
        out, ids = torch.full_like(x, float("nan")), torch.full((M, k), -7, dtype=torch.int32, device=dev)
        ws = torch.empty(B.moe_i8_workspace_bytes(M, H, E, I, k, block), dtype=torch.uint8, device=dev)
        B.moe_forward_i8(x, wr, None, w13, s13, w2, s2, x, one, 1e-5, k, block, out, ws, topk_ids_out=ids)
        torch.cuda.synchronize()
        return out, ids

    want, wids = run(x)
    assert torch.isfinite(want.float()).all()
    out, ids = run(x.repeat(times, 1))
    for i in range(times):
        at = slice(i * part, (i + 1) * part)
        assert torch.equal(ids[at], wids) and torch.equal(out[at], want)
