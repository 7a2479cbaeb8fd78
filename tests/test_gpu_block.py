"""Block norm, bf16 products and the layer for a few tokens on the GPU against 64 bits.

Bounds count roundings: u = 2^-24 for one in fp32, 2^-8 for the last one to bf16 (2^-24 to fp32).
"""
import math

import numpy as np
import pytest
import torch

import moe_inputs as mi
from oracle import i8_oracle as orc

pytestmark = pytest.mark.gpu
bits = mi.bf16_bits
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


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


def _gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def _randn(g, shape, std=1.0, mean=0.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device=g.device) * std + mean).to(dtype)


class Rows:
    """[M, n] inside a larger buffer of 77s: `pad` values behind every row, a guard before and
    behind all of them."""

    def __init__(self, M, n, dtype, dev, pad=0, fill=None):
        self.flat = torch.full((128 + M * (n + pad),), 77.0, dtype=dtype, device=dev)
        self.t = self.flat[64:64 + M * (n + pad)].view(M, n + pad)[:, :n]
        if fill is not None:
            self.t.copy_(fill)

    def untouched(self):
        rest = self.flat.clone()
        M, n = self.t.shape
        if M:
            rest[64:-64].view(M, -1)[:, :n] = 77.0
        return bool((rest == 77.0).all())


def _round(dtype):
    return 2.0 ** -8 if dtype is BF16 else U


# ---------------------------------------------------------------------------------------
# Block norm
# ---------------------------------------------------------------------------------------
def _norm_ref(v, err, kind, w, b, offset, eps):
    """N(v) in 64 bits, and a bound of the kernel's error where its v is off by up to err.

    A sum over a row is a chain of at most 16 values a thread, 6 steps in the wave and 16 waves:
    40 roundings, of numbers of one sign for the squares.  Mean: off by dm = 42 u mean |v| and the
    mean of err.  The squares' mean m2 then is off by 45 u of itself, by the errors of its terms
    (2 |d| (err + dm)), and for the waves' means by 2 dm times the spread: (50 u + 4 (rms(err) + dm)
    / rms(d)) m2 in all; the root halves that, and root and quotient round once or twice (4 u).
    (v - m) f (offset + w) + b: 5 roundings more."""
    if kind == 0:
        return v, err
    if kind == 2:
        m = v.mean(dim=1, keepdim=True)
        dm = 42 * U * v.abs().mean(dim=1, keepdim=True) + err.mean(dim=1, keepdim=True)
        d = v - m
    else:
        d, dm = v, torch.zeros_like(v[:, :1])
    ms = (d * d).mean(dim=1, keepdim=True)
    f = 1.0 / torch.sqrt(ms + eps)
    rel = 29 * U + 2 * ((err * err).mean(dim=1, keepdim=True).sqrt() + dm) / torch.sqrt(ms + eps)
    g = 1.0 if w is None else offset + w.double()
    out = d * f * g
    off = ((err + dm) * f + (d * f).abs() * (rel + 5 * U)) * (abs(g) if w is None else g.abs())
    if b is not None:
        out = out + b.double()
        off = off + U * out.abs()
    return out, off


def _check_norm(B, dev, M, H, post=1, pre=1, gate="none", yt=BF16, rt=BF16, weights=True, bias=False,
                offset=0.0, a=1.0, b=1.0, pad=0, with_y=True, with_r=True, with_z=True, with_out=True,
                mean=0.0, eps=1e-5, seed=0):
    g = _gen(dev, seed + M * 7 + H)
    y = Rows(M, H, yt, dev, pad, _randn(g, (M, H), 1.0, mean, yt)) if with_y else None
    r = Rows(M, H, rt, dev, 2 * pad, _randn(g, (M, H), 3.0, 2 * mean, rt)) if with_r else None
    zt = rt if with_r else yt
    z = Rows(M, H, zt, dev, pad) if with_z else None
    out = Rows(M, H, BF16, dev, 3 * pad) if with_out else None
    vec = lambda on, m, s: _randn(g, (H,), s, m) if on else None  # noqa: E731
    pw, qw = vec(weights and post, 1.0 - offset, 0.05), vec(weights and pre, 1.0 - offset, 0.05)
    pb, qb = vec(bias and post, 0.0, 0.1), vec(bias and pre, 0.0, 0.1)
    gt = {"none": None, "channel": (H,), "full": (M, H), "token": (M, 1), "one": (1, 1)}[gate]
    gv = None if gt is None else _randn(g, gt, 0.3, 0.7)
    t = lambda x: None if x is None else x.t  # noqa: E731
    B.moe_block_norm(t(y), t(r), t(out), z_out=t(z), gate=gv, post=post, post_w=pw, post_b=pb, pre=pre,
                     pre_w=qw, pre_b=qb, eps=eps, weight_offset=offset, residual_scale=a, block_scale=b)
    torch.cuda.synchronize()
    zero = torch.zeros(M, H, dtype=torch.float64, device=dev)
    want, err = zero, zero
    if with_y:
        want, err = _norm_ref(y.t.double(), zero, post, pw, pb, offset, eps)
        want, err = b * want, abs(b) * err + 2 * U * (b * want).abs()
        if gv is not None:
            gd = gv.double() if gv.dim() == 2 else gv.double()[None, :]
            want, err = gd * want, gd.abs() * err + 2 * U * (gd * want).abs()
    if with_r:
        rd = a * r.t.double()
        err = err + U * rd.abs() + U * (want + rd).abs()
        want = want + rd
    for rows in (y, r, z, out):
        assert rows is None or rows.untouched()
    if with_z:
        off = (z.t.double() - want).abs()
        assert (off <= err + _round(zt) * (want.abs() + err)).all(), off.max().item()
    if with_out:
        w2, e2 = _norm_ref(want, err, pre, qw, qb, offset, eps)
        off = (out.t.double() - w2).abs()
        assert (off <= e2 + 2.0 ** -8 * (w2.abs() + e2)).all(), off.max().item()


@pytest.mark.parametrize("H", [8, 64, 200, 504, 512, 520, 1024, 2056, 4096, 7168, 8192, 8200, 16384])
@pytest.mark.parametrize("M", [1, 3, 70])
def test_norm_sizes(B, dev, M, H):
    _check_norm(B, dev, M, H)
    _check_norm(B, dev, M, H, post=2, pre=2, gate="full", yt=F32, rt=F32, bias=True, offset=1.0, a=0.5,
                b=0.25, pad=8)


@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("gate", ["none", "channel", "full", "token", "one"])
@pytest.mark.parametrize("H", [264, 1544])
def test_norm_kinds_and_gates(B, dev, post, pre, gate, H):
    _check_norm(B, dev, 9, H, post=post, pre=pre, gate=gate, bias=post == pre, pad=16)
    _check_norm(B, dev, 5, H, post=post, pre=pre, gate=gate, weights=False, yt=F32, a=-1.0)


@pytest.mark.parametrize("yt,rt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("H", [56, 3584, 10248])
def test_norm_parts_left_out(B, dev, yt, rt, H):
    _check_norm(B, dev, 6, H, yt=yt, rt=rt, with_r=False, pad=8)
    _check_norm(B, dev, 6, H, yt=yt, rt=rt, with_z=False)
    _check_norm(B, dev, 6, H, yt=yt, rt=rt, with_out=False)
    _check_norm(B, dev, 6, H, yt=yt, rt=rt, post=0, with_y=False)


@pytest.mark.parametrize("H", [512, 4096])
def test_norm_of_rows_far_from_zero(B, dev, H):
    """A LAYER norm of rows whose mean is 64 times their spread."""
    _check_norm(B, dev, 33, H, post=2, pre=2, yt=F32, rt=F32, mean=64.0)


def test_norm_many_rows(B, dev):
    _check_norm(B, dev, 70001, 16, pad=8)
    _check_norm(B, dev, 66000, 1032, rt=F32, gate="token")


def test_norm_in_place(B, dev):
    g = _gen(dev, 5)
    y, r, w = _randn(g, (40, 2048)), _randn(g, (40, 2048)), _randn(g, (2048,), 0.1, 1.0)
    out, z = torch.empty_like(y), torch.empty_like(r)
    B.moe_block_norm(y, r, out, z_out=z, post=1, post_w=w, pre=1, pre_w=w)
    y2, r2 = y.clone(), r.clone()
    B.moe_block_norm(y2, r2, y2, z_out=r2, post=1, post_w=w, pre=1, pre_w=w)
    torch.cuda.synchronize()
    assert torch.equal(y2, out) and torch.equal(r2, z)


def test_norm_rows_of_zeros_and_not_finite(B, dev):
    g = _gen(dev, 6)
    y, r = _randn(g, (5, 1024)), _randn(g, (5, 1024))
    y[1], r[1] = 0.0, 0.0
    y[2, 7], r[3, 9] = float("nan"), float("inf")
    out, z = torch.empty_like(y), torch.empty_like(y)
    B.moe_block_norm(y, r, out, z_out=z, post=2, pre=1)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all(1).tolist() == [True, True, False, False, True]
    assert (out[1] == 0).all() and (z[1] == 0).all()


def test_norm_offsets_past_32_bits(B, dev):
    """Rows whose offsets in values pass 2^32."""
    M, H, ld = 3, 64, (1 << 31) + 64
    flat = torch.empty(2 * ld + H, dtype=BF16, device=dev)
    y = flat.as_strided((M, H), (ld, 1))
    g = _gen(dev, 8)
    v, r = _randn(g, (M, H)), _randn(g, (M, H))
    y.copy_(v)
    want, got = torch.empty(M, H, dtype=BF16, device=dev), torch.empty(M, H, dtype=BF16, device=dev)
    B.moe_block_norm(v, r, want, post=1, pre=2)
    B.moe_block_norm(y, r, got, post=1, pre=2)
    z = flat.as_strided((M, H), (ld, 1))
    B.moe_block_norm(v, r, got, z_out=z, post=1, pre=2)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    near = torch.empty_like(v)
    B.moe_block_norm(v, r, got, z_out=near, post=1, pre=2)
    torch.cuda.synchronize()
    assert torch.equal(z, near)


# ---------------------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------------------
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _act_ref(act, h, err):
    """act(h) and a bound where h is off by err.  Slopes are at most 1.13.  silu and gelu_tanh: a
    sigmoid of an argument w that is off by up to 5 roundings, exp2 of its rounded product (1.5 |w|
    + 2), 1 + exp, the reciprocal (2) and the product: (7 |w| + 8) u relative.  gelu: the argument
    rounds twice, which moves erfc by (h^2 + 1) times that relative, and erfc is good to 16 u."""
    if act == "none":
        return h, err
    if act == "relu":
        return h.clamp(min=0.0), err
    if act == "silu":
        v, rel = h * torch.sigmoid(h), (7 * h.abs() + 8) * U
    elif act == "gelu":
        v, rel = h * torch.special.ndtr(h), (2 * (h * h + 1) + 20) * U
    else:
        w = 2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)
        v, rel = h * torch.sigmoid(w), (7 * w.abs() + 8) * U
    return v, 1.13 * err + rel * v.abs() + 2.0 ** -120


def _check_product(B, dev, M, N, K, act="none", gated=False, bias=False, res=None, ot=BF16, pad=0, seed=0,
                   std=0.02):
    """A product passes at most 40 + K / 32 roundings (32 in its MFMA, one for each MFMA of the sum,
    8 where waves or parts meet), each taken as 2 u (the hardware may truncate)."""
    g = _gen(dev, seed + M * 3 + N * 5 + K)
    rows = 2 * N if gated else N
    x = Rows(M, K, BF16, dev, pad, _randn(g, (M, K)))
    w = _randn(g, (rows, K), std)
    b = _randn(g, (rows,), 0.2) if bias else None
    r = Rows(M, N, res, dev, pad, _randn(g, (M, N), 2.0, 0.0, res)) if res else None
    out = Rows(M, N, ot, dev, pad)
    ws = torch.full((max(1, B.moe_matmul_workspace_bytes(M, N, K, gated)),), 0xFF, dtype=torch.uint8, device=dev)
    B.moe_matmul(x.t, w, out.t, bias=b, act=ACTS.index(act), gated=gated, residual=r.t if r else None,
                 workspace=ws)
    torch.cuda.synchronize()
    xd, wd = x.t.double().contiguous(), w.double().T.contiguous()
    h = xd @ wd
    err = (40 + K / 32) * 2 * U * (xd.abs() @ wd.abs())
    if b is not None:
        h = h + b.double()
        err = err + U * (h.abs() + err)
    v, e = _act_ref(act, h[:, :N], err[:, :N])
    if gated:
        up, eu = h[:, N:], err[:, N:]
        e = e * up.abs() + v.abs() * eu + e * eu + 2 * U * (v * up).abs()
        v = v * up
    if r is not None:
        v = v + r.t.double()
        e = e + U * (v.abs() + e)
    off = (out.t.double() - v).abs()
    assert (off <= e + _round(ot) * (v.abs() + e) + 2.0 ** -126).all(), off.max().item()
    for t in (x, r, out):
        assert t is None or t.untouched()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("N,K", [(1, 8), (33, 72), (64, 64), (136, 520), (1000, 1032), (2048, 512)])
def test_product_sizes(B, dev, M, N, K):
    _check_product(B, dev, M, N, K)
    _check_product(B, dev, M, N, K, act="silu", gated=True, bias=True, res=F32, ot=F32, pad=8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(3, 40, 264), (40, 77, 256), (300, 264, 320), (700, 520, 1088)])
def test_product_epilogues(B, dev, act, gated, M, N, K):
    _check_product(B, dev, M, N, K, act=act, gated=gated, std=0.1)
    _check_product(B, dev, M, N, K, act=act, gated=gated, bias=True, res=BF16, pad=16)
    _check_product(B, dev, M, N, K, act=act, gated=gated, res=F32, ot=F32)
    _check_product(B, dev, M, N, K, act=act, gated=gated, bias=True, res=BF16, ot=F32, pad=24, std=1.0)


@pytest.mark.parametrize("M,N,K,gated", [(1024, 1024, 1024, False), (1024, 512, 1024, True),
                                         (2048, 1536, 2048, False), (2050, 777, 1000, True),
                                         (4096, 1024, 520, False), (1537, 4104, 4096, False),
                                         (3000, 1100, 1160, True), (513, 8192, 256, False),
                                         (5000, 136, 4096, False), (128, 256, 16384, False),
                                         (96, 128, 65536, False), (16, 64, 131072, True)])
def test_product_large(B, dev, M, N, K, gated):
    _check_product(B, dev, M, N, K, gated=gated, act="silu" if gated else "none", bias=True, res=BF16)
    _check_product(B, dev, M, N, K, gated=gated, act="silu" if gated else "none", ot=F32, pad=8)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(33, 40, 4096), (40, 512, 7168), (77, 65, 2056), (130, 24, 4104), (200, 300, 8256),
                                   (64, 1, 2048), (1000, 33, 6144), (77, 4099, 7168), (200, 1024, 8192)])
def test_product_in_parts_of_k(B, dev, M, N, K, gated):
    """Few tiles and a long K: the sums of its parts meet in the workspace (filled with NaN here)."""
    _check_product(B, dev, M, N, K, gated=gated)
    _check_product(B, dev, M, N, K, gated=gated, act="gelu", bias=True, res=BF16, pad=8)
    _check_product(B, dev, M, N, K, gated=gated, act="silu", bias=True, res=F32, ot=F32, pad=24)


def test_product_in_parts_of_k_on_two_streams(B, dev):
    """Two streams with a workspace each, and graphs that share one and are replayed in turn."""
    M, N, K = 200, 1024, 8200
    assert B.moe_matmul_workspace_bytes(M, N, K, False) > 0
    g = _gen(dev, 11)
    x = [_randn(g, (M, K)) for _ in range(2)]
    w = [_randn(g, (N, K), 0.05) for _ in range(2)]
    need = B.moe_matmul_workspace_bytes(M, N, K, False)
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(2)]
    want = [torch.empty(M, N, dtype=BF16, device=dev) for _ in range(2)]
    for i in range(2):
        B.moe_matmul(x[i], w[i], want[i], workspace=ws[0])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(t) for t in want]
    for _ in range(10):
        for i in range(2):
            B.moe_matmul(x[i], w[i], got[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            B.moe_matmul(x[i], w[i], got[i], workspace=ws[0])
    for _ in range(3):
        for t in got:
            t.zero_()
        ws[0].fill_(0xFF)
        for q in graphs:
            q.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,N,K", [(4, 64, 256), (100, 128, 256), (1100, 512, 512)])
def test_product_onto_the_residual(B, dev, M, N, K):
    g = _gen(dev, 3)
    x, w = _randn(g, (M, K)), _randn(g, (N, K), 0.05)
    for t in (BF16, F32):
        r = _randn(g, (M, N), 1.0, 0.0, t)
        want, got = torch.empty_like(r), r.clone()
        B.moe_matmul(x, w, want, residual=r)
        B.moe_matmul(x, w, got, residual=got)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("M,N,K,ld", [(3, 64, 72, (1 << 31) + 64), (40, 512, 2056, 1 << 27), (300, 1024, 328, 1 << 24),
                                      (1000, 4104, 1032, (1 << 23) + 8), (2048, 7168, 520, 1 << 23),
                                      (2048, 7168, 520, (1 << 23) + 8)])
@pytest.mark.parametrize("gated", [False, True])
def test_product_offsets_past_32_bits(B, dev, M, N, K, ld, gated):
    """Rows of x, residual and out whose offsets in values pass 2^32 (out over the residual).  The stride
    may choose another order of sums, so both results are within a product's bound of the exact one."""
    g = _gen(dev, 9)
    rows = 2 * N if gated else N
    x, w, r = _randn(g, (M, K)), _randn(g, (rows, K), 0.05), _randn(g, (M, N))
    want = torch.empty(M, N, dtype=BF16, device=dev)
    ws = torch.empty(max(1, B.moe_matmul_workspace_bytes(M, N, K, gated)), dtype=torch.uint8, device=dev)
    act = dict(act=B.ACT_RELU, gated=True) if gated else {}
    B.moe_matmul(x, w, want, residual=r, workspace=ws, **act)
    flat = torch.empty(M * ld, dtype=BF16, device=dev)
    far_x, far_r = flat.as_strided((M, K), (ld, 1)), flat.as_strided((M, N), (ld, 1), 4096)
    far_x.copy_(x)
    far_r.copy_(r)
    B.moe_matmul(far_x, w, far_r, residual=far_r, workspace=ws, **act)
    torch.cuda.synchronize()
    xs, wd = x.double(), w.double().T.contiguous()
    err = (40 + K / 32) * 2 * U * (xs.abs() @ wd.abs())
    if gated:
        h = xs @ wd
        a, ea, u, eu = h[:, :N].clamp(min=0.0), err[:, :N], h[:, N:], err[:, N:]
        err = ea * u.abs() + a * eu + ea * eu + 2 * U * (a * u).abs()
    err = 2 * (err + U * (want.double().abs() + r.double().abs() + err))
    top = torch.maximum(want.double().abs(), far_r.double().abs()) + err
    assert ((want.double() - far_r.double()).abs() <= err + 2 * _round(BF16) * top).all()
    assert torch.equal(far_x, x)


@pytest.mark.parametrize("M,N,K", [(5, 72, 264), (70, 200, 328), (1100, 520, 1096)])
def test_product_keeps_rows_apart(B, dev, M, N, K):
    """A token or a weight row that is not finite changes its own row or column only."""
    g = _gen(dev, 4)
    x, w = _randn(g, (M, K)), _randn(g, (N, K), 0.05)
    want = torch.empty(M, N, dtype=BF16, device=dev)
    B.moe_matmul(x, w, want)
    x[M - 1, K - 1], w[N // 2, 3] = float("nan"), float("inf")
    got = torch.empty_like(want)
    B.moe_matmul(x, w, got)
    torch.cuda.synchronize()
    assert not torch.isfinite(got[M - 1]).any() and not torch.isfinite(got[:, N // 2]).any()
    keep = torch.ones(M, N, dtype=torch.bool, device=dev)
    keep[M - 1], keep[:, N // 2] = False, False
    assert torch.equal(got[keep], want[keep])


# ---------------------------------------------------------------------------------------
# The layer for a few tokens
# ---------------------------------------------------------------------------------------
def _layer_inputs(dev, M, H, E, I, seed, router_bias=False, select_bias=False, std=0.02):
    g = _gen(dev, seed)
    return dict(x=_randn(g, (M, H)), wr=_randn(g, (E, H), 1.7 / math.sqrt(H)),
                rb=_randn(g, (E,), 0.5, 0.0, F32) if router_bias else None,
                sb=_randn(g, (E,), 0.05, 0.0, F32) if select_bias else None,
                w13=_randn(g, (E, 2 * I, H), std), w2=_randn(g, (E, H, I), std),
                res=_randn(g, (M, H)), norm=_randn(g, (H,), 0.05, 1.0))


def _rule(rule):
    r = dict(softmax=False, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0)
    r.update(rule)
    return r, dict({n: v for n, v in r.items() if n != "softmax"}, score=1 if r["softmax"] else 0)


def _run_few(B, s, k, rule, residual=True, norm=True, ws=None):
    M, H = s["x"].shape
    E, I = s["w13"].shape[0], s["w13"].shape[1] // 2
    dev = s["x"].device
    if ws is None:
        ws = torch.full((B.moe_few_workspace_bytes(M, H, E, I, k),), 0xFF, dtype=torch.uint8, device=dev)
    out, z = Rows(M, H, BF16, dev), Rows(M, H, BF16, dev)
    ids = torch.full((M, k), -7, dtype=torch.int32, device=dev)
    w = torch.full((M, k), float("nan"), device=dev)
    B.moe_forward_few(s["x"], s["wr"], s["rb"], s["w13"], s["w2"], s["res"] if residual else None,
                      s["norm"] if norm else None, 1e-5, k, out.t if norm else None, ws, residual_out=z.t,
                      topk_ids_out=ids, topk_w_out=w, select_bias=s["sb"], **_rule(rule)[1])
    return out, z, ids, w


def _check_few(B, dev, M, H, E, I, k, rule=None, router_bias=False, select_bias=False, residual=True,
               seed=0, inputs=None):
    """Bounds: a dot product of K values is a chain of K / 8 products in a lane, 3 steps between
    lanes, each step taken as 2 u: up sums off by (K / 8 + 3) 2 u sum |x| |w|.  silu(g) u: slope
    1.1, (7 |g| + 8) u of its own as in _act_ref.  Down: the same with act's errors through |w2|.
    The weighted sum: k + 2 roundings."""
    rule = rule or {}
    s = inputs or _layer_inputs(dev, M, H, E, I, seed + M + H, router_bias, select_bias)
    out, z, ids, w = _run_few(B, s, k, rule, residual)
    torch.cuda.synchronize()
    assert out.untouched() and z.untouched()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    logits = f64(s["x"]) @ f64(s["wr"]).T
    if s["rb"] is not None:
        logits = logits + f64(s["rb"])
    r = _rule(rule)[0]
    rid, rw = orc.route_logits(logits, None if s["sb"] is None else f64(s["sb"]), k, **r)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(f64(w) - rw) <= 2.0 ** -23 * np.abs(rw)).all()
    zw = s["res"].double() if residual else torch.zeros(M, H, dtype=torch.float64, device=dev)
    err = torch.zeros_like(zw)
    size = zw.abs()
    for t in range(M):
        x = s["x"][t].double()
        for j in range(k):
            e = int(rid[t, j])
            w13, w2 = s["w13"][e].double(), s["w2"][e].double()
            h, eh = w13 @ x, (H / 8 + 3) * 2 * U * (w13.abs() @ x.abs())
            v, ev = _act_ref("silu", h[:I], eh[:I])
            act = v * h[I:]
            ea = ev * h[I:].abs() + v.abs() * eh[I:] + ev * eh[I:] + 2 * U * act.abs()
            y = w2 @ act
            ey = w2.abs() @ ea + (I / 8 + 3) * 2 * U * (w2.abs() @ act.abs())
            zw[t] += float(rw[t, j]) * y
            err[t] += float(rw[t, j]) * (ey + 2 * U * y.abs())
            size[t] += float(rw[t, j]) * y.abs()
    err = err + (k + 2) * U * size
    off = (z.t.double() - zw).abs()
    assert (off <= err + 2.0 ** -8 * (zw.abs() + err)).all(), off.max().item()
    o, eo = _norm_ref(zw, err, 1, s["norm"], None, 0.0, 1e-5)
    off = (out.t.double() - o).abs()
    assert (off <= eo + 2.0 ** -8 * (o.abs() + eo)).all(), off.max().item()
    return s, out.t, z.t, ids, w


@pytest.mark.parametrize("M,H,E,I,k", [(4, 256, 8, 512, 2), (1, 8, 1, 16, 1), (1, 64, 4, 64, 4), (2, 72, 5, 48, 3),
                                       (3, 200, 60, 80, 4), (5, 1032, 33, 272, 7), (8, 520, 16, 656, 16),
                                       (9, 256, 3, 112, 2), (13, 136, 2, 1040, 2), (16, 2048, 64, 128, 8),
                                       (16, 264, 8, 96, 8), (16, 64, 256, 32, 32), (1, 7168, 8, 256, 2),
                                       (7, 16384, 4, 32, 3), (6, 32, 4, 32768, 2), (1, 128, 1024, 16, 16),
                                       (1, 64, 600, 16, 512), (12, 8200, 3, 144, 2), (4, 1024, 128, 768, 6)])
def test_few_sizes(B, dev, M, H, E, I, k):
    _check_few(B, dev, M, H, E, I, k)


@pytest.mark.parametrize("M,H,E,I,k", [(16, 4104, 8, 2064, 8), (16, 520, 8, 2064, 8), (16, 4104, 8, 528, 8),
                                       (13, 4168, 8, 2080, 5), (16, 8200, 4, 4112, 3)])
def test_few_with_several_rows_per_expert(B, dev, M, H, E, I, k):
    """Enough picks per expert for items of two row groups, in both products, in one, in the other."""
    _check_few(B, dev, M, H, E, I, k)


@pytest.mark.parametrize("rule", [
    dict(softmax=True), dict(softmax=True, renormalize=False, scale=2.5), dict(renormalize=False),
    dict(n_group=4, topk_group=2, group_top=2), dict(n_group=8, topk_group=3, group_top=1, scale=0.5),
    dict(softmax=True, n_group=2, topk_group=1, group_top=2), dict(n_group=40, topk_group=12, group_top=1)])
@pytest.mark.parametrize("router_bias,select_bias", [(False, False), (True, False), (False, True), (True, True)])
def test_few_rules(B, dev, rule, router_bias, select_bias):
    _check_few(B, dev, 5, 256, 80, 64, 6, rule, router_bias, select_bias)


def test_few_without_residual_or_norm(B, dev):
    s, out, z, ids, w = _check_few(B, dev, 4, 512, 8, 256, 2, residual=False)
    _, z2, _, _ = _run_few(B, s, 2, {}, residual=False, norm=False)
    torch.cuda.synchronize()
    assert torch.equal(z2.t, z)


def test_few_agrees_with_the_layer(B, dev):
    """moe_forward's picks and weights, its results within its own roundings of act and the picks'
    rows to bf16 (2^-8 each, of values no larger than the sums of magnitudes allow)."""
    M, H, E, I, k, block = 8, 1024, 32, 512, 4, 16
    s = _layer_inputs(dev, M, H, E, I, 11, router_bias=True)
    out, z, ids, w = _run_few(B, s, k, {})
    ws = torch.empty(B.moe_workspace_bytes(M, H, E, I, k, block), dtype=torch.uint8, device=dev)
    o2, z2 = torch.empty_like(out.t), torch.empty_like(out.t)
    i2, w2 = torch.empty_like(ids), torch.empty_like(w)
    B.moe_forward(s["x"], s["wr"], s["rb"], s["w13"], s["w2"], s["res"], s["norm"], 1e-5, k, block, o2, ws,
                  residual_out=z2, topk_ids_out=i2, topk_w_out=w2)
    torch.cuda.synchronize()
    assert torch.equal(ids, i2)
    assert (w - w2).abs().max().item() <= 2.0 ** -23
    assert (z.t.float() - z2.float()).abs().max().item() <= 2.0 ** -8 * 2 * 6.0


def test_few_masked_experts(B, dev):
    """A bias of -inf takes experts out; picks beyond the others come in id order with weight 0."""
    M, H, E, I, k = 3, 128, 8, 64, 4
    s = _layer_inputs(dev, M, H, E, I, 12)
    s["rb"] = torch.full((E,), -math.inf, device=dev)
    s["rb"][[2, 5]] = 0.0
    out, z, ids, w = _run_few(B, s, k, {})
    torch.cuda.synchronize()
    assert all(sorted(r[:2]) == [2, 5] and r[2:] == [0, 1] for r in ids.tolist())
    assert (w[:, 2:] == 0).all() and torch.isfinite(out.t).all()
    s["rb"][:] = -math.inf
    out, z, ids, w = _run_few(B, s, k, {})
    torch.cuda.synchronize()
    assert (w == 0).all() and torch.equal(z.t, s["res"]) and ids.tolist() == [[0, 1, 2, 3]] * M


def test_few_equal_experts_in_id_order(B, dev):
    M, H, E, I, k = 16, 264, 130, 32, 5
    s = _layer_inputs(dev, M, H, E, I, 13)
    s["wr"][:] = s["wr"][0]
    for rule in ({}, dict(softmax=True), dict(n_group=10, topk_group=2, group_top=2)):
        _, _, ids, w = _run_few(B, s, k, rule)
        torch.cuda.synchronize()
        assert ids.tolist() == [list(range(k))] * M
        assert torch.equal(w, torch.full_like(w, 0.2))


def test_few_is_repeatable(B, dev):
    """The same bits every time, in a workspace that other sizes have used, back to back."""
    sizes = [(8, 1024, 32, 512, 4), (1, 512, 16, 256, 2), (16, 256, 8, 96, 8)]
    room = torch.full((max(B.moe_few_workspace_bytes(*c) for c in sizes),), 0xFF, dtype=torch.uint8, device=dev)
    first = None
    for _ in range(20):
        got = []
        for M, H, E, I, k in sizes:
            s = _layer_inputs(dev, M, H, E, I, M)
            out, z, ids, w = _run_few(B, s, k, {}, ws=room)
            got += [out.t, z.t, ids, w]
        torch.cuda.synchronize()
        first = first or [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_few_two_streams(B, dev):
    """Calls at once on two streams, each with its own workspace."""
    s = [_layer_inputs(dev, 8, 2048, 64, 768, 20 + i) for i in range(2)]
    want = [_run_few(B, t, 8, {})[0].t.clone() for t in s]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in s]
    ws = [torch.empty(B.moe_few_workspace_bytes(8, 2048, 64, 768, 8), dtype=torch.uint8, device=dev) for _ in s]
    outs = []
    for _ in range(10):
        for t, q, room in zip(s, streams, ws):
            with torch.cuda.stream(q):
                outs.append(_run_few(B, t, 8, {}, ws=room)[0].t)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])


# ---------------------------------------------------------------------------------------
# Together, and in graphs
# ---------------------------------------------------------------------------------------
def _block(B, s, k, room, bufs):
    """A block with a shared expert: norm, shared expert's two products, routed experts onto its
    result, then norm, gate and residual and the next norm."""
    B.moe_block_norm(None, s["stream"], bufs["h"], pre=B.NORM_RMS, pre_w=s["w_in"])
    B.moe_matmul(bufs["h"], s["s13"], bufs["a"], act=B.ACT_SILU, gated=True)
    B.moe_matmul(bufs["a"], s["s2"], bufs["shared"])
    B.moe_forward_few(bufs["h"], s["wr"], None, s["w13"], s["w2"], bufs["shared"], None, 1e-5, k, None, room,
                      residual_out=bufs["y"])
    B.moe_block_norm(bufs["y"], s["stream"], bufs["out"], z_out=bufs["z"], post=B.NORM_RMS, post_w=s["w_post"],
                     gate=s["gate"], block_scale=0.5, pre=B.NORM_RMS, pre_w=s["w_next"])


def _block_inputs(dev, M, H, E, I, S, seed):
    g = _gen(dev, seed)
    s = _layer_inputs(dev, M, H, E, I, seed + 1)
    s.update(stream=_randn(g, (M, H), 2.0, 0.0, F32), w_in=_randn(g, (H,), 0.05, 1.0),
             w_post=_randn(g, (H,), 0.05, 1.0), w_next=_randn(g, (H,), 0.05, 1.0), gate=_randn(g, (M, 1), 0.2, 0.8),
             s13=_randn(g, (2 * S, H), 0.02), s2=_randn(g, (H, S), 0.02))
    bufs = {n: torch.empty(M, H, dtype=BF16, device=dev) for n in ("h", "shared", "y", "out")}
    bufs["a"] = torch.empty(M, S, dtype=BF16, device=dev)
    bufs["z"] = torch.empty(M, H, dtype=F32, device=dev)
    return s, bufs


def test_a_block(B, dev):
    """Each step from the buffers that the step before left, in 64 bits: what is left then is one
    rounding to bf16 of a step's result, and 2^-12 of the row's size for fp32 sums and orders."""
    M, H, E, I, S, k = 6, 1024, 32, 384, 512, 4
    s, b = _block_inputs(dev, M, H, E, I, S, 30)
    room = torch.full((B.moe_few_workspace_bytes(M, H, E, I, k),), 0xFF, dtype=torch.uint8, device=dev)
    _block(B, s, k, room, b)
    torch.cuda.synchronize()

    def close(got, want):
        tol = _round(got.dtype) * want.abs() + 2.0 ** -12 * want.abs().amax(1, keepdim=True)
        assert ((got.double() - want).abs() <= tol).all()

    rms = lambda v, w: v / ((v * v).mean(1, keepdim=True) + 1e-5).sqrt() * w.double()  # noqa: E731
    h = b["h"].double()
    close(b["h"], rms(s["stream"].double(), s["w_in"]))
    u = h @ s["s13"].double().T.contiguous()
    close(b["a"], u[:, :S] * torch.sigmoid(u[:, :S]) * u[:, S:])
    close(b["shared"], b["a"].double() @ s["s2"].double().T.contiguous())
    ids, w = orc.route_logits((h @ s["wr"].double().T.contiguous()).cpu().numpy(), None, k)
    y = b["shared"].double()
    for t in range(M):
        for j in range(k):
            e = int(ids[t, j])
            u = s["w13"][e].double() @ h[t]
            y[t] += float(w[t, j]) * (s["w2"][e].double() @ (u[:I] * torch.sigmoid(u[:I]) * u[I:]))
    close(b["y"], y)
    z = s["stream"].double() + 0.5 * s["gate"].double() * rms(b["y"].double(), s["w_post"])
    close(b["z"], z)
    close(b["out"], rms(z, s["w_next"]))


def test_blocks_in_graphs(B, dev):
    """Two captured blocks that share a workspace, replayed in turn with new inputs and eager work
    between the replays."""
    M, H, E, I, S, k = 5, 768, 16, 256, 384, 3
    room = torch.full((B.moe_few_workspace_bytes(M, H, E, I, k),), 0xFF, dtype=torch.uint8, device=dev)
    sets = [_block_inputs(dev, M, H, E, I, S, 40 + 5 * i) for i in range(2)]
    for s, b in sets:
        _block(B, s, k, room, b)
    torch.cuda.synchronize()
    graphs = []
    for s, b in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _block(B, s, k, room, b)
        graphs.append(g)
    for step in range(6):
        i = step % 2
        s, b = sets[i]
        s["stream"].copy_(_randn(_gen(dev, 90 + step), (M, H), 2.0, 0.0, F32))
        graphs[i].replay()
        torch.cuda.synchronize()
        got = [b[n].clone() for n in ("out", "z", "y")]
        _block(B, s, k, room, b)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b[n]) for a, n in zip(got, ("out", "z", "y")))


def test_other_streams_wait_for_nothing_else(B, dev):
    """Every call runs on the stream that it is given."""
    q = torch.cuda.Stream()
    g = _gen(dev, 50)
    x, w = _randn(g, (40, 512)), _randn(g, (256, 512), 0.05)
    want = torch.empty(40, 256, dtype=BF16, device=dev)
    B.moe_matmul(x, w, want)
    got, n1, n2 = torch.empty_like(want), torch.empty_like(x), torch.empty_like(x)
    B.moe_block_norm(x, x, n1, post=1)
    torch.cuda.synchronize()
    B.moe_matmul(x, w, got, stream=q)
    B.moe_block_norm(x, x, n2, post=1, stream=q)
    q.synchronize()
    assert torch.equal(got, want) and torch.equal(n1, n2)


def test_binding_refuses(B, dev):
    bf = lambda *s: torch.zeros(*s, dtype=BF16, device=dev)  # noqa: E731
    x = bf(4, 64)
    with pytest.raises(ValueError):
        B.moe_block_norm(x, bf(4, 72), bf(4, 64))
    with pytest.raises(ValueError):
        B.moe_block_norm(x, x, bf(4, 64), gate=bf(3, 64))
    with pytest.raises(TypeError):
        B.moe_block_norm(x, x, bf(4, 64), gate=bf(4, 64).float())
    with pytest.raises(TypeError):
        B.moe_block_norm(x, x, bf(4, 64).float())
    with pytest.raises(TypeError):
        B.moe_block_norm(x, x, bf(4, 64), z_out=bf(4, 64).float())
    with pytest.raises(ValueError):
        B.moe_block_norm(x.T, bf(64, 4), bf(64, 4))
    with pytest.raises(ValueError):
        B.moe_block_norm(bf(1, 64).expand(4, 64), x, bf(4, 64))
    with pytest.raises(B.MoeError):
        B.moe_block_norm(bf(4, 70)[:, :64], x, bf(4, 64))
    with pytest.raises(ValueError):
        B.moe_matmul(x, bf(32, 72), bf(4, 32))
    with pytest.raises(ValueError):
        B.moe_matmul(x, bf(33, 64), bf(4, 16), gated=True)
    with pytest.raises(ValueError):
        B.moe_matmul(x, bf(32, 64), bf(4, 32), bias=bf(16))
    with pytest.raises(TypeError):
        B.moe_matmul(x, bf(32, 64), bf(4, 32).half())
    with pytest.raises(B.MoeError):
        B.moe_matmul(bf(4, 68)[:, :64], bf(32, 64), bf(4, 32))
    with pytest.raises(B.MoeError):
        B.moe_matmul(x, bf(32, 64), bf(4, 32), act=9)
    few = lambda M: B.moe_forward_few(bf(M, 64), bf(8, 64), None, bf(8, 64, 64), bf(8, 64, 32), bf(M, 64),  # noqa: E731
                                      bf(64), 1e-5, 2, bf(M, 64), torch.zeros(1 << 20, dtype=torch.uint8, device=dev))
    few(16)
    with pytest.raises(B.MoeError):
        few(17)
    torch.cuda.synchronize()
