"""Each variant of the bf16 product on the GPU against 64 bits, at sizes that are known to take it, and
the block norm where its workgroups or waves walk several rows.

Bounds count roundings: u = 2^-24 for one in fp32, 2^-8 for the last one to bf16 (2^-24 to fp32).
"""
import math

import pytest
import torch

from test_gpu_block import ACTS, BF16, F32, U, Rows, _act_ref, _gen, _randn, _round

pytestmark = pytest.mark.gpu


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
# Product
# ---------------------------------------------------------------------------------------
def _check(B, dev, tile, M, N, K, act="none", gated=False, bias=False, res=None, ot=BF16, pad=0, parts=False,
           std=0.02, in_place=False):
    """tile: the token-tile height that these sizes take; parts: whether K is cut into parts.

    A product passes at most 32 roundings in its MFMA (16 in one of 16 values), one for each MFMA of the
    sum (K / 16 of them in tiles of 256, else K / 32) and 16 where waves or parts meet: 48 + K / 16, each
    taken as 2 u (the hardware may truncate)."""
    assert B.moe_matmul_tile_rows(M, N, K, gated, K + pad) == tile
    need = B.moe_matmul_workspace_bytes(M, N, K, gated)
    assert (need > 0) == parts
    g = _gen(dev, M * 3 + N * 5 + K)
    rows = 2 * N if gated else N
    x = Rows(M, K, BF16, dev, pad, _randn(g, (M, K)))
    w = _randn(g, (rows, K), std)
    b = _randn(g, (rows,), 0.2) if bias else None
    r = Rows(M, N, res, dev, pad, _randn(g, (M, N), 2.0, 0.0, res)) if res else None
    rd = r.t.double() if res else None
    out = r if in_place else Rows(M, N, ot, dev, pad)
    ws = torch.full((max(1, need),), 0xFF, dtype=torch.uint8, device=dev)
    B.moe_matmul(x.t, w, out.t, bias=b, act=ACTS.index(act), gated=gated, residual=r.t if r else None,
                 workspace=ws)
    torch.cuda.synchronize()
    xd, wd = x.t.double().contiguous(), w.double().T.contiguous()
    h = xd @ wd
    err = (48 + K / 16) * 2 * U * (xd.abs() @ wd.abs())
    if b is not None:
        h += b.double()
        err += U * (h.abs() + err)
    v, e = _act_ref(act, h[:, :N], err[:, :N])
    if gated:
        up, eu = h[:, N:], err[:, N:]
        e = e * up.abs() + v.abs() * eu + e * eu + 2 * U * (v * up).abs()
        v = v * up
    if r is not None:
        v = v + rd
        e = e + U * (v.abs() + e)
    off = (out.t.double() - v).abs()
    assert (off <= e + _round(ot) * (v.abs() + e) + 2.0 ** -126).all(), off.max().item()
    for t in (x, r, out):
        assert t is None or t.untouched()


# sizes of whole and partial last chunks of K (64 values), two chunks among them; remainders of M and N,
# N % 8 != 0; one tile per workgroup and several
BIG = [(2048, 7168, 2048, False), (2300, 6001, 1032, False), (8192, 8192, 72, False), (8200, 9001, 128, False),
       (5000, 8200, 200, False), (300, 30000, 1000, False), (2050, 4097, 4104, True), (5000, 7000, 72, True),
       (8192, 4100, 128, True), (4096, 4100, 512, True), (1500, 5000, 520, True), (33000, 1000, 200, True),
       (1537, 4104, 4096, True)]


@pytest.mark.parametrize("M,N,K,gated", BIG)
def test_tiles_of_256(B, dev, M, N, K, gated):
    _check(B, dev, 256, M, N, K, gated=gated, act="silu" if gated else "none")
    _check(B, dev, 256, M, N, K, gated=gated, act="gelu", bias=True, res=F32, ot=F32, pad=8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K,gated", [(2300, 6001, 1032, False), (2304, 6000, 1024, False),
                                         (2000, 3501, 1088, True), (2000, 3504, 1096, True)])
def test_epilogues_of_tiles_of_256(B, dev, act, M, N, K, gated):
    _check(B, dev, 256, M, N, K, act, gated, bias=True, std=0.1)
    _check(B, dev, 256, M, N, K, act, gated, res=BF16, pad=24)
    _check(B, dev, 256, M, N, K, act, gated, res=F32, std=1.0)
    _check(B, dev, 256, M, N, K, act, gated, bias=True, res=BF16, ot=F32, pad=16)
    _check(B, dev, 256, M, N, K, act, gated, ot=F32, std=0.1)


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("M,N,K,gated", [(2048, 7168, 2048, False), (8192, 8195, 72, False), (2304, 6000, 1024, False),
                                         (4096, 4100, 512, True), (2000, 3501, 1096, True)])
def test_tiles_of_256_onto_the_residual(B, dev, t, M, N, K, gated):
    _check(B, dev, 256, M, N, K, "relu", gated, bias=True, res=t, ot=t, pad=8, in_place=True)


@pytest.mark.parametrize("M,N,K,gated", [(2300, 6001, 1032, False), (2304, 6000, 1024, False),
                                         (8192, 8192, 72, False), (2000, 3501, 1088, True),
                                         (5000, 7000, 72, True)])
def test_tiles_of_256_keep_rows_apart(B, dev, M, N, K, gated):
    """A token or a weight row that is not finite changes its own row or column only."""
    g = _gen(dev, 4)
    x, w = _randn(g, (M, K)), _randn(g, (2 * N if gated else N, K), 0.05)
    assert B.moe_matmul_tile_rows(M, N, K, gated) == 256
    want = torch.empty(M, N, dtype=BF16, device=dev)
    B.moe_matmul(x, w, want, gated=gated)
    x[M - 1, K - 1], w[N // 2, 3] = float("nan"), float("inf")
    got = torch.empty_like(want)
    B.moe_matmul(x, w, got, gated=gated)
    torch.cuda.synchronize()
    assert not torch.isfinite(got[M - 1]).any() and not torch.isfinite(got[:, N // 2]).any()
    keep = torch.ones(M, N, dtype=torch.bool, device=dev)
    keep[M - 1], keep[:, N // 2] = False, False
    assert torch.equal(got[keep], want[keep])


def test_tiles_of_256_are_repeatable(B, dev):
    """The same bits from calls back to back, on two streams, and from a graph."""
    M, N, K = 4096, 4100, 520
    assert B.moe_matmul_tile_rows(M, N, K, True) == 256
    g = _gen(dev, 6)
    x, w, r = _randn(g, (M, K)), _randn(g, (2 * N, K), 0.05), _randn(g, (M, N))
    want = torch.empty(M, N, dtype=BF16, device=dev)
    call = lambda out, **kw: B.moe_matmul(x, w, out, act=B.ACT_SILU, gated=True, residual=r, **kw)  # noqa: E731
    call(want)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(want) for _ in range(2)]
    for _ in range(5):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        for q, t in zip(streams, got):
            call(t, stream=q)
        torch.cuda.synchronize()
        assert all(torch.equal(t, want) for t in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(got[0])
        call(got[1])
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, want) for t in got)


@pytest.mark.parametrize("tile,M,N,K,gated", [
    (128, 1537, 4104, 4096, False), (128, 640, 4099, 7176, False), (128, 1900, 3600, 2056, False),
    (128, 1030, 7168, 2048, False), (128, 1100, 1030, 1024, True), (128, 513, 2056, 1000, True),
    (128, 1000, 1500, 2056, True), (64, 1100, 1030, 1024, False), (64, 513, 2056, 1000, False),
    (64, 1000, 1500, 2056, False), (64, 8192, 4100, 72, False), (64, 8200, 4100, 120, False),
    (64, 700, 3001, 1088, True), (64, 1300, 1100, 264, True)])
def test_tiles_of_64_and_128(B, dev, tile, M, N, K, gated):
    _check(B, dev, tile, M, N, K, gated=gated, act="silu" if gated else "none")
    _check(B, dev, tile, M, N, K, "gelu", gated, bias=True, res=F32, ot=F32, pad=8)
    _check(B, dev, tile, M, N, K, "gelu_tanh", gated, res=BF16, pad=24, in_place=True)


# Parts: 2, 4, 8 and 16 of them; K % 64 != 0, where a part ends with a partial chunk, and whole chunks
PARTS = [(200, 1024, 8200, False), (77, 4099, 7176, False), (40, 512, 7112, False), (200, 300, 8264, False),
         (100, 256, 16392, False), (130, 520, 9000, False), (33, 257, 16440, False), (300, 140, 12040, False),
         (77, 4099, 7168, False), (65, 64, 65544, False), (200, 1024, 8200, True), (77, 4099, 7176, True),
         (200, 300, 8264, True), (33, 1030, 4104, True), (100, 256, 16392, True), (33, 257, 16440, True),
         (500, 130, 8008, True), (300, 140, 12040, True), (36, 2000, 7168, True), (65, 64, 65544, True)]


@pytest.mark.parametrize("M,N,K,gated", PARTS)
def test_parts_of_k(B, dev, M, N, K, gated):
    """The sums of K's parts meet in the workspace (filled with NaN here)."""
    _check(B, dev, 64, M, N, K, gated=gated, parts=True)
    _check(B, dev, 64, M, N, K, "gelu", gated, bias=True, res=BF16, pad=8, parts=True)
    _check(B, dev, 64, M, N, K, "silu", gated, bias=True, res=F32, ot=F32, pad=24, parts=True, in_place=True)


def test_parts_of_k_keep_rows_apart(B, dev):
    """A token or a weight row that is not finite, in the last, partial chunk, changes its own row or column
    only."""
    for M, N, K, gated in PARTS[:4] + PARTS[10:13]:
        need = B.moe_matmul_workspace_bytes(M, N, K, gated)
        assert need > 0
        g = _gen(dev, 4)
        x, w = _randn(g, (M, K)), _randn(g, (2 * N if gated else N, K), 0.05)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
        want, got = (torch.empty(M, N, dtype=BF16, device=dev) for _ in range(2))
        B.moe_matmul(x, w, want, gated=gated, workspace=ws)
        x[M - 1, K - 1], w[N // 2, K - 3] = float("nan"), float("inf")
        B.moe_matmul(x, w, got, gated=gated, workspace=ws)
        torch.cuda.synchronize()
        assert not torch.isfinite(got[M - 1]).any() and not torch.isfinite(got[:, N // 2]).any()
        keep = torch.ones(M, N, dtype=torch.bool, device=dev)
        keep[M - 1], keep[:, N // 2] = False, False
        assert torch.equal(got[keep], want[keep])


# ---------------------------------------------------------------------------------------
# Block norm: more rows than run at once, in each variant
# ---------------------------------------------------------------------------------------
NONE, RMS, LAYER = 0, 1, 2


def _norm(v, err, kind, w, b, offset, eps):
    """N(v) in 64 bits, and a bound of the kernel's error where its v is off by up to err.

    A sum over a row is a chain of at most 32 values a thread, 6 steps in the wave and 16 waves, 54
    roundings, and a term of it rounds twice.  The mean is off by dm = 57 u mean |v| and the mean of err.
    A difference d from it then is off by err + dm + u |d|, the mean of squares m2 by 58 u of itself and
    2 rms(d) (rms(err) + dm) and the square of those errors, its root by half of that relative to m2 + eps,
    and root and quotient round (4 u).  d f (offset + w) + b: 5 roundings more."""
    if kind == NONE:
        return v, err
    dm = torch.zeros_like(v[:, :1])
    d = v
    if kind == LAYER:
        dm = 57 * U * v.abs().mean(dim=1, keepdim=True) + err.mean(dim=1, keepdim=True)
        d = v - v.mean(dim=1, keepdim=True)
    m2 = (d * d).mean(dim=1, keepdim=True)
    f = 1.0 / torch.sqrt(m2 + eps)
    r = (err * err).mean(dim=1, keepdim=True).sqrt() + dm
    rel = (29 + 4) * U + r * f + 0.5 * (r * f) ** 2
    g = torch.ones_like(v[:1]) if w is None else (offset + w.double())[None, :]
    out = d * f * g
    off = ((err + dm) * f * (1 + rel) + (d * f).abs() * (rel + 6 * U)) * g.abs()
    if b is not None:
        out = out + b.double()
        off = off + U * (out.abs() + off)
    return out, off


def _norm_inputs(dev, M, H, post, pre, gate, yt, rt, weights, bias, offset, pad, y_mean=0.0):
    g = _gen(dev, M * 7 + H)
    s = dict(y=Rows(M, H, yt, dev, pad, _randn(g, (M, H), 1.0, y_mean, yt)),
             r=Rows(M, H, rt, dev, 2 * pad, _randn(g, (M, H), 3.0, 0.0, rt)))
    for n, kind in (("post", post), ("pre", pre)):
        s[n + "_w"] = _randn(g, (H,), 0.05, 1.0 - offset) if weights and kind else None
        s[n + "_b"] = _randn(g, (H,), 0.1) if bias and kind else None
    shape = {"none": None, "channel": (H,), "full": (M, H), "token": (M, 1), "one": (1, 1)}[gate]
    s["gate"] = None if shape is None else _randn(g, shape, 0.3, 0.7)
    return s


def _call(B, s, y, r, out, z, post, pre, offset, a, b):
    B.moe_block_norm(y, r, out, z_out=z, gate=s["gate"], post=post, post_w=s["post_w"], post_b=s["post_b"],
                     pre=pre, pre_w=s["pre_w"], pre_b=s["pre_b"], eps=1e-5, weight_offset=offset,
                     residual_scale=a, block_scale=b)


def _check_norm(B, dev, M, H, post=RMS, pre=RMS, gate="none", yt=BF16, rt=BF16, weights=True, bias=False,
                offset=0.0, a=1.0, b=1.0, pad=0, y_mean=0.0):
    s = _norm_inputs(dev, M, H, post, pre, gate, yt, rt, weights, bias, offset, pad, y_mean)
    z, out = Rows(M, H, rt, dev, pad), Rows(M, H, BF16, dev, 3 * pad)
    _call(B, s, s["y"].t, s["r"].t, out.t, z.t, post, pre, offset, a, b)
    torch.cuda.synchronize()
    yd = s["y"].t.double()
    want, err = _norm(yd, torch.zeros_like(yd), post, s["post_w"], s["post_b"], offset, 1e-5)
    scale = torch.tensor(b, dtype=torch.float64, device=dev)
    if s["gate"] is not None:
        gd = s["gate"].double()
        scale = scale * (gd if gd.dim() == 2 else gd[None, :])
    want, err = scale * want, scale.abs() * (err + 4 * U * want.abs())      # products in any order, sums of two
    rd = a * s["r"].t.double()
    err = err + U * rd.abs() + 2 * U * ((want + rd).abs() + want.abs() + err)
    want = want + rd
    for rows in (s["y"], s["r"], z, out):
        assert rows.untouched()
    off = (z.t.double() - want).abs()
    assert (off <= err + _round(rt) * (want.abs() + err)).all(), off.max().item()
    w2, e2 = _norm(want, err, pre, s["pre_w"], s["pre_b"], offset, 1e-5)
    off = (out.t.double() - w2).abs()
    assert (off <= e2 + _round(BF16) * (w2.abs() + e2)).all(), off.max().item()


# rows of each variant, more than twice as many as 256 CUs hold at once: a wave per row with one chunk
# a lane (8192 rows at once) or two (4096), a workgroup per row with two (4096 at H = 1032, 2560 at
# 2056, 1024 at 7168 and 8192) or four (512)
WALKS = [(17000, 264), (17000, 512), (9001, 520), (9001, 1000), (9001, 1024), (9001, 1032), (6001, 2056),
         (2300, 7168), (2300, 8192), (1300, 8200), (1300, 12296), (1300, 16384)]


@pytest.mark.parametrize("M,H", WALKS)
def test_norm_walks_rows(B, dev, M, H):
    _check_norm(B, dev, M, H, gate="channel", offset=1.0, b=0.25)
    _check_norm(B, dev, M, H, LAYER, LAYER, "full", F32, F32, bias=True, a=0.5, b=1.5, pad=8)
    _check_norm(B, dev, M, H, LAYER, RMS, "token", F32, BF16, bias=True, pad=16)
    _check_norm(B, dev, M, H, RMS, LAYER, "channel", BF16, F32, bias=True, offset=1.0)
    _check_norm(B, dev, M, H, NONE, LAYER, "full", BF16, BF16, weights=False, a=-1.0, pad=8)
    _check_norm(B, dev, M, H, LAYER, NONE, "one", F32, F32, b=0.5)
    _check_norm(B, dev, M, H, LAYER, LAYER, "none", F32, F32, y_mean=64.0)


@pytest.mark.parametrize("M,H", [(9001, 1000), (9001, 264), (2300, 7168), (9001, 1032), (1300, 16384), (600, 2056)])
@pytest.mark.parametrize("yt,rt,gate", [(BF16, BF16, "channel"), (BF16, F32, "full"), (BF16, F32, "none")])
def test_norm_walks_rows_in_place(B, dev, M, H, yt, rt, gate):
    """out over y and z over the residual: the next row is read before this one is written."""
    s = _norm_inputs(dev, M, H, LAYER, RMS, gate, yt, rt, True, True, 0.0, 8)
    z, out = Rows(M, H, rt, dev, 8), Rows(M, H, BF16, dev, 8)
    args = (LAYER, RMS, 0.0, 0.5, 2.0)
    _call(B, s, s["y"].t, s["r"].t, out.t, z.t, *args)
    _call(B, s, s["y"].t, s["r"].t, s["y"].t, s["r"].t, *args)
    torch.cuda.synchronize()
    assert torch.equal(s["y"].t, out.t) and torch.equal(s["r"].t, z.t)
    assert s["y"].untouched() and s["r"].untouched()


@pytest.mark.parametrize("M,H", WALKS)
def test_norm_walks_past_rows_that_are_not_finite(B, dev, M, H):
    """A row with a NaN or an infinity leaves the others as they were, those that its workgroup takes after
    it among them; a row of zeros is one."""
    s = _norm_inputs(dev, M, H, LAYER, RMS, "token", BF16, F32, True, True, 0.0, 0)
    z, out, z2, out2 = Rows(M, H, F32, dev), Rows(M, H, BF16, dev), Rows(M, H, F32, dev), Rows(M, H, BF16, dev)
    args = (LAYER, RMS, 0.0, 1.0, 1.0)
    _call(B, s, s["y"].t, s["r"].t, out.t, z.t, *args)
    rows = torch.arange(0, M, 7, device=dev)
    s["y"].t[rows[0::3], H // 2] = math.nan
    s["r"].t[rows[1::3], H - 1] = math.inf
    s["y"].t[rows[2::3]] = 0.0
    _call(B, s, s["y"].t, s["r"].t, out2.t, z2.t, *args)
    torch.cuda.synchronize()
    keep = torch.ones(M, dtype=torch.bool, device=dev)
    keep[rows] = False
    assert torch.equal(out.t[keep], out2.t[keep]) and torch.equal(z.t[keep], z2.t[keep])
    assert not torch.isfinite(out2.t[rows[0::3]]).any() and torch.isfinite(out2.t[rows[2::3]]).all()
    assert not torch.isfinite(out2.t[rows[1::3], H - 1]).any()
