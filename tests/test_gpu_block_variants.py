"""Each variant of the bf16 product on the GPU against 64 bits, at sizes that are known to take it.

Bounds count roundings: u = 2^-24 for one in fp32, 2^-8 for the last one to bf16 (2^-24 to fp32).
"""
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
