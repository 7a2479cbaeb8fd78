"""int8 rows, their product and the layer on int8 expert weights on the GPU against the
64-bit oracle.

Codes bit for bit; scales within fp32's 2^-24.  Products: the integer sums are exact, their
conversion to fp32, the product of the scales and the product of both round once each (3
times 2^-24), and the result once to its type (bf16 2^-8, fp32 nothing more).
Layer: the bf16 bar of the other weight formats (the rows y round as there), plus what a
scale other than 1 adds to z: every pick's row but the first rounds to bf16 (2^-8), and act
is held to 2^-14 of its neighbours' largest between the products, which moves a code next to
a border by one, a 127th of the row's largest act, in one weight of at most 127 w2_scale: the
row's largest act (taken as 8, twice what these inputs reach) times w2_scale.
"""
import numpy as np
import pytest
import torch

import _bars as bars
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


def _quantize(B, v):
    codes = torch.full(tuple(v.shape), 99, dtype=torch.int8, device=v.device)
    scales = torch.full(tuple(v.shape[:-1]), float("nan"), dtype=torch.float32, device=v.device)
    B.moe_i8_quantize(v, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (5, 512), (8, 2048), (9, 2064), (8, 7168),
                                    (4, 8192), (2, 8208), (1000, 512), (3, 131072)])
def test_quantize(B, dev, rows, K):
    g = torch.Generator(device=dev).manual_seed(rows + K)
    v = torch.randn(rows, K, generator=g, device=dev).bfloat16()
    if rows > 2:
        v[1] = 0.0
        v[2] = (torch.arange(K, device=dev) % 255 - 127).bfloat16()     # whole codes
        v[0] = (torch.arange(K, device=dev) % 64).bfloat16() / 2        # ties: a = 31.5
        v[0, 0] = 127.0
    codes, scales = _quantize(B, v)
    want, ws = orc.quantize(bf16_to_f64(bits(v)))
    assert np.array_equal(codes.cpu().numpy(), want)
    assert (np.abs(scales.cpu().numpy() - ws) <= 2 ** -24 * ws).all()


@pytest.mark.parametrize("power", [-131, -120, -60, 60, 119, 121, 126])
def test_quantize_small_and_large_values(B, dev, power):
    v = torch.randn(6, 256, generator=torch.Generator().manual_seed(1)).mul(2.0 ** power).bfloat16().to(dev)
    codes, scales = _quantize(B, v)
    want, ws = orc.quantize(bf16_to_f64(bits(v)))
    assert np.array_equal(codes.cpu().numpy(), want)
    assert (np.abs(scales.cpu().numpy() - ws) <= 2 ** -24 * ws + 2.0 ** -149).all()


def test_rows_that_are_not_finite(B, dev):
    v = torch.randn(4, 64, generator=torch.Generator().manual_seed(2)).bfloat16().to(dev)
    v[1, 5] = float("nan")
    v[2, 9] = -float("inf")
    codes, scales = _quantize(B, v)
    assert torch.isfinite(scales).tolist() == [True, False, False, True]
    w, ws = _quantize(B, torch.randn(32, 64, generator=torch.Generator().manual_seed(3)).bfloat16().to(dev))
    out = torch.zeros(4, 32, dtype=torch.bfloat16, device=dev)
    B.moe_i8_matmul(codes, scales, w, ws, out)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all(1).tolist() == [True, False, False, True]


def _workspace(B, M, N, K, dev):
    return torch.full((max(1, B.moe_i8_matmul_workspace_bytes(M, N, K)),), 0xFF, dtype=torch.uint8, device=dev)


def _operands(M, N, K, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    a = torch.randint(-127, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, device=dev, dtype=torch.int8)
    sa = torch.rand(M, generator=g, device=dev) + 0.01
    sw = torch.rand(N, generator=g, device=dev) * 1e-4 + 1e-6
    return a, sa, w, sw


def _check_matmul(B, M, N, K, f32, dev, ops=None):
    a, sa, w, sw = ops or _operands(M, N, K, dev, seed=M + N + K)
    guard = 64
    flat = torch.full((M * N + 2 * guard,), 77.0, dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    out = flat[guard:guard + M * N].view(M, N)
    B.moe_i8_matmul(a, sa, w, sw, out, _workspace(B, M, N, K, dev))
    torch.cuda.synchronize()
    want = orc.matmul(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())
    got = out.double().cpu().numpy()
    tol = (3.01 * 2 ** -24 + (0 if f32 else 2 ** -8)) * np.abs(want)
    assert (np.abs(got - want) <= tol).all()
    assert (flat[:guard] == 77.0).all() and (flat[-guard:] == 77.0).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 16, 128), (1, 4096, 7168), (2, 3, 48), (7, 129, 144), (8, 4096, 2048),
    (16, 1000, 1040), (17, 64, 64), (31, 333, 272), (33, 257, 1024), (64, 512, 4112), (65, 255, 80),
    (77, 1537, 2064), (127, 128, 128), (129, 1024, 7168), (200, 96, 8192), (256, 256, 256),
    (257, 513, 400), (300, 2048, 1408), (511, 300, 16), (1030, 1300, 528), (2100, 260, 7168),
    (600, 700, 2064), (1500, 1100, 528), (3000, 2300, 1040), (4100, 513, 656), (900, 4097, 2032)])
def test_matmul(B, dev, M, N, K, f32):
    _check_matmul(B, M, N, K, f32, dev)


@pytest.mark.parametrize("M,N,K", [(3, 40, 131072), (300, 300, 131072), (100, 128, 16384)])
def test_matmul_largest_sums(B, dev, M, N, K):
    """Every product 127^2: the sum comes within 2 % of 2^31."""
    a, sa, w, sw = _operands(M, N, K, dev)
    a.fill_(127)
    w.fill_(-127)
    w[::2] = 127
    _check_matmul(B, M, N, K, True, dev, (a, sa, w, sw))


def test_matmul_many_rows(B, dev):
    """A product of the size of a long prefill against the exact sums in float64."""
    M, N, K = 5000, 1537, 2064
    a, sa, w, sw = _operands(M, N, K, dev)
    out = torch.full((M, N), float("nan"), device=dev)
    B.moe_i8_matmul(a, sa, w, sw, out, _workspace(B, M, N, K, dev))
    want = (a.double() @ w.double().T.contiguous()) * sa.double()[:, None] * sw.double()[None, :]
    assert ((out.double() - want).abs() <= 3.01 * 2 ** -24 * want.abs()).all()


def test_matmul_refuses_wrong_tensors(B, dev):
    a, sa, w, sw = _operands(4, 8, 32, dev)
    out = torch.zeros(4, 8, dtype=torch.bfloat16, device=dev)
    with pytest.raises(TypeError):
        B.moe_i8_matmul(a.float(), sa, w, sw, out)
    with pytest.raises(ValueError):
        B.moe_i8_matmul(a, sa[:3], w, sw, out)
    with pytest.raises(ValueError):
        B.moe_i8_matmul(a, sa, w[:, :16], sw, out)
    with pytest.raises(TypeError):
        B.moe_i8_matmul(a, sa, w, sw, out.half())
    with pytest.raises(B.MoeError):
        B.moe_i8_matmul(a[:, :8].contiguous(), sa, w[:, :8].contiguous(), sw, out)


@pytest.mark.parametrize("M,N,K", [(8, 512, 1024), (300, 512, 1024), (1100, 640, 512), (100, 128, 16384)])
def test_matmul_graph_replays_equal_eager_calls(B, dev, M, N, K):
    a, sa, w, sw = _operands(M, N, K, dev)
    ws = _workspace(B, M, N, K, dev)
    out = torch.zeros(M, N, device=dev)
    other = torch.zeros(M, N, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.moe_i8_matmul(a, sa, w, sw, out, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_i8_matmul(a, sa, w, sw, out, ws)
    for seed in range(4):
        fresh = _operands(M, N, K, dev, seed=30 + seed)
        a.copy_(fresh[0])
        sa.copy_(fresh[1])
        out.zero_()
        B.moe_i8_matmul(fresh[0], fresh[1], w, sw, other, ws)     # eager work between replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, other)


# ---------------------------------------------------------------------------------------
# The layer
# ---------------------------------------------------------------------------------------
def _layer_inputs(B, M, H, E, I, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=dev) * std  # noqa: E731
    L = dict(x=n(M, H).bfloat16(), wr=n(E, H, std=1.7 / H ** 0.5).bfloat16(), bias=n(E, std=0.05),
             residual=n(M, H).bfloat16(), g=(1 + 0.05 * n(H)).bfloat16())
    L["w13"], L["s13"] = _quantize(B, n(E, 2 * I, H, std=1.0 / H ** 0.5).bfloat16())
    L["w2"], L["s2"] = _quantize(B, n(E, H, I, std=1.0 / I ** 0.5).bfloat16())
    return L


def _run_layer(B, L, k, block, rule, dev, with_bias=True, stream=None, events=None):
    M, H = L["x"].shape
    E, I = L["w13"].shape[0], L["w13"].shape[1] // 2
    r = dict(softmax=False, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0)
    r.update(rule)
    cap = B.moe_align_capacity(M, k, E, block)
    o = dict(out=torch.full((M, H), float("nan"), dtype=torch.bfloat16, device=dev),
             z=torch.full((M, H), float("nan"), dtype=torch.bfloat16, device=dev),
             ids=torch.full((M, k), -7, dtype=torch.int32, device=dev),
             w=torch.full((M, k), float("nan"), dtype=torch.float32, device=dev),
             sorted=torch.full((cap,), -7, dtype=torch.int32, device=dev),
             bexp=torch.full((cap // block,), -7, dtype=torch.int32, device=dev),
             npad=torch.full((1,), -7, dtype=torch.int32, device=dev))
    o["ws"] = torch.full((B.moe_i8_workspace_bytes(M, H, E, I, k, block),), 0xFF, dtype=torch.uint8,
                         device=dev)
    B.moe_forward_i8(L["x"], L["wr"], L["bias"] if with_bias else None, L["w13"], L["s13"], L["w2"],
                     L["s2"], L["residual"], L["g"], 1e-5, k, block, o["out"], o["ws"],
                     residual_out=o["z"], topk_ids_out=o["ids"], topk_w_out=o["w"],
                     sorted_ids_out=o["sorted"], block_expert_out=o["bexp"], num_padded_out=o["npad"],
                     score=1 if r["softmax"] else 0, n_group=r["n_group"], topk_group=r["topk_group"],
                     group_top=r["group_top"], renormalize=r["renormalize"], scale=r["scale"],
                     stream=stream, stage_events=events)
    torch.cuda.synchronize()
    return o, r


def _check_layer(B, L, k, block, rule, dev, with_bias=True):
    from oracle import moe_oracle
    o, r = _run_layer(B, L, k, block, rule, dev, with_bias)
    E = L["w13"].shape[0]
    rid, rw = orc.route(bits(L["x"]), bits(L["wr"]), L["bias"].cpu().numpy() if with_bias else None, k, **r)
    assert np.array_equal(o["ids"].cpu().numpy(), rid)
    plan = moe_oracle.align(rid, E, block)
    n_pad = int(o["npad"].item())
    assert n_pad == plan[2]
    assert np.array_equal(o["sorted"].cpu().numpy()[:n_pad], plan[0])
    assert np.array_equal(o["bexp"].cpu().numpy()[:n_pad // block], plan[1])
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    w2 = L["w2"].cpu().numpy()
    out, z, y = orc.layer(bits(L["x"]), rid, rw, L["w13"].cpu().numpy(), f64(L["s13"]), w2,
                          f64(L["s2"]), bits(L["residual"]), bits(L["g"]), 1e-5)
    M, H = z.shape
    wy = rw[:, :, None] * np.abs(y.reshape(M, k, H))
    # bf16 rows y past the first pick, and a moved code in each row
    extra = 2 ** -8 * wy[:, 1:].sum(1) + np.abs(rw).sum(1, keepdims=True) * 8.0 * float(L["s2"].max())
    norm = np.abs(out) / np.maximum(np.abs(z), 1e-9)
    bars.check_close(o["z"], z, "residual_out", extra=extra)
    bars.check_close(o["out"], out, "out", extra=extra * norm + 2 ** -8 * np.abs(out))
    return o


GROUPED = dict(n_group=4, topk_group=2, group_top=2, scale=2.5)
LAYERS = [  # M, H, E, I, k, block, rule: tokens per expert from 0.1 to over 128
    (1, 256, 8, 128, 2, 16, GROUPED), (4, 256, 8, 512, 2, 16, GROUPED),
    (1, 512, 64, 256, 8, 16, GROUPED), (37, 1040, 32, 272, 4, 16, dict(softmax=True)),
    (64, 272, 12, 48, 3, 32, GROUPED), (50, 768, 8, 512, 4, 64, dict(renormalize=False)),
    (203, 512, 60, 352, 4, 32, dict(softmax=True)), (130, 256, 4, 256, 1, 128, dict()),
    (300, 768, 8, 512, 4, 64, GROUPED), (600, 400, 8, 256, 3, 16, dict(softmax=True, renormalize=False)),
    (290, 16, 4, 16, 2, 16, dict()), (1, 16, 1, 16, 1, 16, dict()),
    # both products long enough in K for the step streams, at each token tile height
    (40, 656, 4, 768, 2, 16, dict()), (77, 1024, 8, 640, 4, 32, GROUPED),
    (205, 768, 4, 1408, 1, 16, dict()), (333, 896, 8, 640, 4, 64, GROUPED),
    (450, 784, 4, 768, 2, 16, dict(softmax=True)), (290, 1280, 4, 896, 3, 64, dict(scale=2.5)),
    # and with a partial last chunk of K
    (60, 528, 4, 656, 2, 16, dict()), (205, 784, 4, 1360, 1, 16, dict()),
    (450, 656, 4, 592, 2, 32, dict(softmax=True)), (300, 1040, 2, 624, 2, 64, dict()),
    # more results of the down product than are held in fp32
    (1100, 4096, 4, 640, 4, 64, dict()), (1030, 4096, 4, 48, 4, 16, dict(scale=2.5)),
    (200, 16384, 8, 16, 8, 16, dict(softmax=True)),
]


@pytest.mark.parametrize("case", LAYERS)
@pytest.mark.parametrize("with_bias", [True, False])
def test_layer(B, dev, case, with_bias):
    M, H, E, I, k, block, rule = case
    _check_layer(B, _layer_inputs(B, M, H, E, I, dev, seed=M + E), k, block, rule, dev, with_bias)


def test_layer_every_token_on_one_expert(B, dev):
    """A bias that sends every token to the same experts: one expert with every row."""
    L = _layer_inputs(B, 500, 512, 16, 256, dev, seed=4)
    L["bias"] = torch.zeros(16, device=dev)
    L["bias"][5] = 10.0
    L["bias"][9] = 5.0
    _check_layer(B, L, 2, 64, dict(), dev)


def test_layer_tokens_that_are_not_finite_stay_by_themselves(B, dev):
    L = _layer_inputs(B, 20, 512, 16, 256, dev, seed=5)
    want, _ = _run_layer(B, L, 4, 16, GROUPED, dev)
    L["x"][3, 100] = float("nan")
    got, _ = _run_layer(B, L, 4, 16, GROUPED, dev)
    keep = [t for t in range(20) if t != 3]
    assert torch.equal(got["ids"][keep], want["ids"][keep])
    assert torch.equal(got["out"][keep], want["out"][keep])
    assert not torch.isfinite(got["out"][3]).any()


def test_layer_without_optional_outputs_events_and_repeats(B, dev):
    L = _layer_inputs(B, 70, 512, 16, 256, dev, seed=6)
    events = [B.HipEvent() for _ in range(6)]
    first, _ = _run_layer(B, L, 4, 32, GROUPED, dev, events=events)
    assert all(B.HipEvent.elapsed_ms(events[i], events[i + 1]) >= 0 for i in range(5))
    out = torch.full_like(first["out"], float("nan"))
    B.moe_forward_i8(L["x"], L["wr"], L["bias"], L["w13"], L["s13"], L["w2"], L["s2"], L["residual"],
                     L["g"], 1e-5, 4, 32, out, first["ws"], n_group=4, topk_group=2, group_top=2, scale=2.5)
    torch.cuda.synchronize()
    assert torch.equal(out, first["out"])
    for _ in range(20):
        again, _ = _run_layer(B, L, 4, 32, GROUPED, dev)
        assert torch.equal(again["out"], first["out"]) and torch.equal(again["z"], first["z"])


@pytest.mark.parametrize("M", [4, 300])
def test_layer_graph_replays_equal_eager_calls(B, dev, M):
    L = _layer_inputs(B, M, 512, 16, 256, dev, seed=7)
    k, block = 4, 16
    ws = torch.empty(B.moe_i8_workspace_bytes(M, 512, 16, 256, k, block), dtype=torch.uint8, device=dev)
    out = torch.zeros(M, 512, dtype=torch.bfloat16, device=dev)
    api = dict(n_group=4, topk_group=2, group_top=2, scale=2.5)
    call = lambda: B.moe_forward_i8(  # noqa: E731
        L["x"], L["wr"], L["bias"], L["w13"], L["s13"], L["w2"], L["s2"], L["residual"], L["g"], 1e-5,
        k, block, out, ws, **api)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(4):
        L["x"].copy_(torch.randn(M, 512, generator=torch.Generator().manual_seed(seed)).bfloat16())
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, _ = _run_layer(B, L, k, block, GROUPED, dev)
        assert torch.equal(out, want["out"])


def test_two_layers_at_once_on_two_streams(B, dev):
    layers = [_layer_inputs(B, M, 768, 8, 640, dev, seed=20 + M) for M in (9, 300)]
    want = [_run_layer(B, L, 4, 16, GROUPED, dev)[0] for L in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.full_like(w["out"], float("nan")) for w in want]
    room = [torch.empty_like(w["ws"]) for w in want]
    torch.cuda.synchronize()
    for _ in range(4):
        for L, s, o, ws in zip(layers, streams, outs, room):
            B.moe_forward_i8(L["x"], L["wr"], L["bias"], L["w13"], L["s13"], L["w2"], L["s2"],
                             L["residual"], L["g"], 1e-5, 4, 16, o, ws, n_group=4, topk_group=2,
                             group_top=2, scale=2.5, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w["out"]) for o, w in zip(outs, want))


def test_a_workspace_of_more_tokens_does_for_fewer(B, dev):
    H, E, I, k, block = 768, 8, 640, 4, 16
    ws = torch.empty(B.moe_i8_workspace_bytes(300, H, E, I, k, block), dtype=torch.uint8, device=dev)
    for M in (300, 5, 260, 1, 130):
        assert B.moe_i8_workspace_bytes(M, H, E, I, k, block) <= ws.numel()
        L = _layer_inputs(B, M, H, E, I, dev, seed=M)
        want = _run_layer(B, L, k, block, GROUPED, dev)[0]["out"]
        out = torch.full_like(want, float("nan"))
        B.moe_forward_i8(L["x"], L["wr"], L["bias"], L["w13"], L["s13"], L["w2"], L["s2"],
                         L["residual"], L["g"], 1e-5, k, block, out, ws, n_group=4, topk_group=2,
                         group_top=2, scale=2.5)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_tensors_of_another_device_are_refused(B, dev, monkeypatch):
    v = torch.zeros(4, 32, dtype=torch.bfloat16, device=dev)
    codes, scales = _quantize(B, v)
    l, ids = torch.zeros(4, 8, device=dev), torch.zeros(4, 2, dtype=torch.int32, device=dev)
    out = torch.empty(4, 4, device=dev)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        B.moe_i8_quantize(v, codes, scales)
    with pytest.raises(ValueError, match="current device"):
        B.moe_i8_matmul(codes, scales, codes, scales, out)
    with pytest.raises(ValueError, match="current device"):
        B.moe_route_logits(l, None, 2, ids, torch.zeros(4, 2, device=dev))


def test_layer_beside_a_shared_expert_on_the_same_rows(B, dev):
    """The operators together, as a layer with a shared expert uses them: quantize the tokens
    once, the shared expert through two products, its result in the residual, then the layer
    from logits' routing and from its own: the same experts."""
    M, H, E, I, k = 48, 512, 16, 256, 4
    L = _layer_inputs(B, M, H, E, I, dev, seed=8)
    g = torch.Generator(device=dev).manual_seed(1)
    s13, c13s = _quantize(B, (torch.randn(2 * I, H, generator=g, device=dev) / H ** 0.5).bfloat16())
    s2, c2s = _quantize(B, (torch.randn(H, I, generator=g, device=dev) / I ** 0.5).bfloat16())
    xq, xs = _quantize(B, L["x"])
    h = torch.empty(M, 2 * I, device=dev)
    B.moe_i8_matmul(xq, xs, s13, c13s, h, _workspace(B, M, 2 * I, H, dev))
    act = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]).bfloat16().contiguous()
    aq, a_s = _quantize(B, act)
    shared = torch.empty(M, H, device=dev)
    B.moe_i8_matmul(aq, a_s, s2, c2s, shared, _workspace(B, M, H, I, dev))
    L["residual"] = (L["residual"].float() + shared).bfloat16()
    o = _check_layer(B, L, k, 16, GROUPED, dev)
    logits = (L["x"].double() @ L["wr"].double().T.contiguous()).float()
    ids = torch.empty(M, k, dtype=torch.int32, device=dev)
    w = torch.empty(M, k, device=dev)
    B.moe_route_logits(logits, L["bias"], k, ids, w, **GROUPED)
    torch.cuda.synchronize()
    assert torch.equal(ids, o["ids"])
    assert torch.allclose(w, o["w"], rtol=1e-5)
    want = orc.matmul(xq.cpu().numpy(), xs.cpu().numpy(), s13.cpu().numpy(), c13s.cpu().numpy())
    assert (np.abs(h.double().cpu().numpy() - want) <= 3.01 * 2 ** -24 * np.abs(want)).all()
