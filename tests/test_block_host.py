"""CPU checks of the block norm, the bf16 product and the few-token layer: sizes, and every
refusal of the C entry points and of the binding (these paths return before any HIP call)."""
import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from prefill_sigmoid_router_amd import binding, build
    if not os.path.exists(binding.library_path()):
        build.build()
    binding.load_library()
    return binding


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _norm(lib, **kw):
    a = dict(y=256, y_f32=0, y_ld=64, r=256, r_f32=0, r_ld=64, gate=None, g_cols=64, g_ld=0, post=1,
             post_w=256, post_b=None, pre=1, pre_w=256, pre_b=None, eps=1e-5, off=0.0, a=1.0, b=1.0,
             M=4, H=64, z=256, z_ld=64, out=256, out_ld=64)
    a.update(kw)
    return lib.moe_block_norm(_p(a["y"]), a["y_f32"], a["y_ld"], _p(a["r"]), a["r_f32"], a["r_ld"],
                              _p(a["gate"]), a["g_cols"], a["g_ld"], a["post"], _p(a["post_w"]),
                              _p(a["post_b"]), a["pre"], _p(a["pre_w"]), _p(a["pre_b"]), a["eps"],
                              a["off"], a["a"], a["b"], a["M"], a["H"], _p(a["z"]), a["z_ld"],
                              _p(a["out"]), a["out_ld"], None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(M=(1 << 30) + 1), dict(H=0), dict(H=60), dict(H=16392, y_ld=16392),
    dict(y_f32=2), dict(r_f32=-1), dict(post=3), dict(pre=-1), dict(eps=0.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(off=float("nan")), dict(a=float("inf")), dict(b=float("nan")),
    dict(y=None, r=None, post=0), dict(z=None, out=None), dict(y=None), dict(y=None, post=0, gate=256),
    dict(y_ld=56), dict(y_ld=68), dict(r_ld=0), dict(z_ld=60), dict(out_ld=-64),
    dict(gate=256, g_cols=2), dict(gate=256, g_ld=56), dict(gate=256, g_ld=68), dict(gate=257, g_cols=1),
    dict(gate=256, g_cols=1, g_ld=-1), dict(gate=264), dict(y=264), dict(r=258), dict(z=8), dict(out=24),
    dict(post_w=264), dict(post_b=258), dict(pre_w=8), dict(pre_b=2),
])
def test_block_norm_refuses(B, bad):
    assert _norm(B.load_library(), **bad) == -1


def test_block_norm_without_tokens(B):
    assert _norm(B.load_library(), M=0, y=None, r=None, z=None, out=None) == 0


def _matmul(lib, **kw):
    a = dict(x=256, x_ld=64, w=256, bias=None, M=4, N=32, K=64, act=0, gated=0, r=None, r_f32=0, r_ld=0,
             out=256, out_f32=0, out_ld=32, ws=None, wsb=0)
    a.update(kw)
    return lib.moe_matmul(_p(a["x"]), a["x_ld"], _p(a["w"]), _p(a["bias"]), a["M"], a["N"], a["K"],
                          a["act"], a["gated"], _p(a["r"]), a["r_f32"], a["r_ld"], _p(a["out"]),
                          a["out_f32"], a["out_ld"], _p(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(M=-1), -1), (dict(M=(1 << 24) + 1), -1), (dict(N=0), -1), (dict(N=(1 << 24) + 1), -1),
    (dict(K=0), -1), (dict(K=60), -1), (dict(K=(1 << 20) + 8, x_ld=1 << 21), -1), (dict(act=5), -1),
    (dict(act=-1), -1), (dict(gated=2), -1), (dict(out_f32=2), -1), (dict(r_f32=7), -1),
    (dict(M=1 << 24, N=1 << 14, out_ld=1 << 14), -2), (dict(x=None), -1), (dict(w=None), -1),
    (dict(out=None), -1), (dict(x_ld=56), -1), (dict(x_ld=68), -1), (dict(out_ld=31), -1),
    (dict(r=256, r_ld=31), -1), (dict(x=264), -1), (dict(w=258), -1), (dict(out=8), -1),
    (dict(bias=258), -1), (dict(r=264, r_ld=32), -1),
])
def test_matmul_refuses(B, bad, code):
    assert _matmul(B.load_library(), **bad) == code


def test_matmul_workspace(B):
    assert _matmul(B.load_library(), M=0, x=None, w=None, out=None) == 0
    for bad in ((-1, 32, 64), (4, 0, 64), (4, 32, 60), (4, 32, 0)):
        assert B.moe_matmul_workspace_bytes(*bad) == 0
    for sizes in ((1, 1, 8), (8, 4096, 7168), (300, 512, 7168), (8192, 4096, 7168)):
        need = B.moe_matmul_workspace_bytes(*sizes)
        if need:
            M, N, K = sizes
            ok = dict(M=M, N=N, K=K, x_ld=K, out_ld=N)
            for ws, wsb in ((None, need), (256, need - 1), (264, need)):
                assert _matmul(B.load_library(), ws=ws, wsb=wsb, **ok) == -3


def test_matmul_tile_rows(B):
    rows = B.moe_matmul_tile_rows
    assert [rows(M, 7168, 2048) for M in (1, 8, 9, 16, 17, 32)] == [8, 8, 16, 16, 32, 32]
    assert (rows(640, 2048, 2048), rows(640, 4096, 7168), rows(2048, 7168, 2048)) == (64, 128, 256)
    assert (rows(640, 4096, 7168, True), rows(8192, 2048, 7168, True)) == (128, 256)
    # K in parts: on tiles of 64 rows only
    assert B.moe_matmul_workspace_bytes(200, 1024, 8200) > 0 and rows(200, 1024, 8200) == 64
    # one chunk of K is too short for the largest tiles
    assert rows(8192, 8192, 72) == 256 and rows(8192, 8192, 64) < 256
    # rows of x too far apart for them
    assert rows(2048, 7168, 2048, x_ld=1 << 23) == 256 and rows(2048, 7168, 2048, x_ld=(1 << 23) + 8) == 128
    for bad in ((-1, 32, 64), (4, 0, 64), (4, 32, 60), (1 << 24, 1 << 14, 64)):
        assert rows(*bad) == 0
    assert rows(4, 32, 64, x_ld=56) == 0 and rows(4, 32, 64, x_ld=68) == 0


def _few(lib, **kw):
    a = dict(x=256, rw=256, rb=None, sb=None, w13=256, w2=256, res=256, g=256, eps=1e-5, M=4, H=256, E=8,
             I=512, k=2, score=0, n_group=1, topk_group=1, group_top=1, renorm=1, scale=1.0, out=256,
             rout=None, ids=None, w=None, ws=256, wsb=1 << 40)
    a.update(kw)
    return lib.moe_forward_few(_p(a["x"]), _p(a["rw"]), _p(a["rb"]), _p(a["sb"]), _p(a["w13"]), _p(a["w2"]),
                               _p(a["res"]), _p(a["g"]), a["eps"], a["M"], a["H"], a["E"], a["I"], a["k"],
                               a["score"], a["n_group"], a["topk_group"], a["group_top"], a["renorm"],
                               a["scale"], _p(a["out"]), _p(a["rout"]), _p(a["ids"]), _p(a["w"]),
                               _p(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(M=-1), -1), (dict(M=17), -2), (dict(M=16, E=64, k=33), -2), (dict(k=0), -1), (dict(k=9), -1),
    (dict(E=1025), -1), (dict(H=250), -1), (dict(H=16392), -1), (dict(I=40), -1), (dict(I=32784), -2),
    (dict(eps=0.0), -1), (dict(eps=float("nan")), -1), (dict(score=2), -1), (dict(n_group=3), -1),
    (dict(n_group=4, topk_group=5), -1), (dict(group_top=3), -1), (dict(n_group=4, topk_group=1, k=3), -1),
    (dict(scale=float("inf")), -1), (dict(x=None), -1), (dict(rw=None), -1), (dict(w13=None), -1),
    (dict(w2=None), -1), (dict(out=None), -1), (dict(g=None), -1), (dict(x=264), -1), (dict(w13=264), -1),
    (dict(w2=258), -1), (dict(rw=8), -1), (dict(res=264), -1), (dict(g=8), -1), (dict(out=264), -1),
    (dict(rout=264), -1), (dict(rb=258), -1), (dict(sb=257), -1), (dict(ids=258), -1), (dict(w=258), -1),
    (dict(ws=None), -3), (dict(ws=64), -3), (dict(wsb=1000), -3),
])
def test_few_refuses(B, bad, code):
    assert _few(B.load_library(), **bad) == code


def test_few_sizes(B):
    assert _few(B.load_library(), M=0, x=None, out=None, ws=None, wsb=0) == 0
    assert B.moe_few_workspace_bytes(17, 256, 8, 512, 2) == 0
    assert B.moe_few_workspace_bytes(16, 256, 64, 512, 33) == 0
    assert B.moe_few_workspace_bytes(4, 256, 8, 520, 2) == 0
    M, H, E, I, k = 16, 7168, 256, 2048, 16
    need = M * E * 8 + M * k * (H + I) * 4
    assert need <= B.moe_few_workspace_bytes(M, H, E, I, k) <= need + 8192
    # a workspace for some number of tokens does for fewer
    sizes = [B.moe_few_workspace_bytes(m, H, E, I, k) for m in range(0, 17)]
    assert sizes == sorted(sizes)
    assert (B.FEW_MAX_TOKENS, B.FEW_MAX_PICKS) == (16, 512)


@pytest.mark.parametrize("I", [32784, 65536, 1 << 24, 1 << 29, 1 << 30, (1 << 31) - 16])
def test_few_refuses_wide_experts(B, I):
    """I past what the call takes, also where the bytes of a row of act pass 32 bits."""
    assert B.moe_few_workspace_bytes(1, 8, 1, I, 1) == 0
    assert _few(B.load_library(), M=1, H=8, E=1, I=I, k=1, wsb=1 << 62) == -2


def test_binding_refuses_host_tensors_and_wrong_types(B):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="device"):
        B.moe_block_norm(bf(4, 64), bf(4, 64), bf(4, 64))
    with pytest.raises(ValueError, match="y or residual"):
        B.moe_block_norm(None, None, bf(4, 64))
    with pytest.raises(ValueError, match="device"):
        B.moe_matmul(bf(4, 64), bf(32, 64), bf(4, 32))
    with pytest.raises(TypeError):
        B.moe_matmul([[1.0]], bf(32, 64), bf(4, 32))
    with pytest.raises(ValueError, match="device"):
        B.moe_forward_few(bf(4, 256), bf(8, 256), None, bf(8, 1024, 256), bf(8, 256, 512), bf(4, 256),
                          bf(256), 1e-5, 2, bf(4, 256), torch.zeros(1, dtype=torch.uint8))
