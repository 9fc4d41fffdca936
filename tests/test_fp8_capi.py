"""Arguments of the router and of the block-scaled FP8 calls that the host refuses before any launch.  CPU only."""
import ctypes

import pytest

OK, NULL, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from w8a8_dynamic_quant_gb300 import _capi, build
    build.build()
    return _capi.lib()


P = ctypes.c_void_p(256)
BIG = 1 << 34


def gate(lib, T=4, E=64, bias=None, n_group=1, topk_group=1, k=2, scale=1.0, flags=0, logits=P, ids=P, w=P):
    return lib.moe_gate_topk(logits, T, E, bias, n_group, topk_group, k, scale, flags, ids, w, None)


def test_gate_refusals(lib):
    assert gate(lib, T=0) == OK  # nothing to do
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(k=65, E=64), dict(n_group=0),
                dict(n_group=3), dict(n_group=64), dict(n_group=8, topk_group=0), dict(n_group=8, topk_group=9),
                dict(n_group=8, topk_group=1, k=9), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(flags=16), dict(T=1 << 30)):
        assert gate(lib, **bad) == SHAPE, bad
    for bad in (dict(logits=None), dict(ids=None), dict(w=None)):
        assert gate(lib, **bad) == NULL, bad


def test_quant_refusals(lib):
    for f in (lib.w8a8_fp8_quant, lib.w8a8_fp8_swiglu_quant):
        assert f(P, 0, 128, P, P, None) == OK
        assert f(P, -1, 128, P, P, None) == SHAPE
        assert f(P, 4, 0, P, P, None) == SHAPE
        assert f(P, 4, 65552, P, P, None) == SHAPE
        assert f(P, 4, 136, P, P, None) == ALIGN
        assert f(ctypes.c_void_p(8), 4, 128, P, P, None) == ALIGN
        assert f(P, 4, 128, ctypes.c_void_p(8), P, None) == ALIGN
        assert f(None, 4, 128, P, P, None) == NULL
        assert f(P, 4, 128, None, P, None) == NULL
        assert f(P, 4, 128, P, None, None) == NULL


def dense(lib, q=P, xs=P, M=4, K=128, w=P, ws_=P, N=8, y=P, ws=P, n=BIG):
    return lib.w8a8_fp8_matmul(q, xs, M, K, w, ws_, N, None, y, ws, n, None)


def grouped(lib, q=P, xs=P, gl=P, E=4, R=8, K=128, w=P, ws_=P, N=8, y=P, ws=P, n=BIG):
    return lib.w8a8_fp8_grouped_matmul(q, xs, gl, E, R, K, w, ws_, N, y, ws, n, None)


def test_matmul_refusals(lib):
    assert dense(lib, M=0) == OK and grouped(lib, R=0) == OK
    for f in (dense, grouped):
        for bad in (dict(K=0), dict(K=65552), dict(N=0), dict(N=1 << 31)):
            assert f(lib, **bad) == SHAPE, bad
        for bad in (dict(K=136), dict(q=ctypes.c_void_p(8)), dict(w=ctypes.c_void_p(8))):
            assert f(lib, **bad) == ALIGN, bad
        for bad in (dict(q=None), dict(xs=None), dict(w=None), dict(ws_=None), dict(y=None)):
            assert f(lib, **bad) == NULL, bad
        for bad in (dict(ws=None), dict(n=256), dict(ws=ctypes.c_void_p(8))):
            assert f(lib, **bad) == WORKSPACE, bad
    assert dense(lib, M=-1) == SHAPE and dense(lib, M=1 << 31) == SHAPE
    for bad in (dict(E=0), dict(E=1025), dict(R=-1), dict(E=1024, N=1 << 22)):
        assert grouped(lib, **bad) == SHAPE, bad
    assert grouped(lib, gl=None) == NULL


def test_layer_refusals(lib):
    def layer(x=P, ids=P, wt=P, T=4, k=2, E=8, H=128, I=128, w13=P, s13=P, w2=P, s2=P, ws=P, n=BIG, y=P):
        return lib.moe_fp8_layer(x, ids, wt, T, k, E, H, I, w13, s13, w2, s2, ws, n, y, None)
    assert layer(T=0) == OK
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(E=1025), dict(H=0), dict(I=0), dict(T=1 << 30, k=4),
                dict(E=1024, I=1 << 16 | 16)):
        assert layer(**bad) == SHAPE, bad
    for bad in (dict(H=136), dict(I=72), dict(x=ctypes.c_void_p(8)), dict(y=ctypes.c_void_p(8)),
                dict(w13=ctypes.c_void_p(8)), dict(w2=ctypes.c_void_p(8))):
        assert layer(**bad) == ALIGN, bad
    for bad in (dict(x=None), dict(ids=None), dict(wt=None), dict(w13=None), dict(s13=None), dict(w2=None),
                dict(s2=None), dict(y=None)):
        assert layer(**bad) == NULL, bad
    assert layer(ws=None) == WORKSPACE and layer(n=256) == WORKSPACE


def test_workspace_sizes(lib):
    assert lib.w8a8_fp8_matmul_workspace_bytes(0, 0, 128) == 0
    assert lib.w8a8_fp8_grouped_matmul_workspace_bytes(0, 4, 8, 128) == 0
    assert lib.w8a8_fp8_grouped_matmul_workspace_bytes(1025, 4, 8, 128) == 0
    assert lib.moe_fp8_layer_workspace_bytes(4, 0, 128, 128, 8) == 0
    # a problem whose tiles are not cut needs the status word and counters only, a cut one at most 76 pairs' pieces
    assert lib.w8a8_fp8_matmul_workspace_bytes(8192, 14336, 4096) < 1 << 14
    assert lib.w8a8_fp8_grouped_matmul_workspace_bytes(8, 4096, 4096, 4096) <= 76 * 4 * 128 * 256 * 4 + (1 << 14)
    R, H, I = 77 * 3, 384, 208
    assert lib.moe_fp8_layer_workspace_bytes(77, 3, H, I, 12) >= R * (H + 4 * I + I + 2 * H)


def test_pad_inner():
    """Weights laid out for the layer: each half's channels and w2's columns end on whole blocks, in zero codes."""
    import torch
    import w8a8_dynamic_quant_gb300 as W
    E, I, H = 2, 208, 48
    w13 = torch.randint(0, 127, (E, 2 * I, H), dtype=torch.uint8).view(torch.float8_e4m3fn)
    w2 = torch.randint(0, 127, (E, H, I), dtype=torch.uint8)
    s = torch.rand(E, 2, 2, 1)
    p13, ps, p2 = W.moe_fp8_pad_inner(w13, s, w2)
    assert p13.dtype == w13.dtype and p2.dtype == w2.dtype and torch.equal(ps, s)
    assert p13.shape == (E, 512, H) and p2.shape == (E, H, 256) and p13.is_contiguous() and p2.is_contiguous()
    a, b = p13.view(torch.uint8), w13.view(torch.uint8)
    assert torch.equal(a[:, :I], b[:, :I]) and torch.equal(a[:, 256:256 + I], b[:, I:])
    assert not a[:, I:256].any() and not a[:, 256 + I:].any()
    assert torch.equal(p2[:, :, :I], w2) and not p2[:, :, I:].any()
    whole = torch.zeros(E, 512, H, dtype=torch.uint8)
    p13, ps, p2 = W.moe_fp8_pad_inner(whole, s, torch.zeros(E, H, 256, dtype=torch.uint8))
    assert p13 is whole
    for bad in ((w13, s[:, 0], w2), (w13[:, :-1], s, w2), (w13, s, w2[:, :, 1:]), (w13, s[:, :, :1], w2)):
        with pytest.raises(ValueError):
            W.moe_fp8_pad_inner(*bad)
    for bad in ((w13.float(), s, w2), (w13, s.double(), w2), (w13, s, w2.short())):
        with pytest.raises(TypeError):
            W.moe_fp8_pad_inner(*bad)
