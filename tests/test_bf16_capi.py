"""Arguments of the norm with 8-bit outputs and of the bf16 products that the host refuses before any launch.  CPU only."""
import ctypes

import pytest

OK, NULL, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from w8a8_dynamic_quant_gb300 import _capi, build
    build.build()
    return _capi.lib()


P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)  # 8-byte aligned
INF, NAN = float("inf"), float("nan")


def norms(lib):
    return lib.w8a8_rms_norm_quant, lib.w8a8_fp8_rms_norm_quant, lib.w8a8_mx_rms_norm_quant


def norm(f, x=P, res=None, w=P, M=4, K=128, eps=1e-6, flags=0, out=None, y=None, q=P, s=P):
    return f(x, res, w, M, K, eps, flags, out, y, q, s, None)


def test_norm_refusals(lib):
    for f in norms(lib):
        assert norm(f, M=0) == OK
        for bad in (dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=-16), dict(K=65552), dict(eps=0.0), dict(eps=-1.0),
                    dict(eps=NAN), dict(eps=INF), dict(flags=2)):
            assert norm(f, **bad) == SHAPE, bad
        for bad in (dict(K=136), dict(x=ODD), dict(w=ODD), dict(q=ODD), dict(y=ODD), dict(res=ODD, out=P),
                    dict(res=P, out=ODD)):
            assert norm(f, **bad) == ALIGN, bad
        for bad in (dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(res=P), dict(out=P)):
            assert norm(f, **bad) == NULL, bad
    assert norm(lib.w8a8_mx_rms_norm_quant, K=144) == ALIGN  # a group of 32 must not end inside a row


def dense(lib, x=P, M=4, K=128, w=P, N=8, bias=None, act=0, res=None, flags=0, y=P, ws=P, n=256):
    return lib.w8a8_bf16_matmul(x, M, K, w, N, bias, act, res, flags, y, ws, n, None)


def grouped(lib, x=P, gl=P, E=4, R=8, K=128, w=P, N=8, bias=None, act=0, flags=0, y=P, ws=P, n=256):
    return lib.w8a8_bf16_grouped_matmul(x, gl, E, R, K, w, N, bias, act, flags, y, ws, n, None)


def test_matmul_refusals(lib):
    assert dense(lib, M=0) == OK and grouped(lib, R=0) == OK and grouped(lib, R=0, gl=None) == OK
    for f in (dense, grouped):
        for bad in (dict(K=0), dict(K=65552), dict(N=0), dict(N=1 << 31), dict(N=(1 << 31) - 256), dict(act=-1),
                    dict(act=6), dict(flags=2), dict(act=5, N=1 << 30)):
            assert f(lib, **bad) == SHAPE, bad
        for bad in (dict(K=136), dict(x=ODD), dict(w=ODD)):
            assert f(lib, **bad) == ALIGN, bad
        for bad in (dict(x=None), dict(w=None), dict(y=None)):
            assert f(lib, **bad) == NULL, bad
        for bad in (dict(ws=None), dict(n=255), dict(ws=ODD)):
            assert f(lib, **bad) == WORKSPACE, bad
    # a tile's last rows have coordinates of 32 bits: 256 below 2^31 at most
    assert dense(lib, M=-1) == SHAPE and dense(lib, M=(1 << 31) - 256) == SHAPE
    for bad in (dict(E=0), dict(E=1025), dict(R=-1), dict(R=(1 << 31) - 256), dict(E=1024, N=1 << 21),
                dict(E=1024, N=1 << 20, act=5)):
        assert grouped(lib, **bad) == SHAPE, bad
    assert grouped(lib, gl=None) == NULL


def test_workspace_sizes(lib):
    assert lib.w8a8_bf16_matmul_workspace_bytes(8192, 14336, 4096) >= 256
    assert lib.w8a8_bf16_matmul_workspace_bytes(-1, 8, 128) == 0
    assert lib.w8a8_bf16_matmul_workspace_bytes(4, 0, 128) == 0
    assert lib.w8a8_bf16_grouped_matmul_workspace_bytes(8, 100, 64, 128) >= 256
    assert lib.w8a8_bf16_grouped_matmul_workspace_bytes(1025, 100, 64, 128) == 0


def test_names_and_types():
    """What the binding refuses before it looks for a device."""
    import torch
    import w8a8_dynamic_quant_gb300 as W
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.zeros(8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="activation"):
        W.w8a8_bf16_matmul(x, w, activation="tanh")
    for f in (W.w8a8_rms_norm_quant, W.w8a8_fp8_rms_norm_quant, W.w8a8_mx_rms_norm_quant):
        with pytest.raises(ValueError, match="CUDA"):
            f(x, torch.ones(128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        W.w8a8_bf16_matmul(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        W.w8a8_bf16_grouped_matmul(x, torch.tensor([4]), w[None])
    with pytest.raises(ValueError):
        W.w8a8_bf16_matmul(x[0], w)
    with pytest.raises(TypeError):
        W.w8a8_bf16_matmul(None, w)
