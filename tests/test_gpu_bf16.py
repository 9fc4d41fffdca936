"""The bf16 products with bias, activation and residual, dense and grouped, against plain 64-bit implementations at the
sizes where a tile, a group, a row or a part of K ends early.

Tolerance of an output.  Products of bf16 are exact in binary32.  The sum of K of them is taken in binary32 whose
roundings may truncate: each of the ceil(K / 16) additions into the accumulator loses at most 2^-23 of the largest
partial sum, and within a group of 16 the terms are aligned to the largest with 2^-23 of it lost per term at most, so a
sum is off by at most (K / 16 + 16) 2^-23 A, A the sum of magnitudes; parts of K add 8 roundings, bias one.  An
activation with a derivative of at most 1.13 carries that on and adds its own roundings: exp and the quotient stay within
(2 + 1.17 |z| + 3) 2^-23 relative, where z is at most 88 before the factor vanishes (z = 2u for the tanh form, whose
argument's own five roundings give 5 * 2^-24 |z| more in the exponent): 300 * 2^-23 of the value is above all of them.
The residual's sum rounds once, and the output once: 2^-8 of it for bf16, 2^-24 for fp32."""
import math

import pytest
import torch

import w8a8_dynamic_quant_gb300 as W
from w8a8_dynamic_quant_gb300 import _capi

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def act64(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def reference(x, w, bias, act, residual):
    """(value, bound of the error before the last rounding) in 64 bits; x [M,K], w [rows,K]."""
    K = x.shape[1]
    v = x.double() @ w.double().t()
    a = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        v = v + bias.double()
        a = a + bias.double().abs()
    err = (K / 16 + 16 + 8 + 1) * 2.0 ** -23 * a
    if act == "swiglu":
        g, u = v.chunk(2, 1)
        eg, eu = err.chunk(2, 1)
        s = g * torch.sigmoid(g)
        v = s * u
        err = 1.13 * eg * (u.abs() + eu) + (s.abs() + 1.13 * eg) * eu + 300 * 2.0 ** -23 * v.abs()
    elif act != "none":
        v = act64(v, act)
        err = 1.13 * err + 300 * 2.0 ** -23 * v.abs()
    if residual is not None:
        v = v + residual.double()
        err = err + 2.0 ** -24 * v.abs()
    return v, err


def close(y, v, err):
    half = 2.0 ** -8 if y.dtype is torch.bfloat16 else 2.0 ** -24
    tiny = 2.0 ** -133 if y.dtype is torch.bfloat16 else 2.0 ** -149
    bad = (y.double() - v).abs() > err + half * (v.abs() + err) + tiny
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((y.double() - v).abs().max()))


def inputs(M, N, K, act, bias, residual, seed):
    g = gen(seed)
    rows = 2 * N if act == "swiglu" else N
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(rows, K, generator=g, device="cuda") * 2 * K ** -0.5).to(torch.bfloat16)
    b = torch.randn(rows, generator=g, device="cuda").to(torch.bfloat16) if bias else None
    r = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    return x, w, b, r


# one token; tiles of 32, 64, 128 and 256 tokens, whole and cut; parts of K; rows on no 16-byte boundary; K inside a block
SHAPES = [(1, 1, 16), (1, 8, 16), (1, 7168, 2048), (2, 40, 48), (16, 256, 512), (17, 257, 528), (33, 130, 1040),
          (64, 2048, 7168), (65, 1001, 208), (127, 96, 64), (128, 256, 7168), (129, 384, 4096), (200, 72, 16),
          (257, 129, 144), (300, 4096, 256), (511, 513, 1040), (777, 2056, 96), (1141, 1416, 2000), (3000, 64, 512),
          (2048, 4096, 1024)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_plain(M, N, K):
    x, w, b, r = inputs(M, N, K, "none", True, True, M + N + K)
    for out in (torch.bfloat16, torch.float32):
        for bias, res in ((None, None), (b, r)):
            close(W.w8a8_bf16_matmul(x, w, bias, residual=res, out_dtype=out), *reference(x, w, bias, "none", res))


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("M,N,K", [(1, 24, 80), (5, 2048, 1024), (40, 33, 512), (70, 264, 1024), (128, 192, 2048),
                                   (250, 1000, 336), (1100, 1416, 400), (1500, 2500, 64)])
def test_activations(M, N, K, act):
    x, w, b, r = inputs(M, N, K, act, True, True, M * N + K)
    for out, bias, res in ((torch.bfloat16, b, r), (torch.float32, b, None), (torch.bfloat16, None, None),
                           (torch.float32, None, r)):
        close(W.w8a8_bf16_matmul(x, w, bias, act, res, out), *reference(x, w, bias, act, res))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "swiglu"])
def test_far_activations(act):
    """Values far out on both sides, where exp, erfc or a cube would leave their range."""
    M, K = 8, 16
    far = torch.tensor([-3e38, -1e20, -1000.0, -110.0, -89.0, -40.0, -13.0, -9.0, -5.0, -1.0, -0.0, 0.0, 1.0, 5.0, 9.0,
                        13.0, 89.0, 110.0, 1e4, 1e20, 3e38], device="cuda")
    N = far.numel()
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 1.0
    w = torch.zeros(N, K, device="cuda", dtype=torch.bfloat16)
    w[:, 0] = far
    if act == "swiglu":
        up = torch.zeros(N, K, device="cuda", dtype=torch.bfloat16)
        up[:, 0] = torch.where(far.abs() > 1e19, 1.0, 3.0)
        w = torch.cat([w, up])
    y = W.w8a8_bf16_matmul(x, w, activation=act, out_dtype=torch.float32)
    v, err = reference(x, w, None, act, None)
    # what is below 2^-126 / 88 has lost digits or is gone: exp of less than -87.3 is below the normal values
    assert bool(((y.double() - v).abs() <= err + 2.0 ** -24 * v.abs() + 2.0 ** -119).all()), (y[0].tolist(), v[0].tolist())


def grouped_reference(x, counts, w, bias, act):
    vs, es, at = [], [], 0
    for e, n in enumerate(counts):
        if n:
            v, err = reference(x[at:at + n], w[e], None if bias is None else bias[e], act, None)
            vs.append(v)
            es.append(err)
        at += n
    return torch.cat(vs), torch.cat(es)


COUNTS = [[5], [0, 0, 3, 0], [1, 0, 17, 40, 16, 15, 0, 2], [300, 0, 1, 255, 256, 257, 31, 0, 33], [64] * 20,
          [0, 1000, 3, 0, 0, 129, 128, 127], [1] * 70 + [0] * 30 + [2] * 28]


@pytest.mark.parametrize("counts", COUNTS, ids=[str(i) for i in range(len(COUNTS))])
@pytest.mark.parametrize("act,N,K,bias", [("none", 200, 144, True), ("swiglu", 136, 528, True), ("gelu", 257, 64, False),
                                          ("swiglu", 77, 96, False)])
def test_grouped(counts, act, N, K, bias):
    E, R = len(counts), sum(counts)
    g = gen(R + N)
    rows = 2 * N if act == "swiglu" else N
    x = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(E, rows, K, generator=g, device="cuda") * 2 * K ** -0.5).to(torch.bfloat16)
    b = torch.randn(E, rows, generator=g, device="cuda").to(torch.bfloat16) if bias else None
    gl = torch.tensor(counts, dtype=torch.int64, device="cuda")
    ws = W.workspace(W.bf16_grouped_matmul_workspace_bytes(E, R, N, K))
    v, err = grouped_reference(x, counts, w, b, act)
    for out in (torch.bfloat16, torch.float32):
        close(W.w8a8_bf16_grouped_matmul(x, gl, w, b, act, out, ws=ws), v, err)
    assert W.read_device_status(ws) == 0


@pytest.mark.parametrize("counts", [[3, 4], [3, 6], [-1, 9], [9, -1], [1 << 62, 8], [1 << 40, 8]])
def test_bad_group_list(counts):
    x = torch.randn(8, 64, device="cuda").to(torch.bfloat16)
    w = torch.randn(2, 32, 64, device="cuda").to(torch.bfloat16)
    y = torch.full((8, 32), 5.0, device="cuda", dtype=torch.bfloat16)
    ws = W.workspace(256)
    W.w8a8_bf16_grouped_matmul(x, torch.tensor(counts, dtype=torch.int64, device="cuda"), w, ws=ws, y=y)
    assert W.read_device_status(ws) == 5 and bool((y == 5.0).all())
    W.w8a8_bf16_grouped_matmul(x, torch.tensor([3, 5], dtype=torch.int64, device="cuda"), w, ws=ws, y=y)
    assert W.read_device_status(ws) == 0 and not bool((y == 5.0).all())
