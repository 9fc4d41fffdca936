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


def test_fp32_long_sums():
    """A sum of 32768 positive products as fp32: an accumulator takes 768 of K at most, 48 additions of at most 2^-23 of
    the partial sum, 16 more for the alignment inside each; the chunks' sums add one rounding each.  (In one accumulator
    2048 additions lose 2^-24 of the partial sum on average: 1e-4.)"""
    K = 32768
    for M in (5, 300):
        x = (torch.rand(M, K, generator=gen(1), device="cuda") + 0.5).to(torch.bfloat16)
        w = (torch.rand(40, K, generator=gen(2), device="cuda") + 0.5).to(torch.bfloat16)
        v = x.double() @ w.double().t()
        y = W.w8a8_bf16_matmul(x, w, out_dtype=torch.float32)
        assert bool(((y.double() - v).abs() <= (64 * 2.0 ** -23 + K / 512 * 2.0 ** -24) * v).all())


@pytest.mark.parametrize("M,N,K,act", [(5, 512, 2048, "none"), (300, 512, 256, "silu"), (64, 130, 1024, "none"),
                                       (40, 77, 512, "swiglu"), (200, 264, 64, "swiglu"),
                                       (64, 20480, 2048, "none"), (33, 10200, 4096, "swiglu")])
def test_residual_in_place(M, N, K, act):
    x, w, b, r = inputs(M, N, K, act, True, True, M + N)
    want = W.w8a8_bf16_matmul(x, w, b, act, r)
    stream = r.clone()
    got = W.w8a8_bf16_matmul(x, w, b, act, stream, y=stream)
    assert got is stream and torch.equal(got, want)


def test_empty_and_given_outputs():
    x, w, b, _ = inputs(6, 40, 64, "none", True, False, 3)
    assert W.w8a8_bf16_matmul(x[:0], w, b).shape == (0, 40)
    pad = torch.full((9, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    y = W.w8a8_bf16_matmul(x, w, b, y=pad[:6])
    assert torch.equal(y, W.w8a8_bf16_matmul(x, w, b)) and bool((pad[6:] == 7.0).all())
    gl = torch.tensor([0, 4, 0, 2], dtype=torch.int64, device="cuda")
    w4 = w.expand(4, 40, 64).contiguous()
    pad = torch.full((9, 40), 7.0, device="cuda")
    y = W.w8a8_bf16_grouped_matmul(x, gl, w4, y=pad[:6])  # y's own type decides
    assert y.dtype is torch.float32 and bool((pad[6:] == 7.0).all())
    close(y, *reference(x, w, None, "none", None))
    zero = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert W.w8a8_bf16_grouped_matmul(x[:0], zero, w4).shape == (0, 40)


def test_unaligned_outputs():
    """y and the residual on 2-byte boundaries, and a bias that starts on one."""
    x, w, b, r = inputs(70, 64, 128, "none", True, True, 9)
    buf = torch.empty(3 * 70 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    y, res = buf[1:1 + 70 * 64].view(70, 64), buf[70 * 64 + 3:70 * 64 * 2 + 3].view(70, 64)
    bias = buf[-63 - 2:-1]
    res.copy_(r)
    bias.copy_(b)
    assert torch.equal(W.w8a8_bf16_matmul(x, w, bias, "gelu", res, y=y), W.w8a8_bf16_matmul(x, w, b, "gelu", r))


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_nan_stays_where_it_is(act):
    M, N, K = 40, 96, 256
    x, w, _, _ = inputs(M, N, K, act, False, False, 4)
    want = W.w8a8_bf16_matmul(x, w, activation=act)
    x2, w2 = x.clone(), w.clone()
    x2[7, 3], x2[21, 200], w2[50, 9] = float("nan"), float("inf"), float("nan")
    y = W.w8a8_bf16_matmul(x2, w2, activation=act)
    keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
    keep[[7, 21]], keep[:, 50] = False, False
    assert torch.equal(y[keep], want[keep])
    assert bool(y[7].isnan().all()) and bool(y[:, 50].isnan().all()) and not bool(y[21].isfinite().any())
    # rows of another group, read with a tile and not part of it
    counts = [3, 20, 17]
    gl = torch.tensor(counts, dtype=torch.int64, device="cuda")
    w3 = torch.stack([w, w * float("nan"), w])
    x3 = x.clone()
    x3[3:23] = float("inf")
    y = W.w8a8_bf16_grouped_matmul(x3, gl, w3, activation=act)
    assert torch.equal(y[:3], want[:3]) and torch.equal(y[23:], want[23:]) and bool(y[3:23].isnan().all())


def test_calls_that_follow_one_another():
    """A call's output as the next one's weight, rows, residual and bias, with nothing between the launches."""
    M, K = 64, 512
    x, w, _, _ = inputs(M, K, K, "none", False, False, 12)

    def chain(wait):
        h, out = x, []
        for i in range(6):
            h = W.w8a8_bf16_matmul(h, w, activation="silu" if i % 2 else "none", residual=h, ws=ws)
            wait()
            s = W.w8a8_bf16_matmul(h, h, ws=ws, out_dtype=torch.float32)  # [M,M]: the rows are the weight as well
            wait()
            q, sc, r, y = W.w8a8_fp8_rms_norm_quant(h, w[0], residual=x, want_y=True)
            wait()
            h = W.w8a8_bf16_matmul(y, w, bias=r[0], ws=ws)
            wait()
            out += [h, s, q, sc, r, y]
        return out

    ws = W.workspace(W.bf16_matmul_workspace_bytes(M, K, K))
    want = chain(torch.cuda.synchronize)
    for _ in range(20):
        for a, b in zip(chain(lambda: None), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert W.read_device_status(ws) == 0


def test_graphs_streams_and_repeats():
    """Two captured graphs on one workspace, replayed in turn; another stream; the same bits every time."""
    x, w, b, r = inputs(64, 2048, 2048, "none", True, True, 5)
    x2, w2, _, _ = inputs(300, 256, 512, "swiglu", False, False, 6)
    ws = W.workspace(256)
    y, y2 = torch.empty_like(r), torch.empty(300, 256, dtype=torch.bfloat16, device="cuda")
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        W.w8a8_bf16_matmul(x, w, b, "gelu", r, ws=ws, y=y)
    with torch.cuda.graph(graphs[1]):
        W.w8a8_bf16_matmul(x2, w2, activation="swiglu", ws=ws, y=y2)
    for k in range(3):
        x.mul_(1.5)
        x2.mul_(0.5)
        for g in graphs:
            g.replay()
        assert torch.equal(y, W.w8a8_bf16_matmul(x, w, b, "gelu", r))
        assert torch.equal(y2, W.w8a8_bf16_matmul(x2, w2, activation="swiglu"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = W.w8a8_bf16_matmul(x, w, b, "gelu", r)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, y)
    # two streams at once, each with its own workspace
    ws2 = W.workspace(256)
    with torch.cuda.stream(side):
        a = [W.w8a8_bf16_matmul(x, w, b, "gelu", r, ws=ws2) for _ in range(30)]
    c = [W.w8a8_bf16_matmul(x2, w2, activation="swiglu", ws=ws) for _ in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, y) for t in a) and all(torch.equal(t, y2) for t in c)


@pytest.mark.parametrize("rows,weight,out", [(270000, 16, torch.bfloat16), (3, 280000, torch.float32)])
def test_offsets_past_32_bits(rows, weight, out):
    """x, or w, of more than 2^31 values."""
    K = 8192
    x = torch.randn(min(rows, 1000), K, generator=gen(1), device="cuda").to(torch.bfloat16)
    w = (torch.randn(min(weight, 1000), K, generator=gen(2), device="cuda") * 0.02).to(torch.bfloat16)
    x, w = x.repeat(-(-rows // 1000), 1)[:rows], w.repeat(-(-weight // 1000), 1)[:weight]
    y = W.w8a8_bf16_matmul(x, w, out_dtype=out)
    r, c = min(rows, 700), min(weight, 700)
    close(y[-r:, -c:], *reference(x[-r:], w[-c:], None, "none", None))
    close(y[:r, :c], *reference(x[:r], w[:c], None, "none", None))


def test_output_past_32_bits():
    M, N, K = 70000, 32768, 16
    x, w, b, _ = inputs(M, N, K, "none", True, False, 1)
    y = W.w8a8_bf16_matmul(x, w, b, "relu")
    close(y[-300:], *reference(x[-300:], w, b, "relu", None))
    close(y[:300], *reference(x[:300], w, b, "relu", None))


@pytest.mark.parametrize("R", [9, 700, 40000])
def test_a_thousand_experts(R):
    E, N, K = 1024, 40, 64
    pick = torch.randint(0, E, (R,), generator=gen(R), device="cuda").sort().values
    gl = torch.bincount(pick, minlength=E)
    x = torch.randn(R, K, generator=gen(1), device="cuda").to(torch.bfloat16)
    w = torch.randn(E, 2 * N, K, generator=gen(2), device="cuda").to(torch.bfloat16)
    y = W.w8a8_bf16_grouped_matmul(x, gl, w, activation="swiglu", out_dtype=torch.float32)
    v = torch.bmm(w.double()[pick[:2000]], x.double()[:2000, :, None])[:, :, 0]
    a = torch.bmm(w.double().abs()[pick[:2000]], x.double().abs()[:2000, :, None])[:, :, 0]
    g, u, eg, eu = v[:, :N], v[:, N:], a[:, :N] * 22 * 2.0 ** -23, a[:, N:] * 22 * 2.0 ** -23
    s = g * torch.sigmoid(g)
    err = 1.13 * eg * (u.abs() + eu) + (s.abs() + 1.13 * eg) * eu + 300 * 2.0 ** -23 * (s * u).abs()
    close(y[:2000], s * u, err)


def test_refusals():
    x, w, b, r = inputs(8, 32, 64, "none", True, True, 2)
    for bad in (dict(x=x.float()), dict(w=w.half()), dict(bias=b.float()), dict(residual=r.float()),
                dict(out_dtype=torch.float16), dict(y=r.half()), dict(ws=torch.zeros(256, device="cuda"))):
        with pytest.raises(TypeError):
            W.w8a8_bf16_matmul(**{"x": x, "w": w, **bad})
    for bad in (dict(x=x[:, :48]), dict(w=w[:, ::2]), dict(bias=b[:-1]), dict(residual=r[:7]), dict(y=r[:7]),
                dict(x=x.cpu()), dict(w=w.cpu()), dict(bias=b.cpu()), dict(activation="tanh"), dict(activation=None),
                dict(w=w[:-1], activation="swiglu"), dict(w=w, activation="swiglu", bias=b[:16]), dict(x=x.t())):
        with pytest.raises(ValueError):
            W.w8a8_bf16_matmul(**{"x": x, "w": w, **bad})
    with pytest.raises(W.W8A8Error):
        W.w8a8_bf16_matmul(x, w, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(W.W8A8Error):
        W.w8a8_bf16_matmul(x[:, :40].contiguous(), w[:, :40].contiguous())
    gl = torch.tensor([3, 5], dtype=torch.int64, device="cuda")
    w2 = torch.stack([w, w])
    for bad in (dict(group_list=gl[:1]), dict(w=w), dict(bias=b), dict(group_list=gl.cpu()), dict(x=x.t())):
        with pytest.raises(ValueError):
            W.w8a8_bf16_grouped_matmul(**{"x": x, "group_list": gl, "w": w2, **bad})
    with pytest.raises(TypeError):
        W.w8a8_bf16_grouped_matmul(x, gl.int(), w2)
    assert W.last_engine() == W.ENGINE_TC
    assert _capi.ACTIVATIONS["swiglu"] == 5


# more tiles than CTA pairs by a little: the last ones' K is cut over all pairs and joined through the workspace
CUT = [(16, 20000, 1024, "none"), (40, 20800, 4096, "none"), (64, 20480, 2048, "gelu"), (33, 10200, 4096, "swiglu"),
       (2483, 2048, 7168, "none"), (1241, 2000, 8192, "swiglu"), (64, 40000, 2048, "silu")]


@pytest.mark.parametrize("M,N,K,act", CUT)
def test_cut_tiles(M, N, K, act):
    x, w, b, r = inputs(M, N, K, act, True, True, M + N)
    need = W.bf16_matmul_workspace_bytes(M, N, K)
    assert need > 256, "not a case of this test"
    ws = W.workspace(need)
    bf16 = W.w8a8_bf16_matmul(x, w, b, act, r, ws=ws)
    fp32 = W.w8a8_bf16_matmul(x, w, b, act, None, torch.float32, ws=ws)
    close(bf16, *reference(x, w, b, act, r))
    close(fp32, *reference(x, w, b, act, None))
    assert W.read_device_status(ws) == 0
    # the same bits every time, whichever part comes last, and from a graph; the workspace is as it was
    y = torch.empty_like(bf16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.w8a8_bf16_matmul(x, w, b, act, r, ws=ws, y=y)
    for _ in range(20):
        graph.replay()
        assert torch.equal(y, bf16)
        assert torch.equal(W.w8a8_bf16_matmul(x, w, b, act, None, torch.float32, ws=ws), fp32)
    assert not bool(ws[:256 + 4864].any())
    with pytest.raises(W.W8A8Error):  # (need is the larger of the gated and the plain product's)
        W.w8a8_bf16_matmul(x, w, b, act, r, ws=W.workspace(256))
    # one workspace for products of other sizes in turn
    x2, w2, _, _ = inputs(50, 300, 1024, "none", False, False, 1)
    a = W.w8a8_bf16_matmul(x2, w2, ws=ws)
    assert torch.equal(W.w8a8_bf16_matmul(x, w, b, act, r, ws=ws), bf16)
    assert torch.equal(W.w8a8_bf16_matmul(x2, w2, ws=ws), a)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activation_of_every_value(act):
    """Every bf16 value through an activation, in binary32; the bound of the head, and what exp loses below 2^-126."""
    every = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    every = torch.where(every.float().abs() >= 2.0 ** -100, every, torch.zeros_like(every))  # (normal products)
    every = every[every.isfinite()]
    w = torch.zeros(every.numel(), 16, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = every
    x = torch.zeros(3, 16, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    y = W.w8a8_bf16_matmul(x, w, activation=act, out_dtype=torch.float32)
    v = act64(every.double(), act)
    err = (300 * 2.0 ** -23 if act != "relu" else 0.0) * v.abs() + 2.0 ** -119
    assert bool(((y.double() - v).abs() <= err).all()), act
    # infinities and NaN
    w[:3, 0] = torch.tensor([float("inf"), float("nan"), -float("inf")], device="cuda")
    y = W.w8a8_bf16_matmul(x, w[:3].contiguous(), activation=act)
    assert not bool(y[:, :2].isfinite().any()) and bool(y[:, 1].isnan().all())
