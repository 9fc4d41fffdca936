"""Block-scaled FP8 against plain 64-bit implementations: the quantisers, the dense and grouped contractions and
the MoE layer, at the sizes where a block, a tile or a group ends early."""
import numpy as np
import pytest
import torch

import w8a8_dynamic_quant_gb300 as W
from w8a8_dynamic_quant_gb300 import _capi

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def blocks(n):
    return -(-n // 128)


def spread(s, K):
    return s.double().repeat_interleave(128, -1)[..., :K]


def spread_w(s, N, K):
    return s.double().repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]


def quant_reference(v):
    """binary32 [M,K] -> (codes as float8, scales): s = amax / 448 and RN(v / s) as binary32 operations."""
    M, K = v.shape
    p = torch.nn.functional.pad(v, (0, blocks(K) * 128 - K)).view(M, blocks(K), 128)
    a = torch.where(torch.isnan(p), 0.0, p.abs())
    s = a.amax(2) / torch.full((), 448.0, device=v.device)  # by a tensor: a Python number is multiplied by its inverse
    q = torch.where(s[:, :, None] > 0, p / s[:, :, None], p * 0.0 + 0.0)
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(M, -1)[:, :K].contiguous(), s


def same_codes(a, b):
    x, y = a.view(torch.uint8).int(), b.view(torch.uint8).int()
    nan = ((x & 127) == 127) & ((y & 127) == 127)
    return bool(((x == y) | nan).all())


@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (37, 496), (64, 7168), (300, 1360), (2049, 512)])
def test_quant(M, K):
    x = torch.randn(M, K, generator=gen(M + K), device="cuda") * torch.exp2(
        torch.randint(-30, 30, (M, 1), generator=gen(K), device="cuda").float())
    x[0, :16] = 0.0
    if K >= 256:
        x[0, 128:256] = 0.0  # a block of zeros
    x = x.to(torch.bfloat16)
    q, s = W.w8a8_fp8_quant(x)
    rq, rs = quant_reference(x.float())
    assert torch.equal(s, rs)
    assert same_codes(q, rq)


def test_quant_every_mantissa_and_exponent_distance():
    """The quotient's fast path depends only on the mantissas of the value and of the block's maximum and on the
    distance of their exponents: all 128 x 128 x 20 of them."""
    amax = (1 + torch.arange(128, device="cuda") / 128).view(128, 1, 1)
    v = (1 + torch.arange(128, device="cuda") / 128).view(1, 1, 128) * torch.exp2(
        -torch.arange(20, device="cuda").float()).view(1, 20, 1)
    x = v.expand(128, 20, 128).reshape(128, 20, 128).clone()
    x = torch.where(x > amax, amax, x)
    x[:, :, 0] = amax[:, :, 0]  # the maximum in place of one value ...
    y = x.clone()
    y[:, :, 0], y[:, :, 127] = v.expand(128, 20, 128)[:, :, 0].minimum(amax[:, :, 0]), amax[:, :, 0]  # ... or another
    for z in (x, y):
        z = torch.cat([z, -z]).reshape(256, 20 * 128).to(torch.bfloat16)
        q, s = W.w8a8_fp8_quant(z)
        rq, rs = quant_reference(z.float())
        assert torch.equal(s, rs) and same_codes(q, rq)


def test_quant_special_values():
    x = torch.randn(6, 256, generator=gen(1), device="cuda")
    x[0, 5] = float("nan")
    x[1, 7] = float("inf")
    x[2, :128] = float("nan")
    x[3] = 1e-39  # subnormal bf16, subnormal scale
    x[4] = 3.0e38
    x[5, :128] = -0.0
    x = x.to(torch.bfloat16)
    q, s = W.w8a8_fp8_quant(x)
    rq, rs = quant_reference(x.float())
    assert torch.equal(s, rs)
    assert same_codes(q, rq)
    v = q.float()
    assert bool(v[0, 5].isnan()) and int(v[0].isnan().sum()) == 1
    assert bool(v[1, 7].isnan()) and bool((v[1, :7] == 0).all()) and float(s[1, 0]) == float("inf")


def test_quant_empty_and_uint8_out():
    q, s = W.w8a8_fp8_quant(torch.empty(0, 256, device="cuda", dtype=torch.bfloat16))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    x = torch.randn(5, 160, device="cuda").to(torch.bfloat16)
    out = torch.empty(5, 160, dtype=torch.uint8, device="cuda")
    q, _ = W.w8a8_fp8_quant(x, q=out)
    assert q is out and torch.equal(out, W.w8a8_fp8_quant(x)[0].view(torch.uint8))


@pytest.mark.parametrize("R,I", [(1, 16), (2, 128), (33, 336), (129, 1392), (1000, 2048)])
def test_swiglu_quant(R, I):
    y = (torch.randn(R, 2 * I, generator=gen(R + I), device="cuda") * 3).to(torch.bfloat16)
    if I >= 128:
        y[0, :128] = 0.0  # h = 0 in a whole block
    y[-1, 0] = -200.0     # exp overflows: sigmoid 0
    q, s = W.w8a8_fp8_swiglu_quant(y)
    g, u = y[:, :I].double(), y[:, I:].double()
    h = g * torch.sigmoid(g) * u
    p = torch.nn.functional.pad(h, (0, blocks(I) * 128 - I)).view(R, -1, 128)
    rs = p.abs().amax(2) / 448.0
    # exp within 2 + |g| units, the reciprocal within 2, three products: under 32 * 2^-24 for |g| < 16, where h is
    # not small; the scale's own rounding included
    assert bool(((s.double() - rs).abs() <= 32 * 2.0 ** -24 * rs).all())
    # a code is the value within half a step of E4M3 (2^-4 relative, 2^-10 below 2^-6), and the error above
    want = h / spread(torch.where(s > 0, s, 1.0), I)
    err = (q.double() - want).abs()
    assert bool((err <= torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10)) * (1 + 1e-4)).all())


def test_swiglu_quant_far_gates():
    """Blocks whose gates all lie far out: the sigmoid of a negative gate falls through binary32's smallest normal
    value at -87.3 to its smallest at -103, and h with a large up value stays well above either."""
    gates = [-16.0, -20.0, -60.0, -87.0, -87.5, -88.0, -88.5, -89.0, -95.0, 20.0, 60.0, 88.5, 100.0]
    g = torch.tensor(gates, device="cuda").view(-1, 1).expand(-1, 256)
    u = torch.randn(len(gates), 256, generator=gen(7), device="cuda") * 2.0 ** 30
    y = torch.cat([g, u], 1).to(torch.bfloat16)
    q, s = W.w8a8_fp8_swiglu_quant(y)
    g, u = y[:, :256].double(), y[:, 256:].double()
    t = torch.exp(-g.abs())
    h = g * torch.where(g > 0, 1.0, t) / (1 + t) * u
    # relative to h: exp within 2 + 1.173 |g| units of 2^-23 (for a positive gate they count t / (1 + t) < 1 times) and,
    # below the normal values, 2 of 2^-149; the sum, the quotient and the products 4.5, and half of 2^-149 where one of
    # them is below the normal values
    rel = (2 + 1.173 * g.abs() + 4.5) * 2.0 ** -23 + torch.where(g > 0, 0.0, 2.5 * 2.0 ** -149 / t)
    rs = h.view(len(gates), 2, 128).abs().amax(2) / 448.0
    assert bool(((s.double() - rs).abs() <= rs * (rel[:, :1] + 2.0 ** -24)).all()), (s.double() / rs - 1).tolist()
    want = h / spread(s, 256)
    step = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10))  # half a step of E4M3
    assert bool(((q.double() - want).abs() <= step + want.abs() * (rel + 2.0 ** -24)).all())


def bound(q, xs, w, ws, K, ref):
    """One bf16 rounding of the exact value, and the binary32 sums: 128 products and their sum inside a block by
    the tensor core (held to 2^-20 of the magnitude: its adder may cut a few bits below binary32) and one
    fused multiply-add and a scale product a block."""
    mag = (q.double().abs() * spread(xs, K)) @ (w.double().abs() * spread_w(ws, w.shape[0], K)).t()
    return ref.abs() * 2.0 ** -8 + mag * (2.0 ** -20 + (blocks(K) + 2) * 2.0 ** -24)


def problem(seed, M, N, K, E=None):
    g = gen(seed)
    x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp2(
        torch.randint(-3, 4, (M, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    q, xs = quant_reference(x.float())
    n = 1 if E is None else E
    w = (torch.randn(n, N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(n, blocks(N), blocks(K), generator=g, device="cuda") * 1e-2 + 1e-4
    return (q, xs, w[0], ws[0]) if E is None else (q, xs, w, ws)


def check_dense(M, N, K, bias=False, seed=0):
    q, xs, w, ws = problem(seed + M + N + K, M, N, K)
    b = torch.randn(N, generator=gen(9), device="cuda").to(torch.bfloat16) if bias else None
    work = W.workspace(W.fp8_matmul_workspace_bytes(M, N, K))
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    W.w8a8_fp8_matmul(q, xs, w, ws, bias=b, ws=work, y=y)
    ref = (q.double() * spread(xs, K)) @ (w.double() * spread_w(ws, N, K)).t()
    tol = bound(q, xs, w, ws, K, ref)
    if bias:
        ref = ref + b.double()
        tol = tol + ref.abs() * 2.0 ** -8
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), f"excess {float((err - tol).max())} at {(err - tol).argmax().item()}"
    again = W.w8a8_fp8_matmul(q, xs, w, ws, bias=b, ws=work)  # the workspace was left ready
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    assert W.read_device_status(work) == 0


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 129, 257, 500])
@pytest.mark.parametrize("N,K", [(128, 128), (256, 512), (200, 400), (577, 1040), (1, 16), (1416, 2000)])
def test_dense(M, N, K):
    check_dense(M, N, K, bias=(M + N) % 2 == 1)


@pytest.mark.parametrize("M,N,K", [(64, 2048, 7168), (1, 4096, 7168), (8, 129, 16384), (300, 520, 4096),
                                   (2100, 1111, 1040), (400, 1002, 528), (4096, 2048, 512),
                                   (1024, 1024, 65536), (129, 5000, 16400)])
def test_dense_large(M, N, K):
    check_dense(M, N, K, bias=True)


@pytest.mark.parametrize("M,N,K", [(50, 9900, 8192), (2100, 1111, 16384)])
def test_dense_cut_units(M, N, K):
    """Few long units that are no whole number for the pairs: their pieces meet in the workspace."""
    assert W.fp8_matmul_workspace_bytes(M, N, K) > 1 << 20  # room for pieces
    check_dense(M, N, K, bias=True)


def test_dense_empty_nan_and_stream():
    q, xs, w, ws = problem(3, 40, 300, 528)
    assert W.w8a8_fp8_matmul(q[:0], xs[:0], w, ws).shape == (0, 300)
    want = W.w8a8_fp8_matmul(q, xs, w, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = W.w8a8_fp8_matmul(q, xs, w, ws)
    st.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    bad = q.clone()
    bad.view(torch.uint8)[17, 30] = 0x7F  # a NaN code spoils its own row and no other
    y = W.w8a8_fp8_matmul(bad, xs, w, ws)
    assert bool(y[17].isnan().all()) and torch.equal(y[:17].view(torch.int16), want[:17].view(torch.int16))
    assert torch.equal(y[18:].view(torch.int16), want[18:].view(torch.int16))
    as_bytes = W.w8a8_fp8_matmul(q.view(torch.uint8), xs, w.view(torch.uint8), ws)
    assert torch.equal(as_bytes.view(torch.int16), want.view(torch.int16))


def check_grouped(counts, N, K, seed=0):
    E, R = len(counts), sum(counts)
    q, xs, w, ws = problem(seed + R + N + K, R, N, K, E)
    gl = torch.tensor(counts, dtype=torch.int64, device="cuda")
    work = W.workspace(W.fp8_grouped_matmul_workspace_bytes(E, R, N, K))
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    W.w8a8_fp8_grouped_matmul(q, xs, gl, w, ws, ws=work, y=y)
    r = 0
    for e, n in enumerate(counts):
        if n:
            ref = (q[r:r + n].double() * spread(xs[r:r + n], K)) @ (w[e].double() * spread_w(ws[e], N, K)).t()
            err = (y[r:r + n].double() - ref).abs()
            tol = bound(q[r:r + n], xs[r:r + n], w[e], ws[e], K, ref)
            assert bool((err <= tol).all()), f"expert {e}: excess {float((err - tol).max())}"
        r += n
    again = W.w8a8_fp8_grouped_matmul(q, xs, gl, w, ws, ws=work)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    assert W.read_device_status(work) == 0


@pytest.mark.parametrize("counts", [[1], [0, 5, 0], [3, 0, 17, 1, 64], [130, 1, 0, 257, 40, 2], [0, 0, 0, 600],
                                    [1] * 33, [0] * 40 + [9] + [0] * 23])
@pytest.mark.parametrize("N,K", [(128, 256), (200, 400), (577, 1040)])
def test_grouped(counts, N, K):
    check_grouped(counts, N, K)


@pytest.mark.parametrize("counts", [[3, 0, 17, 1, 64], [130, 1, 0, 257, 40, 2], [2, 1]])
def test_grouped_cut_units(counts):
    check_grouped(counts, 577, 16384)


def test_grouped_large():
    rng = np.random.default_rng(0)
    check_grouped(rng.multinomial(4096, rng.dirichlet(np.full(16, 0.5))).tolist(), 1024, 2048)
    check_grouped(rng.multinomial(300, np.full(96, 1 / 96)).tolist(), 768, 1536)


def test_grouped_bad_list_writes_nothing():
    q, xs, w, ws = problem(1, 32, 256, 256, 4)
    work = W.workspace(W.fp8_grouped_matmul_workspace_bytes(4, 32, 256, 256))
    for counts in ([8, 8, 8, 9], [40, -8, 0, 0], [8, 8, 8, 0], [33, 0, 0, 0], [2 ** 40, 0, 0, 0]):
        y = torch.full((32, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        W.w8a8_fp8_grouped_matmul(q, xs, torch.tensor(counts, device="cuda"), w, ws, ws=work, y=y)
        assert W.read_device_status(work) == 5
        assert bool((y == 5.0).all())


def layer_reference(x, ids, wts, w13, s13, w2, s2):
    """The layer step by step on the host's side of the formulas, in 64 bits but for the roundings it names."""
    T, H = x.shape
    I = w2.shape[2]
    q, s = quant_reference(x.float())
    xd = q.double() * spread(s, H)
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            gu = (xd[t] @ (w13[e].double() * spread_w(s13[e], 2 * I, H)).t()).to(torch.bfloat16)
            g, u = gu[:I].double(), gu[I:].double()
            h = (g * torch.sigmoid(g) * u).float().view(1, I)
            hq, hs = quant_reference(h)
            d = hq.double() * spread(hs, I)
            o = (d[0] @ (w2[e].double() * spread_w(s2[e], H, I)).t()).to(torch.bfloat16)
            y[t] += float(wts[t, j]) * o.double()
    return y


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 128, 128), (9, 8, 3, 272, 144), (40, 16, 4, 512, 256)])
def test_layer(T, E, k, H, I):
    g = gen(T + H)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids, wts = W.moe_gate_topk(torch.randn(T, E, generator=g, device="cuda"), k, scoring="sigmoid")
    w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    w2 = (torch.randn(E, H, I, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    s13 = torch.rand(E, blocks(2 * I), blocks(H), generator=g, device="cuda") * 1e-3 + 1e-4
    s2 = torch.rand(E, blocks(H), blocks(I), generator=g, device="cuda") * 1e-3 + 1e-4
    work = W.workspace(W.moe_fp8_layer_workspace_bytes(T, k, H, I, E))
    y = W.moe_fp8_layer(x, ids, wts, w13, s13, w2, s2, ws=work)
    assert W.read_device_status(work) == 0
    ref = layer_reference(x, ids, wts, w13, s13, w2, s2)
    # bf16 roundings of the W13 output (2^-9) may move a code of h by a step (2^-3 of it) where it sits near a
    # boundary: a few codes in a thousand, so the norm of the difference stays below 2 %; bf16 of y adds 2^-9
    assert float((y.double() - ref).norm() / ref.norm()) < 0.02
    again = W.moe_fp8_layer(x, ids, wts, w13, s13, w2, s2, ws=work)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))


def test_layer_matches_its_parts():
    """The layer's result is that of its parts called one by one, bit for bit."""
    T, E, k, H, I = 77, 12, 3, 384, 208
    g = gen(4)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids, wts = W.moe_gate_topk(torch.randn(T, E, generator=g, device="cuda"), k)
    w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    w2 = (torch.randn(E, H, I, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    s13 = torch.rand(E, blocks(2 * I), blocks(H), generator=g, device="cuda") * 1e-3
    s2 = torch.rand(E, blocks(H), blocks(I), generator=g, device="cuda") * 1e-3
    y = W.moe_fp8_layer(x, ids, wts, w13, s13, w2, s2)
    _, _, gl, pos = W.moe_permute_quant(x, None, ids, E)
    q, s = W.w8a8_fp8_quant(x)
    src = torch.empty(T * k, dtype=torch.int64, device="cuda")
    src[pos.view(-1).long()] = torch.arange(T, device="cuda").repeat_interleave(k)
    xq = q.view(torch.uint8)[src].contiguous()
    y13 = W.w8a8_fp8_grouped_matmul(xq, s[src].contiguous(), gl, w13, s13)
    hq, hs = W.w8a8_fp8_swiglu_quant(y13)
    yr = W.w8a8_fp8_grouped_matmul(hq, hs, gl, w2, s2)
    assert torch.equal(y.view(torch.int16), W.moe_unpermute_combine(yr, pos, wts).view(torch.int16))


@pytest.mark.parametrize("T,E,k,H,I", [(600, 4, 2, 16384, 384), (900, 3, 2, 1040, 528)])
def test_layer_of_many_rows(T, E, k, H, I):
    """Mean rows of an expert above 64: both contractions on tiles of 256 tokens, W13's units cut where K is long."""
    g = gen(T + H)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[:, 0] += 1.0  # uneven groups
    ids, wts = W.moe_gate_topk(logits, k, scoring="sigmoid")
    w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    w2 = (torch.randn(E, H, I, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
    s13 = torch.rand(E, blocks(2 * I), blocks(H), generator=g, device="cuda") * 1e-4 + 1e-5
    s2 = torch.rand(E, blocks(H), blocks(I), generator=g, device="cuda") * 1e-3 + 1e-4
    work = W.workspace(W.moe_fp8_layer_workspace_bytes(T, k, H, I, E))
    y = W.moe_fp8_layer(x, ids, wts, w13, s13, w2, s2, ws=work)
    assert W.read_device_status(work) == 0
    rows = torch.arange(0, T, 37, device="cuda")
    ref = layer_reference(x[rows], ids[rows], wts[rows], w13, s13, w2, s2)
    assert float((y[rows].double() - ref).norm() / ref.norm()) < 0.02  # as in test_layer
    again = W.moe_fp8_layer(x, ids, wts, w13, s13, w2, s2, ws=work)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))


def quantise_blocks(v):
    """[E,N,K] binary32 -> (E4M3 [E,N,K], scale per 128 x 128 block)."""
    E, N, K = v.shape
    p = torch.nn.functional.pad(v, (0, blocks(K) * 128 - K, 0, blocks(N) * 128 - N)).view(
        E, blocks(N), 128, blocks(K), 128)
    s = p.abs().amax((2, 4)) / 448.0
    q = (p / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(E, blocks(N) * 128, -1)
    return q[:, :N, :K].contiguous(), s


@pytest.mark.parametrize("T,E,k,H,I", [(40, 6, 3, 272, 208), (9, 4, 2, 128, 144), (21, 5, 2, 256, 16),
                                       (33, 4, 2, 256, 256)])
def test_layer_from_separately_scaled_halves(T, E, k, H, I):
    """Gate and up matrices quantised on their own, as checkpoints store them: each half has its own blocks."""
    g = gen(T + I)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids, wts = W.moe_gate_topk(torch.randn(T, E, generator=g, device="cuda"), k, scoring="sigmoid")
    # channels of very different size, so that a neighbouring block's scale is a wrong one
    size = torch.exp2(torch.randint(-4, 5, (E, 2 * I, 1), generator=g, device="cuda").float())
    w = torch.randn(E, 2 * I, H, generator=g, device="cuda") * size
    (qg, sg), (qu, su) = quantise_blocks(w[:, :I]), quantise_blocks(w[:, I:])
    q2, s2 = quantise_blocks(torch.randn(E, H, I, generator=g, device="cuda"))
    q13, s13 = torch.cat([qg, qu], 1), torch.stack([sg, su], 1)
    w13, w13_scale, w2 = W.moe_fp8_pad_inner(q13, s13, q2)
    y = W.moe_fp8_layer(x, ids, wts, w13, w13_scale, w2, s2)
    if I % 128 == 0:
        assert w13 is q13 and w2 is q2
    else:
        with pytest.raises(ValueError, match="moe_fp8_pad_inner"):
            W.moe_fp8_layer(x, ids, wts, q13, s13, q2, s2)
    _, _, gl, pos = W.moe_permute_quant(x, None, ids, E)
    q, s = W.w8a8_fp8_quant(x)
    src = torch.empty(T * k, dtype=torch.int64, device="cuda")
    src[pos.view(-1).long()] = torch.arange(T, device="cuda").repeat_interleave(k)
    xq, xs = q.view(torch.uint8)[src].contiguous(), s[src].contiguous()
    y13 = torch.cat([W.w8a8_fp8_grouped_matmul(xq, xs, gl, qg, sg), W.w8a8_fp8_grouped_matmul(xq, xs, gl, qu, su)], 1)
    hq, hs = W.w8a8_fp8_swiglu_quant(y13)
    yr = W.w8a8_fp8_grouped_matmul(hq, hs, gl, q2, s2)
    want = W.moe_unpermute_combine(yr, pos, wts)
    # K is short, so no unit's K is cut in either: the same sums in the same order
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    xd = q.double() * spread(s, H)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            gate = (xd[t] @ (qg[e].double() * spread_w(sg[e], I, H)).t()).to(torch.bfloat16).double()
            up = (xd[t] @ (qu[e].double() * spread_w(su[e], I, H)).t()).to(torch.bfloat16).double()
            d, ds = quant_reference((gate * torch.sigmoid(gate) * up).float().view(1, I))
            o = (d.double() * spread(ds, I))[0] @ (q2[e].double() * spread_w(s2[e], H, I)).t()
            ref[t] += float(wts[t, j]) * o.to(torch.bfloat16).double()
    assert float((y.double() - ref).norm() / ref.norm()) < 0.02  # as in test_layer


def test_layer_bad_ids_set_the_status():
    T, E, k, H, I = 5, 4, 2, 128, 128
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int64, device="cuda")
    ids[3, 1] = E
    w13 = torch.zeros(E, 2 * I, H, device="cuda").to(torch.float8_e4m3fn)
    w2 = torch.zeros(E, H, I, device="cuda").to(torch.float8_e4m3fn)
    one = lambda n, m: torch.ones(E, blocks(n), blocks(m), device="cuda")  # noqa: E731
    work = W.workspace(W.moe_fp8_layer_workspace_bytes(T, k, H, I, E))
    W.moe_fp8_layer(x, ids, torch.ones(T, k, device="cuda"), w13, one(2 * I, H), w2, one(H, I), ws=work)
    assert W.read_device_status(work) == 10


def test_refusals():
    q, xs, w, ws = problem(0, 4, 256, 256)
    with pytest.raises(TypeError):
        W.w8a8_fp8_matmul(q.float(), xs, w, ws)
    with pytest.raises(ValueError):
        W.w8a8_fp8_matmul(q, xs[:, :1].contiguous(), w, ws)
    with pytest.raises(ValueError):
        W.w8a8_fp8_matmul(q, xs, w, ws.t()[:1])
    with pytest.raises(ValueError):
        W.w8a8_fp8_matmul(q.t(), xs, w, ws)
    with pytest.raises(W.W8A8Error):
        W.w8a8_fp8_quant(torch.zeros(2, 24, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(W.W8A8Error):
        W.w8a8_fp8_matmul(q, xs, w, ws, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros(4 * 256 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 256)  # 8 bytes off a 16-byte line
    with pytest.raises(W.W8A8Error):
        W.w8a8_fp8_matmul(odd, xs, w, ws)
    with pytest.raises(ValueError):
        W.w8a8_fp8_swiglu_quant(torch.zeros(2, 33, dtype=torch.bfloat16, device="cuda"))
    assert _capi.STATUS[3] == "W8A8_ERR_ALIGN"


def test_quant_offsets_past_32_bits():
    M, K = 300_000, 8192  # 2.4 G values
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, generator=gen(2), device="cuda").to(torch.bfloat16)
    q, s = W.w8a8_fp8_quant(x)
    rq, rs = quant_reference(x[-4:].float())
    assert torch.equal(s[-4:], rs) and same_codes(q[-4:], rq)
    assert int(q[:-3].view(torch.uint8).amax()) == 0 and float(s[:-3].amax()) == 0.0


def test_dense_offsets_past_32_bits():
    M, N, K = 66_000, 65_792, 128  # 4.3 G outputs
    q, xs, w, ws = problem(5, M, N, K)
    y = W.w8a8_fp8_matmul(q, xs, w, ws)
    rows = torch.tensor([0, 255, 256, 32_767, 65_279, 65_999], device="cuda")
    ref = (q[rows].double() * spread(xs[rows], K)) @ (w.double() * spread_w(ws, N, K)).t()
    err = (y[rows].double() - ref).abs()
    assert bool((err <= bound(q[rows], xs[rows], w, ws, K, ref)).all())


def test_dense_most_rows():
    """The largest number of rows there may be: their last block of 256 ends at 2^31."""
    M, N, K = 2 ** 31 - 1, 1, 16
    w = torch.ones(N, K, device="cuda").to(torch.float8_e4m3fn)
    ws = torch.ones(1, 1, device="cuda")
    q = torch.zeros(M, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    xs = torch.zeros(M, 1, device="cuda")
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 255, 256, M // 2, M - 256, M - 255, M - 2, M - 1], device="cuda")
    q.view(torch.uint8)[rows] = 0x38  # 1.0
    xs[rows, 0] = torch.arange(1, 9, device="cuda").float()
    W.w8a8_fp8_matmul(q, xs, w, ws, y=y)
    assert y[rows, 0].tolist() == [16.0 * (i + 1) for i in range(8)]  # 16 products of ones, times the row's scale
    y[rows] = 0
    assert not bool(y.any())


def test_one_workspace_for_calls_of_every_kind():
    """Calls with few and many tokens, whole and cut units, clusters, groups, and the layer, in turn on one workspace
    that was zeroed once: each gives the bits that it gives on a workspace of its own."""
    calls, need = [], 0

    def dense(M, N, K):
        q, xs, w, ws = problem(M + N + K, M, N, K)
        return W.fp8_matmul_workspace_bytes(M, N, K), lambda work: W.w8a8_fp8_matmul(q, xs, w, ws, ws=work)

    def grouped(counts, N, K):
        E, R = len(counts), sum(counts)
        q, xs, w, ws = problem(R + N + K, R, N, K, E)
        gl = torch.tensor(counts, dtype=torch.int64, device="cuda")
        return (W.fp8_grouped_matmul_workspace_bytes(E, R, N, K),
                lambda work: W.w8a8_fp8_grouped_matmul(q, xs, gl, w, ws, ws=work))

    def layer(T, E, k, H, I):
        g = gen(T + H)
        x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        ids, wts = W.moe_gate_topk(torch.randn(T, E, generator=g, device="cuda"), k)
        w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
        w2 = (torch.randn(E, H, I, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
        s13 = torch.rand(E, blocks(2 * I), blocks(H), generator=g, device="cuda") * 1e-4
        s2 = torch.rand(E, blocks(H), blocks(I), generator=g, device="cuda") * 1e-4
        return (W.moe_fp8_layer_workspace_bytes(T, k, H, I, E),
                lambda work: W.moe_fp8_layer(x, ids, wts, w13, s13, w2, s2, ws=work))

    for nbytes, call in (dense(64, 2048, 7168), dense(50, 9900, 8192), dense(16, 256, 512), dense(2100, 1111, 16384),
                         dense(700, 2000, 1536), grouped([3, 0, 17, 1, 64], 577, 16384), grouped([1] * 33, 200, 400),
                         grouped([130, 1, 0, 257, 40, 2], 577, 16384), layer(9, 8, 3, 272, 144),
                         layer(600, 4, 2, 16384, 384)):
        fresh = W.workspace(nbytes)
        calls.append((call, call(fresh).view(torch.int16)))
        assert W.read_device_status(fresh) == 0
        need = max(need, nbytes)
    shared = W.workspace(need)
    for step in (1, 3, 7):  # three orders, in which every call follows different ones
        for i in range(len(calls)):
            call, want = calls[i * step % len(calls)]
            assert torch.equal(call(shared).view(torch.int16), want)
    assert W.read_device_status(shared) == 0


@pytest.mark.parametrize("M,N,K", [(48, 1100, 4096), (300, 1100, 4096), (700, 2000, 1536)])
def test_matmul_in_a_graph(M, N, K):
    """Captured and replayed on changed inputs: nothing of a call is left on the host, the workspace stays ready."""
    q, xs, w, ws = problem(8, M, N, K)
    work = W.workspace(W.fp8_matmul_workspace_bytes(M, N, K))
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    W.w8a8_fp8_matmul(q, xs, w, ws, ws=work, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            W.w8a8_fp8_matmul(q, xs, w, ws, ws=work, y=y)
    q2, xs2, _, _ = problem(9, M, N, K)
    q.copy_(q2)
    xs.copy_(xs2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), W.w8a8_fp8_matmul(q, xs, w, ws).view(torch.int16))
    assert W.read_device_status(work) == 0
