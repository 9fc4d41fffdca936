"""The norm with 8-bit outputs against its formula: the sum of squares in 64 bits, every step after it one binary32
operation, so that codes, scales and the residual's sum are equal bit for bit."""
import pytest
import torch

import w8a8_dynamic_quant_gb300 as W

pytestmark = pytest.mark.gpu

FORMS = {"int8": W.w8a8_rms_norm_quant, "fp8": W.w8a8_fp8_rms_norm_quant, "mx": W.w8a8_mx_rms_norm_quant}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def full(value):
    return torch.full((), float(value), device="cuda")  # by a tensor: a Python number is multiplied by its inverse


def norm_reference(x, weight, eps, residual):
    """(r, v): the residual's sum in bf16 and the norm in binary32."""
    r = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    total = r.double().square().sum(1, keepdim=True).float()
    g = torch.rsqrt((total / full(x.shape[1]) + torch.tensor(eps, device="cuda")).double()).float()
    return r, r.float() * g * weight.float()


def codes_reference(v, form):
    """The codes as bytes and the scales of binary32 values v [M,K]."""
    M, K = v.shape
    width = {"int8": K, "fp8": 128, "mx": 32}[form]
    p = torch.nn.functional.pad(v, (0, -K % width)).view(M, -1, width)
    top = torch.where(p.isnan(), 0.0, p.abs()).amax(2)
    if form == "mx":
        e = torch.where(top.isinf(), 120, torch.frexp(top).exponent - 9).clamp(-127, 127)
        q = (p.double() * torch.exp2(-e.double())[:, :, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        s = torch.where(p.isnan().any(2), 255, torch.where(top > 0, e + 127, 0)).to(torch.uint8)
        return q.view(torch.uint8).view(M, K), s
    s = top / full(127.0 if form == "int8" else 448.0)
    d = torch.where(s[:, :, None] > 0, p / s[:, :, None], p * 0.0 + 0.0)
    if form == "int8":
        return d.nan_to_num(0.0).round().clamp(-127, 127).to(torch.int8).view(M, K), s[:, 0]
    return d.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(M, -1)[:, :K], s


def same_codes(a, b, form):
    if form == "int8":
        return torch.equal(a, b)
    x, y = a.view(torch.uint8).int(), b.int()
    nan = ((x & 127) == 127) & ((y & 127) == 127)
    return bool(((x == y) | nan).all())


def check(form, x, weight, eps=1e-6, residual=None, want_y=False):
    q, s, r, y = FORMS[form](x, weight, eps, residual=residual, want_y=want_y)
    rr, v = norm_reference(x, weight, eps, residual)
    rq, rs = codes_reference(v, form)
    assert torch.equal(s, rs), "scales"
    assert same_codes(q, rq, form), "codes"
    assert (r is None) if residual is None else torch.equal(r.view(torch.int16), rr.view(torch.int16))
    if want_y:
        want = v.to(torch.bfloat16)
        assert bool(((y == want) | (y.isnan() & want.isnan())).all())
    else:
        assert y is None


# groups of 1 to 32 warps with one chunk a thread, above 8192 values four and eight; rows that end inside a group of each
# (four chunks of shorter rows take more of them: test_gpu_norm_arms.py)
SIZES = [(1, 32), (3, 160), (5, 256), (7, 288), (9, 512), (130, 1024), (33, 1504), (400, 2016), (5, 2080), (400, 4096),
         (700, 2176), (310, 7168), (64, 7168), (400, 8192), (3, 8224), (11, 16384), (2, 17408), (3, 32768), (2, 65536)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("form", list(FORMS))
def test_sizes(form, M, K):
    g = gen(M * 7 + K)
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, ::97] *= 30.0
    size = torch.exp2(torch.randint(-20, 20, (M, 1), generator=g, device="cuda").float())
    res = (torch.randn(M, K, generator=g, device="cuda") * size).to(torch.bfloat16)
    w = 1.0 + 0.3 * torch.randn(K, generator=g, device="cuda")
    check(form, x.to(torch.bfloat16), w, residual=res, want_y=True)
    check(form, x.to(torch.bfloat16), w.to(torch.bfloat16))


@pytest.mark.parametrize("form", ["int8", "fp8"])
@pytest.mark.parametrize("M,K", [(1, 16), (4, 48), (19, 144), (300, 2064), (5, 7184)])
def test_sixteen_values_over(form, M, K):
    g = gen(K)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    check(form, x, torch.rand(K, generator=g, device="cuda") + 0.5, residual=x.flip(0).contiguous(), want_y=True)


@pytest.mark.parametrize("form", list(FORMS))
def test_special_rows(form):
    """Zeros, values whose squares overflow or vanish, NaN and infinities, a weight of zeros and one with a NaN."""
    K = 1024
    x = torch.randn(12, K, generator=gen(3), device="cuda")
    x[0] = 0.0
    x[1] = -0.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4, :9] = -float("inf")
    x[5] *= 1e30          # S is infinite: g = 0
    x[6] *= 1e18          # S near the top of binary32
    x[7] *= 1e-30         # squares below binary32: eps alone
    x[8] *= 1e-19
    x[9] = float("nan")
    x[10, 128:] = 0.0     # blocks of zeros
    x[11] = 1.0
    x = x.to(torch.bfloat16)
    w = torch.rand(K, generator=gen(4), device="cuda") + 0.5
    q, s, _, y = FORMS[form](x, w, 1e-6, want_y=True)
    rows = [0, 1, 2, 3, 4, 5, 6, 8, 9, 10, 11]
    _, v = norm_reference(x, w, 1e-6, None)
    rq, rs = codes_reference(v, form)
    assert torch.equal(s[rows], rs[rows]) and same_codes(q[rows], rq[rows], form)
    # row 7: eps decides g, the squares are below 2^-149 and count as nothing
    check(form, x[7:8].contiguous(), w)
    w[5] = float("nan")
    w[300] = 0.0
    check(form, x[6:12].contiguous(), w, want_y=True)
    check(form, x[:3].contiguous(), torch.zeros(K, device="cuda"))
    w[9] = float("inf")
    check(form, x[8:].contiguous(), w)


def test_sum_is_the_rounded_exact_sum():
    """Rows on which a plain binary32 sum goes wrong: many small squares behind a large one, in every place."""
    K = 4096
    x = torch.full((256, K), 2.0 ** -9, device="cuda")
    x[torch.arange(256), torch.arange(256) * 16 + 3] = 8.0
    x[:, 1::2] *= 1.0 + torch.rand(256, K // 2, generator=gen(0), device="cuda")
    x = x.to(torch.bfloat16)
    w = torch.ones(K, device="cuda")
    for form in FORMS:
        check(form, x, w)


def test_int8_ties_and_every_quotient():
    """Values that fall on and beside half steps of the scale: g is a power of two, so v holds the chosen values."""
    K = 256
    rows = []
    for top in (127.0, 126.5, 100.25, 64.0, 90.5):
        v = torch.arange(K, device="cuda").float() * 0.5 - 64.0
        v = v.clamp(-top, top)
        v[0] = top
        rows.append(v)
    x = torch.stack(rows).to(torch.bfloat16)
    check("int8", x, torch.ones(K, device="cuda"))
    w = torch.rand(K, generator=gen(8), device="cuda") * 2.0 ** torch.randint(-12, 12, (K,), generator=gen(9), device="cuda").float()
    for form in FORMS:
        check(form, x, w)
        check(form, x, w * 2.0 ** -60)
        check(form, x, w * 2.0 ** 60)


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -110, 2.0 ** -98, 2.0 ** 100, 2.0 ** 112])
@pytest.mark.parametrize("form", list(FORMS))
def test_far_weights(form, scale):
    """Scales out of the range in which the quotient comes from the reciprocal."""
    x = torch.randn(5, 512, generator=gen(11), device="cuda").to(torch.bfloat16)
    check(form, x, (torch.rand(512, generator=gen(12), device="cuda") + 0.5) * scale)


@pytest.mark.parametrize("form", list(FORMS))
def test_in_place_residual(form):
    x = torch.randn(37, 1536, generator=gen(1), device="cuda").to(torch.bfloat16)
    res = torch.randn(37, 1536, generator=gen(2), device="cuda").to(torch.bfloat16)
    w = torch.ones(1536, dtype=torch.bfloat16, device="cuda")
    want = FORMS[form](x, w, residual=res)
    for into in ("residual", "x"):
        a, b = x.clone(), res.clone()
        out = b if into == "residual" else a
        got = FORMS[form](a, w, residual=b, residual_out=out)
        assert got[2] is out
        for p, q in zip(got[:3], want[:3]):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("form", list(FORMS))
def test_empty_and_given_outputs(form):
    w = torch.ones(256, device="cuda")
    q, s, r, y = FORMS[form](torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), w, want_y=True)
    assert q.shape == (0, 256) and s.shape[0] == 0 and r is None and y.shape == (0, 256)
    x = torch.randn(6, 256, generator=gen(5), device="cuda").to(torch.bfloat16)
    q, s, _, _ = FORMS[form](x, w)
    # rows behind the last one are left as they were
    pad = torch.full((8, 256), 77, dtype=torch.uint8, device="cuda")
    q2 = pad[:6] if form != "int8" else pad.view(torch.int8)[:6]
    y2 = torch.full((8, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    out = FORMS[form](x, w, q=q2, y=y2[:6])
    assert out[0] is q2 and torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
    assert bool((pad[6:] == 77).all()) and bool((y2[6:] == 3.0).all())
    assert torch.equal(y2[:6], norm_reference(x, w, 1e-6, None)[1].to(torch.bfloat16))


def test_refusals():
    x = torch.randn(4, 256, device="cuda").to(torch.bfloat16)
    w = torch.ones(256, device="cuda")
    f = W.w8a8_rms_norm_quant
    for bad in (dict(x=x.float()), dict(weight=w.half()), dict(residual=x.float()), dict(q=torch.empty(4, 256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(TypeError):
            f(**{"x": x, "weight": w, **bad})
    for bad in (dict(weight=w[:-1]), dict(residual=x[:3]), dict(residual_out=x), dict(x=x[:, ::2]), dict(weight=w.cpu()),
                dict(x=x.cpu()), dict(y=x[:2])):
        with pytest.raises(ValueError):
            f(**{"x": x, "weight": w, **bad})
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        with pytest.raises(W.W8A8Error):
            f(x, w, eps)
    with pytest.raises(W.W8A8Error):
        W.w8a8_mx_rms_norm_quant(x[:, :48].contiguous(), w[:48].contiguous())
    with pytest.raises(W.W8A8Error):
        f(torch.empty(4 * 256 + 8, device="cuda", dtype=torch.bfloat16)[1:1025].view(4, 256), w)  # 2-byte aligned


def test_other_stream_and_graph():
    x = torch.randn(64, 7168, generator=gen(21), device="cuda").to(torch.bfloat16)
    res = torch.randn(64, 7168, generator=gen(22), device="cuda").to(torch.bfloat16)
    w = torch.ones(7168, device="cuda")
    want = W.w8a8_fp8_rms_norm_quant(x, w, residual=res, want_y=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = W.w8a8_fp8_rms_norm_quant(x, w, residual=res, want_y=True)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.w8a8_fp8_rms_norm_quant(x, w, residual=res, q=out[0], scale=out[1], residual_out=out[2], y=out[3])
    x.mul_(2.0)
    graph.replay()
    want = W.w8a8_fp8_rms_norm_quant(x, w, residual=res, want_y=True)
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("form", list(FORMS))
def test_offsets_past_32_bits(form):
    """More than 2^31 values; the last rows and those around the border against the formula."""
    M, K = 270000, 8192
    x = torch.randn(1000, K, generator=gen(31), device="cuda").to(torch.bfloat16).repeat(M // 1000, 1)
    w = torch.rand(K, generator=gen(32), device="cuda") + 0.5
    q, s, r, y = FORMS[form](x, w, residual=x, want_y=True)
    for rows in (slice(0, 300), slice(262100, 262200), slice(M - 300, M)):
        rr, v = norm_reference(x[rows], w, 1e-6, x[rows])
        rq, rs = codes_reference(v, form)
        assert torch.equal(s[rows], rs) and same_codes(q[rows].contiguous(), rq, form)
        assert torch.equal(r[rows], rr) and torch.equal(y[rows], v.to(torch.bfloat16))


@pytest.mark.parametrize("form", list(FORMS))
def test_same_bits_at_every_batch(form):
    """A row's codes do not hang on how many rows there are: one chunk a thread for few, four for many."""
    K = 4096
    x = torch.randn(3000, K, generator=gen(41), device="cuda").to(torch.bfloat16)
    w = torch.rand(K, generator=gen(42), device="cuda") + 0.5
    q, s, _, _ = FORMS[form](x, w)
    for n in (1, 7, 200, 700):
        qn, sn, _, _ = FORMS[form](x[:n], w)
        assert torch.equal(qn.view(torch.uint8), q[:n].view(torch.uint8)) and torch.equal(sn, s[:n])


def test_residual_sum_of_every_value():
    """All 65536 bf16 values plus 96 of them, zeros, subnormals, the largest and non-numbers among those: the binary32
    sum rounded to bf16."""
    every = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    some = [0, 1, 0x7f, 0x80, 0x3f80, 0x3f81, 0x4000, 0x7f7f, 0x7f80, 0x7fc0, 0x4b00, 0x2f55]
    some += [v | 0x8000 for v in some] + torch.randint(0, 65536, (72,), generator=torch.Generator().manual_seed(3)).tolist()
    other = torch.tensor(some, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    x, res = every.expand(96, 65536).contiguous(), other[:, None].expand(96, 65536).contiguous()
    r = W.w8a8_rms_norm_quant(x, torch.ones(65536, device="cuda"), residual=res)[2]
    want = (x.float() + res.float()).to(torch.bfloat16)
    assert bool(((r.view(torch.int16) == want.view(torch.int16)) | (r.isnan() & want.isnan())).all())
