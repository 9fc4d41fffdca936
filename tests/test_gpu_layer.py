"""The operators together, as a decoder layer's second half uses them: output projection onto the residual stream, norm
with codes and the bf16 row, router logits, router, expert layer, the next norm; against the formulas in 64 bits.  And
an expert stack kept in bf16 through the grouped product."""
import pytest
import torch

import w8a8_dynamic_quant_gb300 as W

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def norm64(r, w, eps):
    return r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * w


@pytest.mark.parametrize("T", [1, 48, 300])
def test_half_a_layer(T):
    H, E, k, inner, eps = 256, 16, 2, 128, 1e-5
    g = gen(T)
    attn, stream = randn(g, T, H).to(torch.bfloat16), randn(g, T, H, scale=2.0).to(torch.bfloat16)
    wo, gate = randn(g, H, H, scale=H ** -0.5).to(torch.bfloat16), randn(g, E, H, scale=H ** -0.5).to(torch.bfloat16)
    norm1, norm2 = 1.0 + randn(g, H, scale=0.1), (1.0 + randn(g, H, scale=0.1)).to(torch.bfloat16)
    w13 = randn(g, E, 2 * inner, H, scale=H ** -0.5).to(torch.bfloat16)
    w2 = randn(g, E, H, inner, scale=inner ** -0.5).to(torch.bfloat16)
    ws = W.workspace(256)

    # the output projection lands on the residual stream; the norm's bf16 row feeds the router, its codes a dense layer
    r = W.w8a8_bf16_matmul(attn, wo, residual=stream, ws=ws)
    q, s, _, y = W.w8a8_fp8_rms_norm_quant(r, norm1, eps, want_y=True)
    logits = W.w8a8_bf16_matmul(y, gate, out_dtype=torch.float32, ws=ws)
    ids, wts = W.moe_gate_topk(logits, k, scoring="sigmoid")

    r64 = attn.double() @ wo.double().t() + stream.double()
    assert float((r.double() - r64).norm() / r64.norm()) < 2.0 ** -8  # one rounding, half a step at most
    y64 = norm64(r.double(), norm1.double(), eps)
    assert float((y.double() - y64).norm() / y64.norm()) < 2.0 ** -8
    wide = q.double() * s.double().repeat_interleave(128, 1)
    assert float((wide - y64).norm() / y64.norm()) < 2.0 ** -4
    l64 = y.double() @ gate.double().t()
    # a sum of 256 products: (256 / 16 + 16) additions, 2^-23 of the sum of magnitudes each at most
    assert bool(((logits.double() - l64).abs() <= 32 * 2.0 ** -23 * (y.double().abs() @ gate.double().abs().t())).all())
    p = torch.sigmoid(logits.double())
    best = p.sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids, best.indices[:, :k])

    # the experts in bf16: rows sorted by expert, gated first product, second product, weighted sum
    order = ids.flatten().sort(stable=True).indices
    rows, group_list = order // k, torch.bincount(ids.flatten(), minlength=E)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device="cuda")
    h = W.w8a8_bf16_grouped_matmul(y[rows], group_list, w13, activation="swiglu", ws=ws)
    out = W.w8a8_bf16_grouped_matmul(h, group_list, w2, ws=ws)
    moe = W.moe_unpermute_combine(out, pos.view(T, k).int(), wts)
    expert = ids.flatten()[order]
    gu = torch.bmm(w13.double()[expert], y.double()[rows][:, :, None])[:, :, 0]
    h64 = gu[:, :inner] * torch.sigmoid(gu[:, :inner]) * gu[:, inner:]
    o64 = torch.bmm(w2.double()[expert], h64[:, :, None])[:, :, 0]
    m64 = (o64[pos].view(T, k, H) * wts.double()[:, :, None]).sum(1)
    # h, the experts' outputs and the sum are rounded once each
    assert float((moe.double() - m64).norm() / m64.norm()) < 3 * 2.0 ** -8

    # and the next layer's norm adds it to the stream, in place, with int8 codes
    was = r.clone()
    qi, si, r2, _ = W.w8a8_rms_norm_quant(moe, norm2, eps, residual=r, residual_out=r)
    assert r2 is r and torch.equal(r, was + moe)
    n64 = norm64(r.double(), norm2.double(), eps)
    # half a step of the row's scale, and what binary32 adds to it
    assert bool(((qi.double() * si.double()[:, None] - n64).abs() <= si.double()[:, None] * (0.5 + 2.0 ** -10)).all())
    assert W.read_device_status(ws) == 0


def test_codes_feed_the_products():
    """Each norm's codes and scales are the operands of the product of its format: the same bits as the quantiser's on
    the norm's bf16 row wherever that row loses nothing (a weight of ones and rows whose g is a power of two)."""
    M, H, N = 64, 512, 256
    sign = torch.where(torch.rand(M, H, generator=gen(1), device="cuda") < 0.5, -1.0, 1.0)
    x = (sign * 2.0).to(torch.bfloat16)  # S / K = 4; eps below half a unit of it: g = 1/2, v = +-1
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    for norm, quant in ((W.w8a8_rms_norm_quant, W.w8a8_dynamic_quant), (W.w8a8_fp8_rms_norm_quant, W.w8a8_fp8_quant),
                        (W.w8a8_mx_rms_norm_quant, W.w8a8_mx_quant)):
        q, s, _, y = norm(x, one, 1e-8, want_y=True)
        assert torch.equal(y, sign.to(torch.bfloat16))
        q2, s2 = quant(y)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    w = randn(gen(2), N, H, scale=0.05)
    q, s, _, _ = W.w8a8_rms_norm_quant(x, one, 1e-8)
    wq, wsc = W.w8a8_quantize_weight(w.to(torch.bfloat16))
    y = W.w8a8_quant_matmul(q, s, W.w8a8_prepack_weight(wq), wsc, N)
    want = sign.double() @ (wq.double() * wsc.double()[:, None]).t()
    assert float((y.double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) * 1.01
    q, s, _, _ = W.w8a8_fp8_rms_norm_quant(x, one, 1e-8)
    ones = torch.ones(N // 128, H // 128, device="cuda")
    w8 = w.to(torch.float8_e4m3fn)
    y = W.w8a8_fp8_matmul(q, s, w8, ones)
    want = sign.double() @ w8.double().t()
    assert float((y.double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) * 1.01
