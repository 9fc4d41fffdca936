"""Weights as modules hold them, torch.nn.Parameter: taken by the norm and the bf16 products, with the bits of the plain
tensor."""
import pytest
import torch
from torch.nn import Parameter

import w8a8_dynamic_quant_gb300 as W

pytestmark = pytest.mark.gpu


def same(a, b):
    for s, t in zip(a, b):
        assert (s is None and t is None) or (not s.requires_grad and torch.equal(s.view(torch.uint8), t.view(torch.uint8)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("f", [W.w8a8_rms_norm_quant, W.w8a8_fp8_rms_norm_quant, W.w8a8_mx_rms_norm_quant])
def test_norm_weight(f, dtype):
    x = torch.randn(9, 288, device="cuda").to(torch.bfloat16)
    w = (torch.rand(288, device="cuda") + 0.5).to(dtype)
    same(f(x, Parameter(w), residual=x, want_y=True), f(x, w, residual=x, want_y=True))
    with pytest.raises(TypeError):
        f(x, Parameter(w.half()))
    with pytest.raises(ValueError):
        f(x, Parameter(w[:-1].clone()))


def test_products():
    x = torch.randn(9, 64, device="cuda").to(torch.bfloat16)
    w = torch.randn(2, 40, 64, device="cuda").to(torch.bfloat16)
    b = torch.randn(2, 40, device="cuda").to(torch.bfloat16)
    same([W.w8a8_bf16_matmul(x, Parameter(w[0].clone()), Parameter(b[0].clone()), "gelu")],
         [W.w8a8_bf16_matmul(x, w[0], b[0], "gelu")])
    gl = torch.tensor([4, 5], device="cuda")
    same([W.w8a8_bf16_grouped_matmul(x, gl, Parameter(w), Parameter(b), "swiglu")],
         [W.w8a8_bf16_grouped_matmul(x, gl, w, b, "swiglu")])
