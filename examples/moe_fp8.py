"""An MoE layer on block-scaled FP8 weights: router logits -> experts -> routed FP8 layer, against the same layer in
plain torch on the unquantised weights.

    python examples/moe_fp8.py                          # 64 tokens, 16 experts
    python examples/moe_fp8.py --tokens 4096 --experts 64 --hidden 4096 --inner 2048 --top 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w8a8_dynamic_quant_gb300 as W  # noqa: E402


def block_quantise(w: torch.Tensor):
    """bf16 weight [N,K] -> (E4M3 [N,K], float32 scale per 128 x 128 block), the layout of FP8 checkpoints."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = torch.nn.functional.pad(w.float(), (0, kb * 128 - K, 0, nb * 128 - N)).view(nb, 128, kb, 128)
    s = p.abs().amax(dim=(1, 3)).clamp(min=1e-12) / 448.0
    q = (p / s[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * 128, kb * 128)
    return q[:N, :K].contiguous(), s


def plain_layer(x, ids, weights, w13, w2):
    """The layer in bf16 torch, expert by expert."""
    y = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    inner = w2.shape[2]
    for e in range(w13.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            gu = x[t] @ w13[e].t()
            h = torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]
            y.index_add_(0, t, (h @ w2[e].t()).float() * weights[t, j, None])
    return y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--top", type=int, default=4)
    a = ap.parse_args()
    T, E, H, I, k = a.tokens, a.experts, a.hidden, a.inner, a.top
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    balance = torch.zeros(E, device="cuda")
    w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5).to(torch.bfloat16)

    # at load: the weights' codes and block scales, and a workspace (zeroed once, reused by every call)
    q13, s13 = map(torch.stack, zip(*(block_quantise(w) for w in w13)))
    q2, s2 = map(torch.stack, zip(*(block_quantise(w) for w in w2)))
    ws = W.workspace(W.moe_fp8_layer_workspace_bytes(T, k, H, I, E))

    # a step: route, then the layer
    logits = x.float() @ gate.t()
    ids, weights = W.moe_gate_topk(logits, k, bias=balance, scoring="sigmoid", routed_scale=1.0)
    y = W.moe_fp8_layer(x, ids, weights, q13, s13, q2, s2, ws=ws)
    if W.read_device_status(ws) != 0:
        raise SystemExit("the layer reported a device error")

    ref = plain_layer(x, ids, weights, w13, w2)
    err = float((y.float() - ref).norm() / ref.norm())
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        W.moe_fp8_layer(x, ids, weights, q13, s13, q2, s2, ws=ws, y=y)
    start.record()
    for _ in range(10):
        W.moe_fp8_layer(x, ids, weights, q13, s13, q2, s2, ws=ws, y=y)
    end.record()
    torch.cuda.synchronize()
    print(f"T={T} E={E} H={H} I={I} top-{k}: {start.elapsed_time(end) * 100:.1f} us a layer, "
          f"relative difference from the bf16 layer {err:.3f}")
    # FP8 codes keep three mantissa bits: 2^-4 of a value at most, about 0.026 in the mean, on two operands of two products
    assert err < 0.1


if __name__ == "__main__":
    main()
