"""GB300 (sm_103a) W8A8_DYNAMIC linear layer and MoE-expert path.

A thin torch binding over the C ABI of libw8a8.so (include/w8a8.h): every
function below only checks tensor shapes/dtypes/devices, takes data pointers
and the current CUDA stream, and calls the library.  All arithmetic runs in
the library's CUDA kernels; nothing here computes, and there is no fallback.

BF16 tensors are torch.bfloat16; INT8 tensors torch.int8; scales float32;
group lists int64 (on the device).  Workspaces are zero-filled uint8 device
tensors that can be reused across calls of one kind on one stream: the int8
products and layers of one shape, the FP8 calls, or the bf16 products.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _capi
from ._capi import PACK_F16, PACK_GATE_UP, W8A8Error

__all__ = [
    "PACK_F16", "PACK_GATE_UP", "W8A8Error", "prepacked_bytes", "w8a8_prepack_weight",
    "w8a8_dynamic_quant", "quant_matmul_workspace_bytes", "w8a8_quant_matmul",
    "w8a8_int8_matmul_acc", "grouped_matmul_workspace_bytes", "w8a8_grouped_matmul",
    "w8a8_grouped_matmul_acc", "moe_workspace_bytes", "moe_workspace_offset",
    "moe_w13_swiglu_requant_w2", "read_device_status", "workspace", "w8a8_quant_matmul_noalloc",
    "last_engine", "ENGINE_NONE", "ENGINE_WARP", "ENGINE_DECODE", "ENGINE_TC", "ENGINE_TC_I8",
    "w8a8_quantize_weight", "w8a8_quantize_prepack_weight", "w8a8_static_quant", "w8a8_static_prepare",
    "w8a8_static_quant_matmul", "w8a8_mx_quant", "w8a8_mx_matmul", "moe_route_workspace_bytes", "moe_permute_quant", "moe_unpermute_combine", "moe_layer_workspace_bytes",
    "moe_layer_workspace_offset", "moe_layer", "moe_gate_topk", "w8a8_fp8_quant", "w8a8_fp8_swiglu_quant",
    "fp8_matmul_workspace_bytes", "w8a8_fp8_matmul", "fp8_grouped_matmul_workspace_bytes",
    "w8a8_fp8_grouped_matmul", "moe_fp8_layer_workspace_bytes", "moe_fp8_pad_inner", "moe_fp8_layer",
    "w8a8_rms_norm_quant", "w8a8_fp8_rms_norm_quant", "w8a8_mx_rms_norm_quant", "bf16_matmul_workspace_bytes",
    "w8a8_bf16_matmul", "bf16_grouped_matmul_workspace_bytes", "w8a8_bf16_grouped_matmul",
]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device: torch.device):
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zero-filled device workspace of `nbytes` bytes (256-byte aligned by the caching allocator)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def prepacked_bytes(E: int, N: int, K: int, flags: int = 0) -> int:
    return int(_capi.lib().w8a8_prepacked_bytes(E, N, K, flags))


def w8a8_prepack_weight(w: torch.Tensor, flags: int = 0) -> torch.Tensor:
    """INT8 weight [N,K] or expert stack [E,N,K] -> packed device buffer (uint8)."""
    w3 = w.unsqueeze(0) if w.dim() == 2 else w
    if w3.dim() != 3:
        raise ValueError("w must be [N,K] or [E,N,K]")
    _need(w3, "w", torch.int8)
    E, N, K = w3.shape
    nbytes = prepacked_bytes(E, N, K, flags)
    if nbytes == 0:
        raise ValueError("bad weight shape")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    with torch.cuda.device(w.device):
        _capi.check("w8a8_prepack_weight", _capi.lib().w8a8_prepack_weight(
            w3.data_ptr(), E, N, K, flags, packed.data_ptr(), _stream(w.device)))
    return packed


def _weight3(w: torch.Tensor):
    w3 = w.unsqueeze(0) if w.dim() == 2 else w
    if w3.dim() != 3:
        raise ValueError("w must be [N,K] or [E,N,K]")
    _need(w3, "w", torch.bfloat16)
    return w3


def w8a8_quantize_weight(w: torch.Tensor):
    """BF16 weight [N,K] or [E,N,K] -> (int8 q of the same shape, float32 per-channel scales [N] / [E,N])."""
    w3 = _weight3(w)
    E, N, K = w3.shape
    q = torch.empty((E, N, K), dtype=torch.int8, device=w.device)
    scale = torch.empty((E, N), dtype=torch.float32, device=w.device)
    with torch.cuda.device(w.device):
        _capi.check("w8a8_quantize_weight", _capi.lib().w8a8_quantize_weight(
            w3.data_ptr(), E, N, K, q.data_ptr(), scale.data_ptr(), _stream(w.device)))
    return (q[0], scale[0]) if w.dim() == 2 else (q, scale)


def w8a8_quantize_prepack_weight(w: torch.Tensor, flags: int = 0, packed: Optional[torch.Tensor] = None,
                                 scale: Optional[torch.Tensor] = None):
    """BF16 weight [N,K] or [E,N,K] -> (packed device buffer, float32 per-channel scales [N] / [E,N]),
    quantised per channel and packed in one pass."""
    w3 = _weight3(w)
    E, N, K = w3.shape
    nbytes = prepacked_bytes(E, N, K, flags)
    if nbytes == 0:
        raise ValueError("bad weight shape")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=w.device) if packed is None else packed
    _need(packed, "packed", torch.uint8, (nbytes,), w.device)
    scale = torch.empty((E, N), dtype=torch.float32, device=w.device) if scale is None else scale.view(E, N)
    _need(scale, "scale", torch.float32, (E, N), w.device)
    with torch.cuda.device(w.device):
        _capi.check("w8a8_quantize_prepack_weight", _capi.lib().w8a8_quantize_prepack_weight(
            w3.data_ptr(), E, N, K, flags, packed.data_ptr(), scale.data_ptr(), _stream(w.device)))
    return packed, (scale[0] if w.dim() == 2 else scale)


def w8a8_dynamic_quant(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                       scale: Optional[torch.Tensor] = None):
    """BF16 x [M,K] -> (int8 q [M,K], float32 scale [M])."""
    _need(x, "x", torch.bfloat16)
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device) if q is None else q
    scale = torch.empty((M,), dtype=torch.float32, device=x.device) if scale is None else scale
    _need(q, "q", torch.int8, (M, K), x.device)
    _need(scale, "scale", torch.float32, (M,), x.device)
    with torch.cuda.device(x.device):
        _capi.check("w8a8_dynamic_quant", _capi.lib().w8a8_dynamic_quant(
            x.data_ptr(), M, K, q.data_ptr(), scale.data_ptr(), _stream(x.device)))
    return q, scale


def w8a8_mx_quant(x: torch.Tensor, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None):
    """MXFP8: bf16 x [M,K] (K % 32 == 0) -> (uint8 E4M3 codes [M,K], uint8 E8M0 scales [M,K/32])."""
    _need(x, "x", torch.bfloat16)
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device) if q is None else q
    scale = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device) if scale is None else scale
    _need(q, "q", torch.uint8, (M, K), x.device)
    _need(scale, "scale", torch.uint8, (M, K // 32), x.device)
    with torch.cuda.device(x.device):
        _capi.check("w8a8_mx_quant", _capi.lib().w8a8_mx_quant(
            x.data_ptr(), M, K, q.data_ptr(), scale.data_ptr(), _stream(x.device)))
    return q, scale


def w8a8_mx_matmul(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                   y: Optional[torch.Tensor] = None):
    """MXFP8 contraction: E4M3 qa [M,K] + E8M0 sa [M,K/32], E4M3 qw [N,K] + E8M0 sw [N,K/32] -> bf16 y [M,N]."""
    _need(qa, "qa", torch.uint8)
    M, K = qa.shape
    dev = qa.device
    _need(sa, "sa", torch.uint8, (M, K // 32), dev)
    _need(qw, "qw", torch.uint8, None, dev)
    N = qw.shape[0]
    _need(sw, "sw", torch.uint8, (N, K // 32), dev)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, (M, N), dev)
    with torch.cuda.device(dev):
        _capi.check("w8a8_mx_matmul", _capi.lib().w8a8_mx_matmul(
            qa.data_ptr(), sa.data_ptr(), M, K, qw.data_ptr(), sw.data_ptr(), N, y.data_ptr(), _stream(dev)))
    return y


def w8a8_static_quant(x: torch.Tensor, input_scale: float, input_offset: int, q: Optional[torch.Tensor] = None):
    """Static W8A8 quantisation: bf16 x [M,K] -> int8 q = clamp(rint(x / s) + o, -128, 127)."""
    _need(x, "x", torch.bfloat16)
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device) if q is None else q
    _need(q, "q", torch.int8, (M, K), x.device)
    with torch.cuda.device(x.device):
        _capi.check("w8a8_static_quant", _capi.lib().w8a8_static_quant(
            x.data_ptr(), M, K, float(input_scale), int(input_offset), q.data_ptr(), _stream(x.device)))
    return q


def w8a8_static_prepare(w: torch.Tensor, weight_scale: torch.Tensor, input_scale: float, input_offset: int,
                        bias: Optional[torch.Tensor] = None):
    """Load time: int8 W [N,K], float32 weight scales [N] (+ bf16 bias [N]) -> (float32 deq_scale [N],
    int32 quant_bias [N])."""
    _need(w, "w", torch.int8)
    N, K = w.shape
    dev = w.device
    _need(weight_scale, "weight_scale", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, (N,), dev)
    deq = torch.empty((N,), dtype=torch.float32, device=dev)
    qb = torch.empty((N,), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _capi.check("w8a8_static_prepare", _capi.lib().w8a8_static_prepare(
            w.data_ptr(), N, K, weight_scale.data_ptr(), float(input_scale), int(input_offset), _ptr(bias),
            deq.data_ptr(), qb.data_ptr(), _stream(dev)))
    return deq, qb


def w8a8_static_quant_matmul(q: torch.Tensor, w_packed: torch.Tensor, deq_scale: torch.Tensor,
                             quant_bias: torch.Tensor, ws: Optional[torch.Tensor] = None,
                             y: Optional[torch.Tensor] = None):
    """Static W8A8 matmul: int8 q [M,K] x packed W [N,K] -> bf16 y = bf16(float(acc + quant_bias) * deq_scale)."""
    _need(q, "q", torch.int8)
    M, K = q.shape
    dev = q.device
    _need(deq_scale, "deq_scale", torch.float32, None, dev)
    N = deq_scale.shape[0]
    _need(quant_bias, "quant_bias", torch.int32, (N,), dev)
    _need(w_packed, "w_packed", torch.uint8, None, dev)
    ws = workspace(quant_matmul_workspace_bytes(M, N, K), dev) if ws is None else ws
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, (M, N), dev)
    with torch.cuda.device(dev):
        _capi.check("w8a8_static_quant_matmul", _capi.lib().w8a8_static_quant_matmul(
            q.data_ptr(), M, K, w_packed.data_ptr(), deq_scale.data_ptr(), quant_bias.data_ptr(), N, y.data_ptr(),
            ws.data_ptr(), ws.numel(), _stream(dev)))
    return y


def quant_matmul_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_capi.lib().w8a8_quant_matmul_workspace_bytes(M, N, K))


def w8a8_quant_matmul(q: torch.Tensor, x_scale: torch.Tensor, w_packed: torch.Tensor,
                      w_scale: torch.Tensor, N: int, bias: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """int8 q [M,K] x packed W [N,K] -> bf16 y [M,N] = ((acc * x_scale) * w_scale) + bias."""
    _need(q, "q", torch.int8)
    M, K = q.shape
    dev = q.device
    _need(x_scale, "x_scale", torch.float32, (M,), dev)
    _need(w_packed, "w_packed", torch.uint8, None, dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, (N,), dev)
    ws = workspace(quant_matmul_workspace_bytes(M, N, K), dev) if ws is None else ws
    _need(ws, "ws", torch.uint8, None, dev)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, (M, N), dev)
    with torch.cuda.device(dev):
        _capi.check("w8a8_quant_matmul", _capi.lib().w8a8_quant_matmul(
            q.data_ptr(), x_scale.data_ptr(), M, K, w_packed.data_ptr(), w_scale.data_ptr(), N,
            _ptr(bias), y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(dev)))
    return y


def w8a8_quant_matmul_noalloc(q: torch.Tensor, x_scale: torch.Tensor, w_packed: torch.Tensor,
                              w_scale: torch.Tensor, N: int, bias: Optional[torch.Tensor] = None,
                              y: Optional[torch.Tensor] = None):
    """w8a8_quant_matmul for callers that cannot allocate device memory: the
    library's built-in scratch array replaces the workspace (y must be given by
    such callers; it is allocated here only for convenience)."""
    _need(q, "q", torch.int8)
    M, K = q.shape
    dev = q.device
    _need(x_scale, "x_scale", torch.float32, (M,), dev)
    _need(w_packed, "w_packed", torch.uint8, None, dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, (N,), dev)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, (M, N), dev)
    with torch.cuda.device(dev):
        _capi.check("w8a8_quant_matmul_noalloc", _capi.lib().w8a8_quant_matmul_noalloc(
            q.data_ptr(), x_scale.data_ptr(), M, K, w_packed.data_ptr(), w_scale.data_ptr(), N,
            _ptr(bias), y.data_ptr(), _stream(dev)))
    return y


def w8a8_int8_matmul_acc(q: torch.Tensor, w_packed: torch.Tensor, N: int,
                         ws: Optional[torch.Tensor] = None):
    """Exact INT32 accumulators acc [M,N] = q [M,K] x W[N,K]^T (validation entry)."""
    _need(q, "q", torch.int8)
    M, K = q.shape
    dev = q.device
    ws = workspace(quant_matmul_workspace_bytes(M, N, K), dev) if ws is None else ws
    acc = torch.empty((M, N), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _capi.check("w8a8_int8_matmul_acc", _capi.lib().w8a8_int8_matmul_acc(
            q.data_ptr(), M, K, w_packed.data_ptr(), N, acc.data_ptr(), ws.data_ptr(), ws.numel(),
            _stream(dev)))
    return acc


def grouped_matmul_workspace_bytes(E: int, R: int, N: int, K: int) -> int:
    return int(_capi.lib().w8a8_grouped_matmul_workspace_bytes(E, R, N, K))


def w8a8_grouped_matmul(q: torch.Tensor, x_scale: torch.Tensor, group_list: torch.Tensor,
                        w_packed: torch.Tensor, w_scale: torch.Tensor,
                        ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """int8 q [R,K] (rows grouped by expert) x packed W [E,N,K] -> bf16 [R,N]."""
    _need(q, "q", torch.int8)
    R, K = q.shape
    dev = q.device
    _need(group_list, "group_list", torch.int64, None, dev)
    E = group_list.numel()
    _need(w_scale, "w_scale", torch.float32, None, dev)
    N = w_scale.shape[-1]
    _need(x_scale, "x_scale", torch.float32, (R,), dev)
    ws = workspace(grouped_matmul_workspace_bytes(E, R, N, K), dev) if ws is None else ws
    y = torch.empty((R, N), dtype=torch.bfloat16, device=dev) if y is None else y
    with torch.cuda.device(dev):
        _capi.check("w8a8_grouped_matmul", _capi.lib().w8a8_grouped_matmul(
            q.data_ptr(), x_scale.data_ptr(), group_list.data_ptr(), E, R, K, w_packed.data_ptr(),
            w_scale.data_ptr(), N, y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(dev)))
    return y


def w8a8_grouped_matmul_acc(q: torch.Tensor, group_list: torch.Tensor, w_packed: torch.Tensor,
                            N: int, ws: Optional[torch.Tensor] = None):
    _need(q, "q", torch.int8)
    R, K = q.shape
    dev = q.device
    _need(group_list, "group_list", torch.int64, None, dev)
    E = group_list.numel()
    ws = workspace(grouped_matmul_workspace_bytes(E, R, N, K), dev) if ws is None else ws
    acc = torch.empty((R, N), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _capi.check("w8a8_grouped_matmul_acc", _capi.lib().w8a8_grouped_matmul_acc(
            q.data_ptr(), group_list.data_ptr(), E, R, K, w_packed.data_ptr(), N, acc.data_ptr(),
            ws.data_ptr(), ws.numel(), _stream(dev)))
    return acc


def moe_workspace_bytes(R: int, H: int, I: int, E: int) -> int:
    return int(_capi.lib().moe_workspace_bytes(R, H, I, E))


def moe_workspace_offset(R: int, H: int, I: int, E: int, which: int) -> int:
    return int(_capi.lib().moe_workspace_offset(R, H, I, E, which))


def moe_w13_swiglu_requant_w2(x: torch.Tensor, x_scale: Optional[torch.Tensor],
                              group_list: torch.Tensor, w13_packed: torch.Tensor,
                              w13_scale: torch.Tensor, w2_packed: torch.Tensor,
                              w2_scale: torch.Tensor, ws: Optional[torch.Tensor] = None,
                              y: Optional[torch.Tensor] = None):
    """MoE expert FFN: x bf16 [R,H] (x_scale None) or int8 [R,H] with x_scale [R] -> bf16 [R,H]."""
    R, H = x.shape
    dev = x.device
    if x_scale is None:
        _need(x, "x", torch.bfloat16)
    else:
        _need(x, "x", torch.int8)
        _need(x_scale, "x_scale", torch.float32, (R,), dev)
    _need(group_list, "group_list", torch.int64, None, dev)
    E = group_list.numel()
    _need(w13_scale, "w13_scale", torch.float32, None, dev)
    I = w13_scale.shape[-1] // 2
    _need(w2_scale, "w2_scale", torch.float32, (E, H), dev)
    ws = workspace(moe_workspace_bytes(R, H, I, E), dev) if ws is None else ws
    y = torch.empty((R, H), dtype=torch.bfloat16, device=dev) if y is None else y
    with torch.cuda.device(dev):
        _capi.check("moe_w13_swiglu_requant_w2", _capi.lib().moe_w13_swiglu_requant_w2(
            x.data_ptr(), _ptr(x_scale), group_list.data_ptr(), E, R, H, I, w13_packed.data_ptr(),
            w13_scale.data_ptr(), w2_packed.data_ptr(), w2_scale.data_ptr(), ws.data_ptr(),
            ws.numel(), y.data_ptr(), _stream(dev)))
    return y


def moe_route_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(_capi.lib().moe_route_workspace_bytes(T, k, E))


def moe_permute_quant(x: torch.Tensor, x_scale: Optional[torch.Tensor], topk_ids: torch.Tensor, E: int,
                      ws: Optional[torch.Tensor] = None, out=None):
    """Token rows -> routed rows grouped by expert.  x bf16 [T,H] (x_scale None: each token quantised
    once) or int8 [T,H] with x_scale [T]; topk_ids int64 [T,k].  Returns (int8 xq [T*k,H],
    float32 xs [T*k], int64 group_list [E], int32 pos [T,k]), written into `out` when given."""
    T, H = x.shape
    dev = x.device
    if x_scale is None:
        _need(x, "x", torch.bfloat16)
    else:
        _need(x, "x", torch.int8)
        _need(x_scale, "x_scale", torch.float32, (T,), dev)
    _need(topk_ids, "topk_ids", torch.int64, None, dev)
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError("topk_ids must be [T,k]")
    k = topk_ids.shape[1]
    ws = workspace(moe_route_workspace_bytes(T, k, E), dev) if ws is None else ws
    _need(ws, "ws", torch.uint8, None, dev)
    if out is None:
        out = (torch.empty((T * k, H), dtype=torch.int8, device=dev),
               torch.empty((T * k,), dtype=torch.float32, device=dev),
               torch.empty((E,), dtype=torch.int64, device=dev),
               torch.empty((T, k), dtype=torch.int32, device=dev))
    xq, xs, group_list, pos = out
    _need(xq, "xq", torch.int8, (T * k, H), dev)
    _need(xs, "xs", torch.float32, (T * k,), dev)
    _need(group_list, "group_list", torch.int64, (E,), dev)
    _need(pos, "pos", torch.int32, (T, k), dev)
    with torch.cuda.device(dev):
        _capi.check("moe_permute_quant", _capi.lib().moe_permute_quant(
            x.data_ptr(), _ptr(x_scale), topk_ids.data_ptr(), T, k, E, H, xq.data_ptr(), xs.data_ptr(),
            group_list.data_ptr(), pos.data_ptr(), ws.data_ptr(), ws.numel(), _stream(dev)))
    return xq, xs, group_list, pos


def moe_unpermute_combine(y_routed: torch.Tensor, pos: torch.Tensor, topk_weights: torch.Tensor,
                          ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """bf16 y_routed [T*k,H], int32 pos [T,k], float32 topk_weights [T,k] -> bf16 y [T,H]."""
    _need(y_routed, "y_routed", torch.bfloat16)
    dev = y_routed.device
    _need(pos, "pos", torch.int32, None, dev)
    if pos.dim() != 2:
        raise ValueError("pos must be [T,k]")
    T, k = pos.shape
    H = y_routed.shape[1]
    if y_routed.shape[0] != T * k:
        raise ValueError("y_routed must have T*k rows")
    _need(topk_weights, "topk_weights", torch.float32, (T, k), dev)
    ws = workspace(_capi.STATUS_BYTES, dev) if ws is None else ws
    _need(ws, "ws", torch.uint8, None, dev)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, (T, H), dev)
    with torch.cuda.device(dev):
        _capi.check("moe_unpermute_combine", _capi.lib().moe_unpermute_combine(
            y_routed.data_ptr(), pos.data_ptr(), topk_weights.data_ptr(), T, k, H, y.data_ptr(),
            ws.data_ptr(), ws.numel(), _stream(dev)))
    return y


def moe_layer_workspace_bytes(T: int, k: int, H: int, I: int, E: int) -> int:
    return int(_capi.lib().moe_layer_workspace_bytes(T, k, H, I, E))


def moe_layer_workspace_offset(T: int, k: int, H: int, I: int, E: int, which: int) -> int:
    return int(_capi.lib().moe_layer_workspace_offset(T, k, H, I, E, which))


def moe_layer(x: torch.Tensor, x_scale: Optional[torch.Tensor], topk_ids: torch.Tensor,
              topk_weights: torch.Tensor, w13_packed: torch.Tensor, w13_scale: torch.Tensor,
              w2_packed: torch.Tensor, w2_scale: torch.Tensor, ws: Optional[torch.Tensor] = None,
              y: Optional[torch.Tensor] = None):
    """MoE layer from token rows and router output: x bf16 [T,H] (or int8 with x_scale [T]),
    topk_ids int64 [T,k], topk_weights float32 [T,k] -> bf16 y [T,H]."""
    T, H = x.shape
    dev = x.device
    if x_scale is None:
        _need(x, "x", torch.bfloat16)
    else:
        _need(x, "x", torch.int8)
        _need(x_scale, "x_scale", torch.float32, (T,), dev)
    _need(topk_ids, "topk_ids", torch.int64, None, dev)
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError("topk_ids must be [T,k]")
    k = topk_ids.shape[1]
    _need(topk_weights, "topk_weights", torch.float32, (T, k), dev)
    _need(w13_scale, "w13_scale", torch.float32, None, dev)
    E = w13_scale.shape[0]
    I = w13_scale.shape[-1] // 2
    _need(w2_scale, "w2_scale", torch.float32, (E, H), dev)
    ws = workspace(moe_layer_workspace_bytes(T, k, H, I, E), dev) if ws is None else ws
    _need(ws, "ws", torch.uint8, None, dev)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, (T, H), dev)
    with torch.cuda.device(dev):
        _capi.check("moe_layer", _capi.lib().moe_layer(
            x.data_ptr(), _ptr(x_scale), topk_ids.data_ptr(), topk_weights.data_ptr(), T, k, E, H, I,
            w13_packed.data_ptr(), w13_scale.data_ptr(), w2_packed.data_ptr(), w2_scale.data_ptr(),
            ws.data_ptr(), ws.numel(), y.data_ptr(), _stream(dev)))
    return y


# The calls below run a few microseconds of GPU work at decode sizes, so their host side is kept short: plain attribute
# tests of a tensor in one expression (the full _need only to say what is wrong), no device guard where the tensors'
# device is already current, and the library's functions looked up once.  On the GPU host (aarch64) a quantisation
# call takes about 9 us this way, 16 us with a guard, _stream and _need for every tensor; its two allocations
# and the launch are 5 of them.

_bound = {}
_raw_stream = _get_device = None  # torch's own, looked up with the first function: a torch without CUDA lacks them
_empty, _empty_like, _Tensor = torch.empty, torch.empty_like, torch.Tensor
_BF16, _F32, _I64, _E4M3 = torch.bfloat16, torch.float32, torch.int64, torch.float8_e4m3fn


def _bind(name: str):
    global _raw_stream, _get_device
    _raw_stream, _get_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    fn = _bound[name] = getattr(_capi.lib(), name)
    return fn


def _call(name: str, index: int, *args):
    """The library's `name` on the current stream of CUDA device `index` (the last argument)."""
    fn = _bound.get(name)
    if fn is None:
        fn = _bind(name)
    if _get_device() == index:
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code:
        raise W8A8Error(name, code)


def _size(name: str, *args) -> int:
    return int(getattr(_capi.lib(), name)(*args))


def _check(t, name: str, dtype: torch.dtype, shape, index: int):
    """_need for a tensor of known shape on CUDA device `index`."""
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == index >= 0 and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, dtype, shape, torch.device("cuda", index) if index >= 0 else None)


def _check_e4m3(t, name: str, shape, index: int):
    """E4M3 codes: torch.float8_e4m3fn, or their bytes as torch.uint8."""
    if not (type(t) is torch.Tensor and t.dtype is torch.float8_e4m3fn and t.get_device() == index >= 0
            and t.shape == shape and t.is_contiguous()):
        as_bytes = isinstance(t, torch.Tensor) and t.dtype is torch.uint8
        _need(t, name, torch.uint8 if as_bytes else torch.float8_e4m3fn, shape,
              torch.device("cuda", index) if index >= 0 else None)


def _dims(t, name: str, n: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")
    return t.shape


def _check_ws(ws, need_fn, index: int):
    if ws is None:
        return workspace(need_fn(), torch.device("cuda", index))
    if not (type(ws) is torch.Tensor and ws.dtype is torch.uint8 and ws.get_device() == index and ws.is_contiguous()):
        _need(ws, "ws", torch.uint8, None, torch.device("cuda", index))
    return ws


def _blocks(n: int) -> int:
    return (n + 127) // 128


def moe_gate_topk(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None, scoring: str = "softmax",
                  n_group: int = 1, topk_group: int = 1, group_score: str = "max", renormalize: bool = True,
                  routed_scale: float = 1.0, ids: Optional[torch.Tensor] = None,
                  weights: Optional[torch.Tensor] = None):
    """Expert router: float32 or bfloat16 logits [T,E] -> (int64 topk_ids [T,k], float32 topk_weights [T,k]).

    scoring "softmax" or "sigmoid"; bias float32 [E] is added to the scores for the choice alone, not to the
    weights; n_group runs of E / n_group experts of which the topk_group best stay, by their largest key
    (group_score "max") or the sum of their two largest ("top2").  Ties go to the lowest index; an expert whose
    logit is -inf or NaN is chosen only when no other is left, with weight 0."""
    T, E = _dims(logits, "logits", 2)
    dtype, dev = logits.dtype, logits.get_device()
    if dtype is not _F32 and dtype is not _BF16:
        raise TypeError(f"logits must be torch.float32 or torch.bfloat16, got {dtype}")
    if not (dev >= 0 and logits.is_contiguous()):
        _check(logits, "logits", dtype, (T, E), dev)
    if bias is not None:
        _check(bias, "bias", _F32, (E,), dev)
    if scoring == "sigmoid":
        flags = _capi.GATE_SIGMOID
    elif scoring == "softmax":
        flags = 0
    else:
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
    if group_score == "top2":
        flags |= _capi.GATE_GROUP_TOP2
    elif group_score != "max":
        raise ValueError(f"group_score must be 'max' or 'top2', got {group_score!r}")
    if 1 <= topk_group <= n_group and E % n_group == 0 and k > topk_group * (E // n_group):
        raise ValueError(f"k = {k} exceeds the {topk_group * (E // n_group)} experts of {topk_group} groups")
    if renormalize:
        flags |= _capi.GATE_RENORM
    if dtype is torch.bfloat16:
        flags |= _capi.GATE_BF16
    if ids is None:
        ids = _empty((T, max(k, 0)), dtype=_I64, device=logits.device)
    else:
        _check(ids, "ids", torch.int64, (T, k), dev)
    if weights is None:
        weights = _empty((T, max(k, 0)), dtype=_F32, device=logits.device)
    else:
        _check(weights, "weights", torch.float32, (T, k), dev)
    _call("moe_gate_topk", dev, logits.data_ptr(), T, E, None if bias is None else bias.data_ptr(), n_group, topk_group,
          k, routed_scale, flags, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def _quant_checks(x, name: str, columns: int, q, scale):
    """The quantisers' tensors where one is not as the common call has it: [M, columns * K] bf16 and given outputs."""
    M, width = _dims(x, name, 2)
    dev = x.get_device()
    _check(x, name, _BF16, (M, width), dev)
    if width % columns:
        raise ValueError(f"{name} must be [R,{columns}I]")
    K = width // columns
    if q is not None:
        _check_e4m3(q, "q", (M, K), dev)
    if scale is not None:
        _check(scale, "scale", _F32, (M, _blocks(K)), dev)


def w8a8_fp8_quant(x: torch.Tensor, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None):
    """BF16 x [M,K] (K % 16 == 0) -> (float8_e4m3fn q [M,K], float32 scale [M, ceil(K/128)])."""
    if not (q is None and scale is None and type(x) is _Tensor and x.dtype is _BF16 and x.dim() == 2 and x.is_cuda
            and x.is_contiguous()):
        _quant_checks(x, "x", 1, q, scale)
    M, K = x.shape
    dev = x.get_device()
    if q is None:
        q = _empty((M, K), dtype=_E4M3, device=x.device)
    if scale is None:
        scale = _empty((M, (K + 127) // 128), dtype=_F32, device=x.device)
    _call("w8a8_fp8_quant", dev, x.data_ptr(), M, K, q.data_ptr(), scale.data_ptr())
    return q, scale


def w8a8_fp8_swiglu_quant(y13: torch.Tensor, q: Optional[torch.Tensor] = None,
                          scale: Optional[torch.Tensor] = None):
    """BF16 y13 [R,2I] (gate half, up half) -> SwiGLU, quantised: (float8_e4m3fn q [R,I], float32 scale
    [R, ceil(I/128)])."""
    if not (q is None and scale is None and type(y13) is _Tensor and y13.dtype is _BF16 and y13.dim() == 2
            and y13.is_cuda and y13.is_contiguous() and y13.shape[1] % 2 == 0):
        _quant_checks(y13, "y13", 2, q, scale)
    R, two = y13.shape
    I, dev = two // 2, y13.get_device()
    if q is None:
        q = _empty((R, I), dtype=_E4M3, device=y13.device)
    if scale is None:
        scale = _empty((R, (I + 127) // 128), dtype=_F32, device=y13.device)
    _call("w8a8_fp8_swiglu_quant", dev, y13.data_ptr(), R, I, q.data_ptr(), scale.data_ptr())
    return q, scale


def fp8_matmul_workspace_bytes(M: int, N: int, K: int) -> int:
    return _size("w8a8_fp8_matmul_workspace_bytes", M, N, K)


def w8a8_fp8_matmul(q: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None):
    """E4M3 q [M,K] with x_scale [M, ceil(K/128)] x E4M3 w [N,K] with w_scale [ceil(N/128), ceil(K/128)]
    (+ bf16 bias [N]) -> bf16 y [M,N].  Keep a workspace (`ws`) over calls: without one every call zero-fills its own."""
    M, K = _dims(q, "q", 2)
    N = _dims(w, "w", 2)[0]
    dev, kb = q.get_device(), (K + 127) // 128
    if not (dev >= 0 and q.dtype is _E4M3 and w.dtype is _E4M3 and type(x_scale) is _Tensor and type(w_scale) is _Tensor
            and x_scale.dtype is _F32 and w_scale.dtype is _F32 and w.get_device() == dev
            and x_scale.get_device() == dev and w_scale.get_device() == dev and w.shape[1] == K
            and x_scale.shape == (M, kb) and w_scale.shape == ((N + 127) // 128, kb) and q.is_contiguous()
            and w.is_contiguous() and x_scale.is_contiguous() and w_scale.is_contiguous()):
        _check_e4m3(q, "q", (M, K), dev)
        _check_e4m3(w, "w", (N, K), dev)
        _check(x_scale, "x_scale", _F32, (M, kb), dev)
        _check(w_scale, "w_scale", _F32, (_blocks(N), kb), dev)
    if bias is not None:
        _check(bias, "bias", torch.bfloat16, (N,), dev)
    ws = _check_ws(ws, lambda: fp8_matmul_workspace_bytes(M, N, K), dev)
    if y is None:
        y = _empty((M, N), dtype=_BF16, device=q.device)
    else:
        _check(y, "y", _BF16, (M, N), dev)
    _call("w8a8_fp8_matmul", dev, q.data_ptr(), x_scale.data_ptr(), M, K, w.data_ptr(), w_scale.data_ptr(), N,
          None if bias is None else bias.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel())
    return y


def fp8_grouped_matmul_workspace_bytes(E: int, R: int, N: int, K: int) -> int:
    return _size("w8a8_fp8_grouped_matmul_workspace_bytes", E, R, N, K)


def w8a8_fp8_grouped_matmul(q: torch.Tensor, x_scale: torch.Tensor, group_list: torch.Tensor, w: torch.Tensor,
                            w_scale: torch.Tensor, ws: Optional[torch.Tensor] = None,
                            y: Optional[torch.Tensor] = None):
    """E4M3 q [R,K] (rows grouped by expert) with x_scale [R, ceil(K/128)] x E4M3 w [E,N,K] with w_scale
    [E, ceil(N/128), ceil(K/128)] -> bf16 y [R,N].  Keep a workspace (`ws`) over calls: without one every call
    zero-fills its own."""
    R, K = _dims(q, "q", 2)
    E, N, K2 = _dims(w, "w", 3)
    dev, kb = q.get_device(), (K + 127) // 128
    if not (dev >= 0 and q.dtype is _E4M3 and w.dtype is _E4M3 and type(x_scale) is _Tensor and type(w_scale) is _Tensor
            and type(group_list) is _Tensor and x_scale.dtype is _F32 and w_scale.dtype is _F32
            and group_list.dtype is _I64 and w.get_device() == dev and x_scale.get_device() == dev
            and w_scale.get_device() == dev and group_list.get_device() == dev and K2 == K
            and x_scale.shape == (R, kb) and w_scale.shape == (E, (N + 127) // 128, kb) and group_list.shape == (E,)
            and q.is_contiguous() and w.is_contiguous() and x_scale.is_contiguous() and w_scale.is_contiguous()
            and group_list.is_contiguous()):
        _check_e4m3(q, "q", (R, K), dev)
        _check_e4m3(w, "w", (E, N, K), dev)
        _check(group_list, "group_list", _I64, (E,), dev)
        _check(x_scale, "x_scale", _F32, (R, kb), dev)
        _check(w_scale, "w_scale", _F32, (E, _blocks(N), kb), dev)
    ws = _check_ws(ws, lambda: fp8_grouped_matmul_workspace_bytes(E, R, N, K), dev)
    if y is None:
        y = _empty((R, N), dtype=_BF16, device=q.device)
    else:
        _check(y, "y", _BF16, (R, N), dev)
    _call("w8a8_fp8_grouped_matmul", dev, q.data_ptr(), x_scale.data_ptr(), group_list.data_ptr(), E, R, K,
          w.data_ptr(), w_scale.data_ptr(), N, y.data_ptr(), ws.data_ptr(), ws.numel())
    return y


def moe_fp8_layer_workspace_bytes(T: int, k: int, H: int, I: int, E: int) -> int:
    return _size("moe_fp8_layer_workspace_bytes", T, k, H, I, E)


def moe_fp8_pad_inner(w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor):
    """Weights whose gate and up halves have their own scale blocks, laid out once for moe_fp8_layer where I % 128 != 0.

    E4M3 w13 [E,2I,H] (gate rows, then up rows), its float32 scales [E,2,ceil(I/128),ceil(H/128)] (torch.stack of
    the two stored ones, dim 1) and E4M3 w2 [E,H,I] -> the same with I rounded up to a multiple of 128: the halves'
    rows and w2's columns end in zero codes, which add nothing.  w2's scales serve both.  The tensors themselves
    where I % 128 == 0.  Any device."""
    E, two, H = _dims(w13, "w13", 3)
    I, pad = two // 2, -(two // 2) % 128
    for t, name in ((w13, "w13"), (w2, "w2")):
        if isinstance(t, torch.Tensor) and t.dtype not in (_E4M3, torch.uint8):
            raise TypeError(f"{name} must be {_E4M3}, got {t.dtype}")
    if two % 2 or tuple(_dims(w2, "w2", 3)) != (E, H, I):
        raise ValueError("w13 must be [E,2I,H] and w2 [E,H,I]")
    if tuple(_dims(w13_scale, "w13_scale", 4)) != (E, 2, _blocks(I), _blocks(H)):
        raise ValueError(f"w13_scale has shape {tuple(w13_scale.shape)}, expected {(E, 2, _blocks(I), _blocks(H))}")
    if w13_scale.dtype is not _F32:
        raise TypeError(f"w13_scale must be {_F32}, got {w13_scale.dtype}")
    if pad == 0:
        return w13, w13_scale, w2
    # (as bytes: torch pads no float8)
    p13 = torch.nn.functional.pad(w13.view(torch.uint8).view(E, 2, I, H), (0, 0, 0, pad)).view(E, two + 2 * pad, H)
    p2 = torch.nn.functional.pad(w2.view(torch.uint8), (0, pad))
    return p13.view(w13.dtype), w13_scale, p2.view(w2.dtype)


def moe_fp8_layer(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, w13: torch.Tensor,
                  w13_scale: torch.Tensor, w2: torch.Tensor, w2_scale: torch.Tensor,
                  ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """MoE layer on block-scaled FP8 weights: bf16 x [T,H], topk_ids int64 [T,k] and topk_weights float32 [T,k]
    (moe_gate_topk), E4M3 w13 [E,2I,H] (gate rows, then up rows) and w2 [E,H,I] with float32 block scales -> bf16
    y [T,H].

    w2_scale [E,ceil(H/128),ceil(I/128)].  w13_scale in one of two forms:
      [E,2,ceil(I/128),ceil(H/128)]  gate and up scaled on their own, as checkpoints store the two matrices:
                                     torch.stack([gate_scale, up_scale], 1).  I % 128 == 0; other I are laid out
                                     for it once by moe_fp8_pad_inner.
      [E,ceil(2I/128),ceil(H/128)]   blocks over the 2I joined rows (the two forms are the same for I % 128 == 0).
                                     Where I % 128 != 0 a block spans both halves: two scale arrays made for the
                                     halves are NOT this form, even where their rows add up to the same number.
    Keep a workspace (`ws`) over calls: without one every call zero-fills its own."""
    T, H = _dims(x, "x", 2)
    T2, k = _dims(topk_ids, "topk_ids", 2)
    E, two, _ = _dims(w13, "w13", 3)
    if T2 != T:
        raise ValueError("topk_ids must be [T,k]")
    if two % 2:
        raise ValueError("w13 must be [E,2I,H]")
    I, dev = two // 2, x.get_device()
    _check(x, "x", torch.bfloat16, (T, H), dev)
    _check(topk_ids, "topk_ids", torch.int64, (T, k), dev)
    _check(topk_weights, "topk_weights", torch.float32, (T, k), dev)
    _check_e4m3(w13, "w13", (E, two, H), dev)
    _check_e4m3(w2, "w2", (E, H, I), dev)
    if isinstance(w13_scale, torch.Tensor) and w13_scale.dim() == 4:
        if I % 128:
            raise ValueError(f"w13_scale [E,2,ceil(I/128),...] needs I % 128 == 0 (I = {I}): see moe_fp8_pad_inner")
        _check(w13_scale, "w13_scale", torch.float32, (E, 2, _blocks(I), _blocks(H)), dev)
    else:
        _check(w13_scale, "w13_scale", torch.float32, (E, _blocks(two), _blocks(H)), dev)
    _check(w2_scale, "w2_scale", torch.float32, (E, _blocks(H), _blocks(I)), dev)
    ws = _check_ws(ws, lambda: moe_fp8_layer_workspace_bytes(T, k, H, I, E), dev)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    else:
        _check(y, "y", torch.bfloat16, (T, H), dev)
    _call("moe_fp8_layer", dev, x.data_ptr(), topk_ids.data_ptr(), topk_weights.data_ptr(), T, k, E, H, I,
          w13.data_ptr(), w13_scale.data_ptr(), w2.data_ptr(), w2_scale.data_ptr(), ws.data_ptr(), ws.numel(),
          y.data_ptr())
    return y


def _rms_norm(name, x, weight, eps, residual, want_y, q, scale, residual_out, y, q_dtype, s_dtype, s_cols):
    M, K = _dims(x, "x", 2)
    dev, device = x.get_device(), x.device
    if not (dev >= 0 and x.dtype is _BF16 and x.is_contiguous()):
        _check(x, "x", _BF16, (M, K), dev)
    f32 = isinstance(weight, _Tensor) and weight.dtype is _F32  # (a Parameter too)
    _check(weight, "weight", _F32 if f32 else _BF16, (K,), dev)
    r_ptr = out_ptr = y_ptr = None
    if residual is not None:
        _check(residual, "residual", _BF16, (M, K), dev)
        r_ptr = residual.data_ptr()
        if residual_out is None:
            residual_out = _empty_like(residual)
        else:
            _check(residual_out, "residual_out", _BF16, (M, K), dev)
        out_ptr = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if y is not None:
        _check(y, "y", _BF16, (M, K), dev)
        y_ptr = y.data_ptr()
    elif want_y:
        y = _empty_like(x)
        y_ptr = y.data_ptr()
    if q is None:
        q = _empty_like(x, dtype=q_dtype)
    elif q_dtype is _E4M3:
        _check_e4m3(q, "q", (M, K), dev)
    else:
        _check(q, "q", q_dtype, (M, K), dev)
    shape = (M,) if s_cols == 0 else (M, (K + s_cols - 1) // s_cols)
    if scale is None:
        scale = _empty(shape, dtype=s_dtype, device=device)
    else:
        _check(scale, "scale", s_dtype, shape, dev)
    _call(name, dev, x.data_ptr(), r_ptr, weight.data_ptr(), M, K, eps, 1 if f32 else 0, out_ptr, y_ptr, q.data_ptr(),
          scale.data_ptr())
    return q, scale, residual_out, y


def w8a8_rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                        residual: Optional[torch.Tensor] = None, want_y: bool = False,
                        q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                        residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """Root-mean-square norm of bf16 x [M,K] (+ residual [M,K]) with weight [K] (bf16 or float32), quantised:
    (int8 q [M,K], float32 scale [M], r, y).

    r = bf16(x + residual), or None without a residual; the norm is of r.  y: the norm in bf16 where want_y (or a
    tensor `y`) asks for it, else None.  residual_out may be x or residual itself: the residual stream in place."""
    return _rms_norm("w8a8_rms_norm_quant", x, weight, eps, residual, want_y, q, scale, residual_out, y, torch.int8,
                     _F32, 0)


def w8a8_fp8_rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                            residual: Optional[torch.Tensor] = None, want_y: bool = False,
                            q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                            residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """w8a8_rms_norm_quant with block-scaled FP8 codes: (float8_e4m3fn q [M,K], float32 scale [M, ceil(K/128)], r, y),
    the operands of w8a8_fp8_matmul."""
    return _rms_norm("w8a8_fp8_rms_norm_quant", x, weight, eps, residual, want_y, q, scale, residual_out, y, _E4M3,
                     _F32, 128)


def w8a8_mx_rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                           residual: Optional[torch.Tensor] = None, want_y: bool = False,
                           q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                           residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """w8a8_rms_norm_quant with MXFP8 codes (K % 32 == 0): (uint8 E4M3 codes q [M,K], uint8 E8M0 scales [M,K/32], r, y),
    the operands of w8a8_mx_matmul."""
    return _rms_norm("w8a8_mx_rms_norm_quant", x, weight, eps, residual, want_y, q, scale, residual_out, y,
                     torch.uint8, torch.uint8, 32)


def _activation(name: str) -> int:
    act = _capi.ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(map(repr, _capi.ACTIVATIONS))}, got {name!r}")
    return act


def _out_dtype(dtype, y):
    if y is not None:
        dtype = y.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"y must be {_BF16} or {_F32}, got {dtype}")
    return dtype


def bf16_matmul_workspace_bytes(M: int, N: int, K: int) -> int:
    """The bytes of a workspace for every w8a8_bf16_matmul of at most M rows to at most N channels, whatever its K."""
    return _size("w8a8_bf16_matmul_workspace_bytes", M, N, K)


def w8a8_bf16_matmul(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: str = "none",
                     residual: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                     ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """bf16 x [M,K] x bf16 w [N,K] -> y [M,N] = activation(x w^T + bias) (+ residual), bf16 or float32.

    activation: "none", "relu", "silu", "gelu", "gelu_tanh", or "swiglu" with w [2N,K] (the gate's rows, then the up
    projection's; bias [2N]): silu(gate) * up.  bias bf16 [rows of w], residual bf16 [M,N] (y itself is allowed).  The
    layers that a quantised model keeps in bf16; with out_dtype float32 the router's logits.  Keep a workspace (`ws`)
    over calls, one for the largest batch serves the smaller ones: without one every call zeroes its own."""
    M, K = _dims(x, "x", 2)
    rows = _dims(w, "w", 2)[0]
    dev, act = x.get_device(), _activation(activation)
    if not (dev >= 0 and x.dtype is _BF16 and type(w) is _Tensor and w.dtype is _BF16 and w.get_device() == dev
            and w.shape[1] == K and x.is_contiguous() and w.is_contiguous()):
        _check(x, "x", _BF16, (M, K), dev)
        _check(w, "w", _BF16, (rows, K), dev)
    N = rows
    if act == 5:
        if rows % 2:
            raise ValueError("w must be [2N,K] for 'swiglu'")
        N = rows // 2
    if bias is not None:
        _check(bias, "bias", _BF16, (rows,), dev)
    if residual is not None:
        _check(residual, "residual", _BF16, (M, N), dev)
    if ws is None:  # what this call needs, of which only the status word and the counters have to be zero
        ws = _empty(max(_size("w8a8_bf16_matmul_call_bytes", M, N, K, act), 256), dtype=torch.uint8, device=x.device)
        (ws[:_capi.BF16_ZERO_BYTES] if ws.numel() > _capi.BF16_ZERO_BYTES else ws).zero_()
    else:
        _check_ws(ws, None, dev)
    out_dtype = _out_dtype(out_dtype, y)
    if y is None:
        y = _empty((M, N), dtype=out_dtype, device=x.device)
    else:
        _check(y, "y", out_dtype, (M, N), dev)
    _call("w8a8_bf16_matmul", dev, x.data_ptr(), M, K, w.data_ptr(), N, None if bias is None else bias.data_ptr(), act,
          None if residual is None else residual.data_ptr(), 0 if out_dtype is _BF16 else _capi.MM_F32, y.data_ptr(),
          ws.data_ptr(), ws.numel())
    return y


def bf16_grouped_matmul_workspace_bytes(E: int, R: int, N: int, K: int) -> int:
    return _size("w8a8_bf16_grouped_matmul_workspace_bytes", E, R, N, K)


def w8a8_bf16_grouped_matmul(x: torch.Tensor, group_list: torch.Tensor, w: torch.Tensor,
                             bias: Optional[torch.Tensor] = None, activation: str = "none",
                             out_dtype: torch.dtype = torch.bfloat16, ws: Optional[torch.Tensor] = None,
                             y: Optional[torch.Tensor] = None):
    """w8a8_bf16_matmul for rows grouped by expert: bf16 x [R,K], int64 group_list [E] (rows of every expert), bf16
    w [E,N,K] ("swiglu": [E,2N,K]), bf16 bias [E, rows of w] -> y [R,N].  A group list that does not fit R leaves y as
    it was (read_device_status)."""
    R, K = _dims(x, "x", 2)
    E, rows, K2 = _dims(w, "w", 3)
    dev, act = x.get_device(), _activation(activation)
    if not (dev >= 0 and x.dtype is _BF16 and type(w) is _Tensor and w.dtype is _BF16 and w.get_device() == dev
            and K2 == K and x.is_contiguous() and w.is_contiguous()):
        _check(x, "x", _BF16, (R, K), dev)
        _check(w, "w", _BF16, (E, rows, K), dev)
    _check(group_list, "group_list", _I64, (E,), dev)
    N = rows
    if act == 5:
        if rows % 2:
            raise ValueError("w must be [E,2N,K] for 'swiglu'")
        N = rows // 2
    if bias is not None:
        _check(bias, "bias", _BF16, (E, rows), dev)
    ws = _check_ws(ws, lambda: bf16_grouped_matmul_workspace_bytes(E, R, N, K), dev)
    out_dtype = _out_dtype(out_dtype, y)
    if y is None:
        y = _empty((R, N), dtype=out_dtype, device=x.device)
    else:
        _check(y, "y", out_dtype, (R, N), dev)
    _call("w8a8_bf16_grouped_matmul", dev, x.data_ptr(), group_list.data_ptr(), E, R, K, w.data_ptr(), N,
          None if bias is None else bias.data_ptr(), act, 0 if out_dtype is _BF16 else _capi.MM_F32, y.data_ptr(),
          ws.data_ptr(), ws.numel())
    return y


def read_device_status(ws: torch.Tensor) -> int:
    """Synchronise the current stream and return (and clear) the device status word of `ws`."""
    with torch.cuda.device(ws.device):
        return int(_capi.lib().w8a8_read_device_status(ws.data_ptr(), _stream(ws.device)))


ENGINE_NONE, ENGINE_WARP, ENGINE_DECODE, ENGINE_TC, ENGINE_TC_I8 = 0, 1, 2, 3, 4


def last_engine() -> int:
    """Engine the calling thread's last contraction ran on (ENGINE_WARP / ENGINE_DECODE / ENGINE_TC /
    ENGINE_TC_I8)."""
    return int(_capi.lib().w8a8_last_engine())
