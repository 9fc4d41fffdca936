"""Measured cases of the norm that feeds the quantised layers and of the bf16 products beside them.

Three operators, each in its plain form (elementary torch operations in 32 bits, sums of squares in 64) and, with `own`
set, as a user calls the library:

  norm     bf16 rows (+ residual) -> root-mean-square norm -> 8-bit codes with scales, in the three layouts that the
           quantised products take: int8 with a scale a row, E4M3 with a scale per 128 values, E4M3 with a power of two
           per 32; and the residual's sum, and the norm itself in bf16
  linear   bf16 rows x bf16 weight -> bias -> activation -> residual -> bf16 or fp32
  grouped  the same product for rows grouped by expert, each expert with its own weight

A case is a dict of plain values; inputs come from the seed alone (rows per expert from the case alone, so that
what a pass has to read is known without them).
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    return [
        # one token in a chat: the first norm of a layer, nothing but latency
        dict(name="norm int8 token", op="norm", form="int8", M=1, H=4096, residual=False, y=False, weight="bfloat16"),
        # a decode batch before an expert layer: codes for the experts, the bf16 row for the router
        dict(name="norm fp8 decode", op="norm", form="fp8", M=64, H=7168, residual=True, y=True, weight="bfloat16"),
        # a ragged batch in the layout with powers of two as scales, the norm's weight kept in fp32
        dict(name="norm mx odd", op="norm", form="mx", M=1021, H=1504, residual=True, y=False, weight="float32"),
        # a prefill step, bound by memory
        dict(name="norm int8 prefill", op="norm", form="int8", M=8192, H=4096, residual=True, y=False,
             weight="bfloat16"),
        # one token through an output projection, added to the residual stream: the weight stream is the cost
        dict(name="linear token", op="linear", M=1, N=7168, K=2048, act="none", bias=False, residual=True,
             out="bfloat16"),
        # a decode batch's router logits
        dict(name="linear router", op="linear", M=128, N=256, K=7168, act="none", bias=False, residual=False,
             out="float32"),
        # a decode batch through a layer with bias and residual
        dict(name="linear decode", op="linear", M=64, N=2048, K=7168, act="none", bias=True, residual=True,
             out="bfloat16"),
        # a gated unit's first product with sizes that end inside tiles
        dict(name="linear odd", op="linear", M=1141, N=1416, K=2000, act="swiglu", bias=True, residual=True,
             out="bfloat16"),
        # a prefill step's first product of a feed-forward block, bound by the tensor cores
        dict(name="linear prefill", op="linear", M=8192, N=14336, K=4096, act="gelu_tanh", bias=True, residual=False,
             out="bfloat16"),
        # a small expert layer with ragged groups and empty experts
        dict(name="grouped small odd", op="grouped", T=53, topk=2, E=8, N=1416, K=2000, act="none", bias=True,
             routing="zipf", dead=2),
        # the gated first product of a decode step over many experts, about sixteen rows each
        dict(name="grouped decode", op="grouped", T=128, topk=8, E=64, N=2048, K=7168, act="swiglu", bias=False,
             routing="uniform", dead=0),
        # the gated first product of a prefill step, experts of very different popularity
        dict(name="grouped prefill", op="grouped", T=4096, topk=8, E=64, N=2048, K=4096, act="swiglu", bias=False,
             routing="zipf", dead=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "grouped"])
    if op == "norm":
        form = rng.choice(["int8", "fp8", "mx"])
        H = (32 if form == "mx" else 16) * _log(rng, 8, 256)
        return dict(op=op, form=form, M=_log(rng, 1, max(1, min(16384, 8192 * 4096 // H))), H=H,
                    residual=rng.random() < 0.7, y=rng.random() < 0.4, weight=rng.choice(["bfloat16", "float32"]))
    act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh", "swiglu", "swiglu"])
    rows = 2 if act == "swiglu" else 1  # weight rows per output channel
    if op == "linear":
        N, K = _log(rng, 64, 14336 // rows), 16 * _log(rng, 8, 448)
        return dict(op=op, M=_log(rng, 1, max(1, min(8192, 8192 * 14336 * 4096 // (rows * N * K)))), N=N, K=K, act=act,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5, out=rng.choice(["bfloat16", "bfloat16", "float32"]))
    E = rng.choice([4, 8, 16, 32, 64])
    N, K = _log(rng, 64, 4096 // rows), 16 * _log(rng, 8, 256)
    topk = rng.choice([1, 2, 4, min(8, E - 1)])
    return dict(op=op, T=_log(rng, 1, 4096), topk=topk, E=E, N=N, K=K, act=act, bias=rng.random() < 0.3,
                routing=rng.choice(["zipf", "uniform"]), dead=rng.randint(0, (E - topk) // 4))


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _activations(g, rows, K):
    """N(0,1) rows with a few outlier columns, as bf16."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    cols = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 200)]
    x[:, cols] *= 20.0
    return x.to(torch.bfloat16)


def _weight(g, N, K):
    return (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)


def _rows_per_expert(case):
    """Rows of every expert: each of T tokens picks topk distinct experts; from the case alone."""
    E, T, topk, dead = case["E"], case["T"], case["topk"], case["dead"]
    r = random.Random("%d %d %d %s %d" % (E, T, topk, case["routing"], dead))
    weight = [0.0 if i >= E - dead else (i + 1) ** -1.1 if case["routing"] == "zipf" else 1.0 for i in range(E)]
    r.shuffle(weight)
    counts = [0] * E
    for _ in range(T):
        keys = sorted(((math.log(r.random() + 1e-300) / weight[e] if weight[e] else -math.inf), e) for e in range(E))
        for _, e in keys[-topk:]:
            counts[e] += 1
    return counts


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "norm":
        M, H = case["M"], case["H"]
        st["x"] = _activations(g, M, H)
        # the residual stream: rows of very different size
        size = torch.exp2(torch.randint(-3, 4, (M, 1), generator=g, device="cuda").float())
        st["residual"] = (torch.randn(M, H, generator=g, device="cuda") * size).to(torch.bfloat16) \
            if case["residual"] else None
        st["weight"] = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(getattr(torch, case["weight"]))
        return st
    N, K = case["N"], case["K"]
    rows = 2 * N if case["act"] == "swiglu" else N
    if op == "linear":
        M = case["M"]
        st["x"], st["w"] = _activations(g, M, K), _weight(g, rows, K)
        st["bias"] = (torch.randn(rows, generator=g, device="cuda") * 0.1).to(torch.bfloat16) if case["bias"] else None
        st["residual"] = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16) if case["residual"] else None
        return st
    E, counts = case["E"], _rows_per_expert(case)
    st["x"] = _activations(g, sum(counts), K)
    st["w"] = torch.empty(E, rows, K, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        st["w"][e] = _weight(g, rows, K)
    st["bias"] = (torch.randn(E, rows, generator=g, device="cuda") * 0.1).to(torch.bfloat16) if case["bias"] else None
    st["group_list"] = torch.tensor(counts, dtype=torch.int64, device="cuda")
    st["most"] = max(counts)  # the host made the list: it knows the longest group
    return st


# ------------------------------------------------------------------ the plain forms


def _codes_plain(v, group, top):
    """fp32 [M,H] in groups of `group` values -> v / s as fp32 [M,G,group] and the scales s = max|v| / top [M,G]."""
    M, H = v.shape
    G = -(-H // group)
    if H % group:
        v = torch.nn.functional.pad(v, (0, G * group - H))
    v = v.view(M, G, group)
    s = v.abs().amax(2) / torch.full((), top, device=v.device)  # by a tensor: a true quotient
    return torch.where(s[:, :, None] > 0, v / s[:, :, None], 0.0), s


def _norm_plain(x, residual, weight, form, want_y):
    M, H = x.shape
    r = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    total = r.double().square().sum(1, keepdim=True).float()
    g = torch.rsqrt((total / torch.full((), float(H), device=x.device) + EPS).double()).float()
    v = r.float() * g * weight.float()
    if form == "int8":
        q, s = _codes_plain(v, H, 127.0)
        q, s = q.round().clamp(-127, 127).to(torch.int8).view(M, H), s[:, 0]
    elif form == "fp8":
        q, s = _codes_plain(v, 128, E4M3_MAX)
        q = q.to(torch.float8_e4m3fn).view(M, -1)[:, :H].contiguous()
    else:
        b = v.view(M, H // 32, 32)
        amax = b.abs().amax(2)
        e = (torch.frexp(amax).exponent - 1 - 8).clamp(-127, 127)
        q = (b.double() * torch.exp2(-e.double())[:, :, None]).float().clamp(-E4M3_MAX, E4M3_MAX)
        q = q.to(torch.float8_e4m3fn).view(M, H)
        s = torch.where(amax > 0, e + 127, 0).to(torch.uint8).view(torch.float8_e8m0fnu)
    return q, s, None if residual is None else r, v.to(torch.bfloat16) if want_y else None


def _act_plain(v, act):
    if act == "swiglu":
        gate, up = v.chunk(2, -1)
        return gate / (1.0 + torch.exp(-gate)) * up
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -(0.5 ** 0.5))
    if act == "gelu_tanh":  # 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
        return v / (1.0 + torch.exp(-2.0 * (2.0 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    return v


def _linear_plain(x, w, bias, act, residual, out):
    v = x.float() @ w.float().t()
    if bias is not None:
        v = v + bias.float()
    v = _act_plain(v, act)
    return (v if residual is None else v + residual.float()).to(out)


def _grouped_plain(x, group_list, most, w, bias, act):
    R, E = x.shape[0], w.shape[0]
    start = group_list.cumsum(0) - group_list
    slot = torch.arange(most, device=x.device)
    row = (start[:, None] + slot).clamp(max=R - 1)  # [E, most]; places past an expert's rows are dropped below
    v = torch.bmm(x.float()[row], w.float().transpose(1, 2))
    if bias is not None:
        v = v + bias.float()[:, None]
    expert = torch.repeat_interleave(torch.arange(E, device=x.device), group_list, output_size=R)
    return _act_plain(v[expert, torch.arange(R, device=x.device) - start[expert]], act).to(torch.bfloat16)


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import w8a8_dynamic_quant_gb300 as W
        if op == "norm":
            f = {"int8": W.w8a8_rms_norm_quant, "fp8": W.w8a8_fp8_rms_norm_quant, "mx": W.w8a8_mx_rms_norm_quant}[c["form"]]
            q, s, r, y = f(st["x"], st["weight"], EPS, residual=st["residual"], want_y=c["y"])
            if c["form"] == "mx":  # bytes: the values that they stand for
                q, s = q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)
            return q, s, r, y
        if op == "linear":
            if "work" not in st:  # the workspace that a program keeps beside its weight
                st["work"] = W.workspace(W.bf16_matmul_workspace_bytes(c["M"], c["N"], c["K"]))
            return W.w8a8_bf16_matmul(st["x"], st["w"], bias=st["bias"], activation=c["act"], residual=st["residual"],
                                      out_dtype=getattr(torch, c["out"]), ws=st["work"])
        if "work" not in st:
            st["work"] = W.workspace(W.bf16_grouped_matmul_workspace_bytes(c["E"], st["x"].shape[0], c["N"], c["K"]))
        return W.w8a8_bf16_grouped_matmul(st["x"], st["group_list"], st["w"], bias=st["bias"], activation=c["act"],
                                          ws=st["work"])
    if op == "norm":
        return _norm_plain(st["x"], st["residual"], st["weight"], c["form"], c["y"])
    if op == "linear":
        return _linear_plain(st["x"], st["w"], st["bias"], c["act"], st["residual"], getattr(torch, c["out"]))
    return _grouped_plain(st["x"], st["group_list"], st["most"], st["w"], st["bias"], c["act"])


# ------------------------------------------------------------------ the definition in 64 bits


def _e4m3_nearest(v):
    """Nearest E4M3 value, ties to even, saturating at 448, of float64 values."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(st, c):
    r, H = st["x"], c["H"]
    total = None
    if st["residual"] is not None:
        total = r.double() + st["residual"].double()
        r = total.float().to(torch.bfloat16)  # the stream's type: what the norm sees
    r = r.double()
    v = r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * st["weight"].double()
    y = v if c["y"] else None
    if c["form"] == "int8":
        return None, v.abs().amax(1) / 127.0, total, y
    width = 128 if c["form"] == "fp8" else 32
    q, scales = torch.empty_like(v), []
    for b in range(0, H, width):
        part = v[:, b:b + width]
        top = part.abs().amax(1, keepdim=True)
        if c["form"] == "fp8":
            s = top / E4M3_MAX
        else:
            s = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -119))) - 8)
        q[:, b:b + width] = _e4m3_nearest(part / torch.where(s > 0, s, 1.0))
        scales.append(s)
    return q, torch.cat(scales, 1), total, y


def _exact_act(v, act):
    if act == "swiglu":
        n = v.shape[1] // 2
        return v[:, :n] * torch.sigmoid(v[:, :n]) * v[:, n:]
    if act == "relu":
        return torch.maximum(v, torch.zeros_like(v))
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def exact(case, seed):
    if work(case)["flops"] > 1e13:
        return None
    st, op = prepare(case, seed), case["op"]
    if op == "norm":
        return _exact_norm(st, case)
    if op == "linear":
        v = st["x"].double() @ st["w"].double().t()
        if st["bias"] is not None:
            v += st["bias"].double()
        v = _exact_act(v, case["act"])
        return v if st["residual"] is None else v + st["residual"].double()
    out, at = [], 0
    for e, n in enumerate(st["group_list"].tolist()):
        if n:
            v = st["x"][at:at + n].double() @ st["w"][e].double().t()
            if st["bias"] is not None:
                v += st["bias"][e].double()
            out.append(_exact_act(v, case["act"]))
        at += n
    return torch.cat(out)


def work(case):
    op = case["op"]
    if op == "norm":
        M, H = case["M"], case["H"]
        scales = {"int8": 4, "fp8": 4 * -(-H // 128), "mx": H // 32}[case["form"]]
        a_value = 3 + (4 if case["residual"] else 0) + (2 if case["y"] else 0)
        return {"bytes": M * (a_value * H + scales) + H * (2 if case["weight"] == "bfloat16" else 4), "flops": 8 * M * H}
    N, K = case["N"], case["K"]
    rows = 2 * N if case["act"] == "swiglu" else N
    weight = 2 * rows * K + (2 * rows if case["bias"] else 0)
    if op == "linear":
        M = case["M"]
        size = 4 if case["out"] == "float32" else 2
        return {"bytes": 2 * M * K + weight + M * N * (size + (2 if case["residual"] else 0)), "flops": 2 * M * rows * K}
    counts = _rows_per_expert(case)
    R = sum(counts)
    return {"bytes": 2 * R * K + sum(1 for n in counts if n) * weight + 8 * case["E"] + 2 * R * N,
            "flops": 2 * R * rows * K}
