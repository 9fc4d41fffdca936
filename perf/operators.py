"""Measured cases of the block-scaled FP8 operators and of the expert router.

Five operators, each in its plain form (elementary torch operations in 32 bits) and, with `own` set, as a
user calls the library:

  gate      router logits [T,E] -> the k chosen experts of every token and their weights
  quant     bf16 rows -> E4M3 codes with one fp32 scale per 128 values
  swiglu    bf16 [R,2I] (gate half, up half) -> SwiGLU -> E4M3 codes with one fp32 scale per 128 values
  dense     E4M3 rows x E4M3 weight with a scale per 128 values of a row and per 128 x 128 weight block -> bf16
  grouped   the same contraction for rows grouped by expert, each expert with its own weight

A case is a dict of plain values; inputs come from the seed alone (rows per expert from the case alone, so that
what a pass has to read is known without them).
"""
import math
import random

import torch

own = False

BLOCK = 128  # values that share a scale
E4M3_MAX = 448.0


def listed():
    return [
        # a decode batch through a large router: sigmoid scores, a balance bias, 8 groups of which 4 are kept
        dict(name="gate decode", op="gate", T=128, E=256, k=8, scoring="sigmoid", bias=True, n_group=8, topk_group=4,
             group_score="top2", renorm=True, scale=2.5, dtype="float32", masked=False),
        # a prefill batch: softmax over 64 experts from bf16 logits, ties and masked experts among them
        dict(name="gate prefill", op="gate", T=16384, E=64, k=8, scoring="softmax", bias=False, n_group=1, topk_group=1,
             group_score="max", renorm=True, scale=1.0, dtype="bfloat16", masked=True),
        # activations of a decode step, latency-bound
        dict(name="quant decode", op="quant", M=64, K=7168),
        # activations of a prefill step, bound by memory
        dict(name="quant prefill", op="quant", M=8192, K=4096),
        # between the two expert products of a decode step, an inner size that is no multiple of 128
        dict(name="swiglu decode odd", op="swiglu", R=1021, I=1392),
        # between the two expert products of a prefill step
        dict(name="swiglu prefill", op="swiglu", R=32768, I=2048),
        # the smallest linear layer, latency-bound, with a bias
        dict(name="dense tiny", op="dense", M=16, N=256, K=512, bias=True),
        # a decode step's linear layer: the weight stream is the cost
        dict(name="dense decode", op="dense", M=64, N=2048, K=7168, bias=False),
        # a prefill step's linear layer, bound by the tensor cores
        dict(name="dense prefill", op="dense", M=8192, N=14336, K=4096, bias=False),
        # a small expert layer with ragged groups, empty experts, and N, K that end inside a block
        dict(name="grouped small odd", op="grouped", T=53, topk=2, E=8, N=1416, K=2000, routing="zipf", dead=2),
        # the up projection of a decode step over many experts: about four rows an expert
        dict(name="grouped decode", op="grouped", T=128, topk=8, E=256, N=4096, K=7168, routing="uniform", dead=0),
        # the up projection of a prefill step, experts of very different popularity
        dict(name="grouped prefill", op="grouped", T=4096, topk=8, E=64, N=4096, K=4096, routing="zipf", dead=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "quant", "swiglu", "dense", "grouped"])
    if op == "gate":
        E = rng.choice([8, 16, 40, 60, 64, 96, 128, 160, 256, 384, 512])
        n_group = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        topk_group = rng.randint(1, n_group)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(8, topk_group * (E // n_group))),
                    scoring=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5, n_group=n_group,
                    topk_group=topk_group, group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice(["float32", "bfloat16"]),
                    masked=rng.random() < 0.5)
    if op == "quant":
        K = 16 * _log(rng, 16, 512)
        return dict(op=op, M=_log(rng, 1, max(1, min(16384, 8192 * 4096 // K))), K=K)
    if op == "swiglu":
        inner = 16 * _log(rng, 8, 256)
        return dict(op=op, R=_log(rng, 1, max(1, min(32768, 32768 * 2048 // inner))), I=inner)
    if op == "dense":
        N, K = _log(rng, 128, 14336), 16 * _log(rng, 16, 448)
        return dict(op=op, M=_log(rng, 1, max(1, min(8192, 8192 * 14336 * 4096 // (N * K)))), N=N, K=K,
                    bias=rng.random() < 0.5)
    E = rng.choice([4, 8, 16, 32, 64, 128])
    N, K = _log(rng, 256, 4096), 16 * _log(rng, 16, 256)
    topk = rng.choice([1, 2, 4, min(8, E - 1)])
    routing = rng.choice(["zipf", "uniform"])
    return dict(op=op, T=_log(rng, 1, 4096), topk=topk, E=E, N=N, K=K, routing=routing,
                dead=rng.randint(0, (E - topk) // 4))


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _quantise(v, rows):
    """v [A,K] fp32 -> (E4M3 [A,K], scales [ceil(A/rows), ceil(K/128)]): blocks of `rows` x 128."""
    A, K = v.shape
    ab, kb = -(-A // rows), -(-K // BLOCK)
    p = torch.nn.functional.pad(v, (0, kb * BLOCK - K, 0, ab * rows - A)).view(ab, rows, kb, BLOCK)
    s = p.abs().amax(dim=(1, 3)) / E4M3_MAX
    q = torch.where(s[:, None, :, None] > 0, p / s[:, None, :, None], torch.zeros_like(p))
    q = q.to(torch.float8_e4m3fn).view(ab * rows, kb * BLOCK)[:A, :K].contiguous()
    return q, s.contiguous()


def _activations(g, rows, K):
    """N(0,1) rows with a few outlier columns, as bf16."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    cols = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 200)]
    x[:, cols] *= 20.0
    return x.to(torch.bfloat16)


def _weight(g, N, K):
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    kb = -(-K // BLOCK)
    spread = torch.exp2(torch.randint(-2, 3, (1, kb), generator=g, device="cuda").float())
    return w * spread.repeat_interleave(BLOCK, 1)[:, :K]


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
    if op == "gate":
        T, E = case["T"], case["E"]
        x = torch.randn(T, E, generator=g, device="cuda") * 1.5 + torch.randn(1, E, generator=g, device="cuda") * 0.5
        if case["masked"]:
            x = x.masked_fill(torch.rand(T, E, generator=g, device="cuda") < 0.05, -math.inf)
            if T > 3:
                x[T // 2] = -math.inf  # a padding row: no expert left
        st["logits"] = x.to(getattr(torch, case["dtype"]))
        st["bias"] = torch.randn(E, generator=g, device="cuda") * (0.05 if case["scoring"] == "sigmoid" else 0.002) \
            if case["bias"] else None
    elif op == "quant":
        st["x"] = _activations(g, case["M"], case["K"])
    elif op == "swiglu":
        st["y13"] = (torch.randn(case["R"], 2 * case["I"], generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    elif op == "dense":
        M, N, K = case["M"], case["N"], case["K"]
        st["q"], st["xs"] = _quantise(_activations(g, M, K).float(), 1)
        st["w"], st["ws"] = _quantise(_weight(g, N, K), BLOCK)
        st["bias"] = (torch.randn(N, generator=g, device="cuda") * 0.1).to(torch.bfloat16) if case["bias"] else None
    else:
        E, N, K = case["E"], case["N"], case["K"]
        counts = _rows_per_expert(case)
        st["q"], st["xs"] = _quantise(_activations(g, sum(counts), K).float(), 1)
        st["w"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        st["ws"] = torch.empty(E, -(-N // BLOCK), -(-K // BLOCK), device="cuda")
        for e in range(E):
            st["w"][e], st["ws"][e] = _quantise(_weight(g, N, K), BLOCK)
        st["group_list"] = torch.tensor(counts, dtype=torch.int64, device="cuda")
        st["most"] = max(counts)  # the host made the list: it knows the longest group
    return st


# ------------------------------------------------------------------ the plain forms


def _gate_plain(logits, k, bias, scoring, n_group, topk_group, group_score, renorm, scale):
    T, E = logits.shape
    x = logits.float()
    live = x > -math.inf  # masked experts: -inf or NaN
    if scoring == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
        key = s if bias is None else s + bias
    else:
        m = torch.where(live, x, -math.inf).amax(1, keepdim=True)
        s = torch.where(x == m, 1.0, torch.exp(x - m))
        s = torch.where(live, s, 0.0)
        key = s  # in the order of the probabilities
        total = s.sum(1, keepdim=True, dtype=torch.float64).float()
        if bias is not None:
            key = s / total + bias
    key = torch.where(live & (key > -math.inf), key, -math.inf)
    gs = E // n_group
    ids = torch.arange(E, device=x.device).expand(T, E)
    if topk_group < n_group:
        two = key.view(T, n_group, gs).sort(dim=2, descending=True, stable=True).values
        gscore = two[:, :, 0]
        if group_score == "top2":
            gscore = gscore + torch.where(two[:, :, 1] > -math.inf, two[:, :, 1], 0.0)
        keep = gscore.sort(dim=1, descending=True, stable=True).indices[:, :topk_group].sort(1).values
        ids = (keep[:, :, None] * gs + torch.arange(gs, device=x.device)).reshape(T, topk_group * gs)
    top, at = key.gather(1, ids).sort(dim=1, descending=True, stable=True)
    ids = ids.gather(1, at[:, :k])
    w = torch.where(top[:, :k] > -math.inf, s.gather(1, ids), 0.0)
    if renorm:
        d = w.sum(1, keepdim=True)
        w = torch.where(d > 0, w / d, 0.0)
    elif scoring == "softmax":
        w = torch.where(total > 0, w / total, 0.0)
    return ids, w * scale


def _codes_plain(v):
    """fp32 [M,K] -> E4M3 codes and a scale per 128 values of a row."""
    M, K = v.shape
    kb = -(-K // BLOCK)
    if K % BLOCK:
        v = torch.nn.functional.pad(v, (0, kb * BLOCK - K))
    v = v.view(M, kb, BLOCK)
    s = v.abs().amax(2) / E4M3_MAX
    q = torch.where(s[:, :, None] > 0, v / s[:, :, None], 0.0).to(torch.float8_e4m3fn)
    return q.view(M, kb * BLOCK)[:, :K].contiguous(), s


def _wide(q, s):
    """The values that codes [A,K] with scales [A,K/128] stand for, in fp32."""
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _wide_weight(w, s):
    return _wide(w, s.repeat_interleave(BLOCK, -2)[..., : w.shape[-2], :])


def _grouped_plain(q, xs, group_list, most, w, ws):
    R, (E, N, K) = q.shape[0], w.shape
    a = _wide(q, xs)
    start = group_list.cumsum(0) - group_list
    slot = torch.arange(most, device=q.device)
    row = (start[:, None] + slot).clamp(max=R - 1)  # [E, most]; places past an expert's rows are dropped below
    y = torch.bmm(a[row], _wide_weight(w, ws).transpose(1, 2))
    expert = torch.repeat_interleave(torch.arange(E, device=q.device), group_list, output_size=R)
    return y[expert, torch.arange(R, device=q.device) - start[expert]].to(torch.bfloat16)


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import w8a8_dynamic_quant_gb300 as W
        if op == "gate":
            return W.moe_gate_topk(st["logits"], c["k"], bias=st["bias"], scoring=c["scoring"], n_group=c["n_group"],
                                   topk_group=c["topk_group"], group_score=c["group_score"], renormalize=c["renorm"],
                                   routed_scale=c["scale"])
        if op == "quant":
            return W.w8a8_fp8_quant(st["x"])
        if op == "swiglu":
            return W.w8a8_fp8_swiglu_quant(st["y13"])
        if op == "dense":
            if "work" not in st:  # the workspace that a program keeps beside its weight
                st["work"] = W.workspace(W.fp8_matmul_workspace_bytes(c["M"], c["N"], c["K"]))
            return W.w8a8_fp8_matmul(st["q"], st["xs"], st["w"], st["ws"], bias=st["bias"], ws=st["work"])
        if "work" not in st:
            st["work"] = W.workspace(W.fp8_grouped_matmul_workspace_bytes(c["E"], st["q"].shape[0], c["N"], c["K"]))
        return W.w8a8_fp8_grouped_matmul(st["q"], st["xs"], st["group_list"], st["w"], st["ws"], ws=st["work"])
    if op == "gate":
        return _gate_plain(st["logits"], c["k"], st["bias"], c["scoring"], c["n_group"], c["topk_group"],
                           c["group_score"], c["renorm"], c["scale"])
    if op == "quant":
        return _codes_plain(st["x"].float())
    if op == "swiglu":
        gate, up = st["y13"].float().chunk(2, 1)
        return _codes_plain(gate * (1.0 / (1.0 + torch.exp(-gate))) * up)
    if op == "dense":
        y = _wide(st["q"], st["xs"]) @ _wide_weight(st["w"], st["ws"]).t()
        return (y if st["bias"] is None else y + st["bias"].float()).to(torch.bfloat16)
    return _grouped_plain(st["q"], st["xs"], st["group_list"], st["most"], st["w"], st["ws"])


# ------------------------------------------------------------------ the definition in 64 bits


def _e4m3_nearest(v):
    """Nearest E4M3 value, ties to even, of float64 values within +-448."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_codes(v):
    M, K = v.shape
    q, s = torch.zeros_like(v), torch.zeros(M, -(-K // BLOCK), dtype=v.dtype, device=v.device)
    for b in range(s.shape[1]):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        s[:, b] = part.abs().amax(1) / E4M3_MAX
        d = torch.where(s[:, b:b + 1] > 0, s[:, b:b + 1], 1.0)
        q[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3_nearest(part / d)
    return q, s


def _exact_gate(st, c):
    x = st["logits"].double()
    T, E = x.shape
    n_group, gs = c["n_group"], E // c["n_group"]
    off = ~(x > -math.inf)
    if c["scoring"] == "sigmoid":
        p = torch.sigmoid(x)
        p = torch.where(off, 0.0, p)
    else:
        p = torch.nan_to_num(torch.softmax(torch.where(off, -math.inf, x), 1), nan=0.0)
    rank = torch.where(off, -math.inf, p if st["bias"] is None else p + st["bias"].double())
    if c["topk_group"] < n_group:
        top = rank.view(T, n_group, gs).topk(2, 2).values
        if c["group_score"] == "top2":
            g = top[:, :, 0] + torch.where(top[:, :, 1] > -math.inf, top[:, :, 1], 0.0)
        else:
            g = top[:, :, 0]
        cut = torch.ones(T, n_group, dtype=torch.bool, device=x.device)
        cut.scatter_(1, torch.sort(g, dim=1, descending=True, stable=True).indices[:, : c["topk_group"]], False)
        rank = rank.masked_fill(cut.repeat_interleave(gs, 1), -math.inf)
    best, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    w = torch.where(best[:, : c["k"]] > -math.inf, p.gather(1, ids[:, : c["k"]]), 0.0)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    return None, w * c["scale"]


def _exact_product(q, xs, w, ws):
    """sum over blocks of 128 of the fp64 products of the codes, times both scales."""
    K = q.shape[1]
    a = q.double()
    b = w.double()
    for i in range(0, K, BLOCK):
        a[:, i:i + BLOCK] *= xs[:, i // BLOCK, None].double()
        b[:, i:i + BLOCK] *= ws[:, i // BLOCK].double().repeat_interleave(BLOCK)[: w.shape[0], None]
    return a @ b.t()


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "gate":
        return _exact_gate(st, case)
    if op == "quant":
        return _exact_codes(st["x"].double())
    if op == "swiglu":
        y = st["y13"].double()
        gate, up = y[:, : case["I"]], y[:, case["I"]:]
        return _exact_codes(gate * torch.sigmoid(gate) * up)
    if op == "dense":
        y = _exact_product(st["q"], st["xs"], st["w"], st["ws"])
        return y if st["bias"] is None else y + st["bias"].double()
    out, r = [], 0
    for e, n in enumerate(st["group_list"].tolist()):
        if n:
            out.append(_exact_product(st["q"][r:r + n], st["xs"][r:r + n], st["w"][e], st["ws"][e]))
        r += n
    return torch.cat(out)


def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * E * size + T * k * 12 + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    if op == "quant":
        M, K = case["M"], case["K"]
        return {"bytes": M * (3 * K + 4 * -(-K // BLOCK)), "flops": 3 * M * K}
    if op == "swiglu":
        R, inner = case["R"], case["I"]
        return {"bytes": R * (5 * inner + 4 * -(-inner // BLOCK)), "flops": 8 * R * inner}
    N, K = case["N"], case["K"]
    kb, weight = -(-K // BLOCK), N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK)
    if op == "dense":
        M = case["M"]
        return {"bytes": M * (K + 4 * kb) + weight + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    counts = _rows_per_expert(case)
    R = sum(counts)
    return {"bytes": R * (K + 4 * kb) + sum(1 for n in counts if n) * weight + 8 * case["E"] + 2 * R * N,
            "flops": 2 * R * N * K}
