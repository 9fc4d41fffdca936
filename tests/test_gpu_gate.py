"""Expert router against a plain 64-bit implementation: score functions, bias, groups, ties, masks, odd sizes.

Choices are compared exactly on inputs whose distinct keys are far enough apart (logits on a grid of 1/64 and
biases on a grid of 1/4096 leave keys that are equal or differ by much more than binary32 rounds), so that ties
occur and their order is part of the check."""
import numpy as np
import pytest
import torch

import w8a8_dynamic_quant_gb300 as W

pytestmark = pytest.mark.gpu


def reference(x, k, bias, scoring, n_group, topk_group, group_score, renorm, scale):
    """Loops over tokens in float64; keys rounded to 12 digits so that what is equal by the formula is equal."""
    T, E = x.shape
    gs = E // n_group
    ids = np.zeros((T, k), np.int64)
    wts = np.zeros((T, k))
    for t in range(T):
        l = x[t].astype(np.float64)
        live = l > -np.inf
        s = np.zeros(E)
        if scoring == "sigmoid":
            s[live] = 1.0 / (1.0 + np.exp(np.minimum(-l[live], 700.0)))
        elif live.any():
            m = l[live].max()
            e = np.where(l[live] == m, 1.0, np.exp(l[live] - m)) if np.isfinite(m) else (l[live] == m) * 1.0
            s[live] = e / e.sum()
        s[s < 2.0 ** -149] = 0.0  # scores are binary32
        key = np.round(s + (0.0 if bias is None else bias.astype(np.float64)), 12)
        key = np.where(live & (key > -np.inf), key, -np.inf)
        stays = np.ones(E, bool)
        if topk_group < n_group:
            g = np.sort(key.reshape(n_group, gs), 1)[:, ::-1]
            score = g[:, 0].copy()
            if group_score == "top2" and gs > 1:
                score = np.round(score + np.where(g[:, 1] > -np.inf, g[:, 1], 0.0), 12)
            keep = sorted(range(n_group), key=lambda i: (-score[i], i))[:topk_group]
            stays = np.isin(np.arange(E) // gs, keep)
        order = sorted(np.flatnonzero(stays), key=lambda i: (-key[i], i))[:k]
        ids[t] = order
        w = np.where(key[order] > -np.inf, s[order], 0.0)
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        wts[t] = w * scale
    return ids, wts


def logits(rng, T, E, masked):
    x = (rng.integers(-256, 257, (T, E)) / 64.0).astype(np.float32)
    if masked:
        x[rng.random((T, E)) < 0.2] = -np.inf
        x[rng.random((T, E)) < 0.05] = np.nan
        x[T // 2] = -np.inf             # a row with no expert left
        x[0, 1:] = -np.inf              # a row with one
    return x


def check(x, k, bias, scoring, n_group, topk_group, group_score, renorm, scale, dtype=torch.float32):
    xt = torch.from_numpy(x).to("cuda").to(dtype)
    bt = None if bias is None else torch.from_numpy(bias).to("cuda")
    ids, w = W.moe_gate_topk(xt, k, bias=bt, scoring=scoring, n_group=n_group, topk_group=topk_group,
                             group_score=group_score, renormalize=renorm, routed_scale=scale)
    ri, rw = reference(xt.float().cpu().numpy(), k, bias, scoring, n_group, topk_group, group_score, renorm, scale)
    assert ids.dtype == torch.int64 and w.dtype == torch.float32
    np.testing.assert_array_equal(ids.cpu().numpy(), ri)
    # a score is a handful of binary32 roundings (exp within 2 ulp, a sum, a quotient), the weight a sum of k <= 32
    # of them and a quotient: under 64 * 2^-24 of the weight
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=64 * 2.0 ** -24, atol=0)


CASES = [  # T, E, k, n_group, topk_group
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 31, 4, 1, 1), (5, 33, 8, 1, 1), (64, 64, 8, 1, 1), (7, 60, 6, 4, 2),
    (130, 256, 8, 8, 4), (9, 160, 6, 8, 3), (4, 384, 8, 1, 1), (6, 1000, 32, 8, 2), (3, 1024, 32, 32, 5),
    (2, 32, 3, 32, 7), (11, 40, 16, 2, 1),
]


@pytest.mark.parametrize("T,E,k,n_group,topk_group", CASES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_choice_and_weights(T, E, k, n_group, topk_group, scoring, biased):
    rng = np.random.default_rng(E * 7 + k + biased)
    bias = (rng.integers(-400, 401, E) / 4096.0).astype(np.float32) if biased else None
    for masked in (False, True):
        for group_score in ("max", "top2"):
            check(logits(rng, T, E, masked), k, bias, scoring, n_group, topk_group, group_score,
                  renorm=bool(rng.integers(2)), scale=float(rng.choice([1.0, 2.5])))


def test_bf16_logits_and_all_equal():
    rng = np.random.default_rng(5)
    check(logits(rng, 50, 128, True), 8, None, "softmax", 1, 1, "max", True, 1.0, torch.bfloat16)
    check(np.zeros((4, 96), np.float32), 8, None, "sigmoid", 8, 3, "top2", True, 1.0)  # every key ties
    check(np.full((2, 64), -np.inf, np.float32), 5, None, "softmax", 1, 1, "max", False, 1.0)


def test_extremes():
    x = np.zeros((4, 16), np.float32)
    x[0, 3], x[0, 9] = np.inf, np.inf
    x[1, 5] = 3.0e38
    x[2] = -3.0e38
    x[3] = -200.0
    for scoring in ("softmax", "sigmoid"):
        check(x, 4, None, scoring, 1, 1, "max", True, 1.0)
    bias = np.zeros(16, np.float32)
    bias[0], bias[2], bias[7] = -np.inf, np.nan, np.inf  # disabled, disabled, always first
    xt, bt = torch.from_numpy(x).cuda(), torch.from_numpy(bias).cuda()
    ids, w = W.moe_gate_topk(xt, 14, bias=bt, scoring="sigmoid")
    assert bool((ids[:, 0] == 7).all())
    assert not bool(((ids == 0) | (ids == 2)).any())
    ids, w = W.moe_gate_topk(xt, 16, bias=bt, scoring="sigmoid")
    assert ids[:, 14:].tolist() == [[0, 2]] * 4 and bool((w[:, 14:] == 0).all())


def test_softmax_sum_order_does_not_matter():
    """softmax with a bias on a million keys: the kernel's keys are binary32 with a correctly rounded sum, so the
    choice equals that of torch's binary32 operations with the sum taken in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(4096, 256, generator=g, device="cuda") * 2
    b = torch.randn(256, generator=g, device="cuda") * 0.002
    ids, _ = W.moe_gate_topk(x, 8, bias=b)
    e = torch.exp(x - x.amax(1, keepdim=True))
    key = e / e.sum(1, keepdim=True, dtype=torch.float64).float() + b
    assert torch.equal(ids, key.sort(dim=1, descending=True, stable=True).indices[:, :8])


@pytest.mark.parametrize("T,E,k,n_group,topk_group", [
    (2050, 64, 8, 1, 1), (2049, 32, 8, 8, 3), (2051, 60, 5, 1, 1), (2048, 8, 2, 1, 1), (2061, 64, 6, 4, 2),
    (2053, 60, 6, 4, 2), (8193, 128, 16, 16, 9), (8200, 100, 8, 1, 1), (8192, 72, 9, 1, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_many_tokens(T, E, k, n_group, topk_group, scoring):
    """Batches of many tokens: the first and last rows against the plain implementation, every row against the same
    rows in calls of few tokens (the choice exactly, the weight within a few of its own roundings)."""
    rng = np.random.default_rng(T)
    x = logits(rng, T, E, True)
    x[-1] = -np.inf
    x[-2, : E // 2] = np.nan
    bias = (rng.integers(-400, 401, E) / 4096.0).astype(np.float32) if T % 2 else None
    args = dict(scoring=scoring, n_group=n_group, topk_group=topk_group, group_score="top2", renormalize=k % 2 == 0,
                routed_scale=2.5)
    for dtype in (torch.float32, torch.bfloat16):
        xt = torch.from_numpy(x).cuda().to(dtype)
        bt = None if bias is None else torch.from_numpy(bias).cuda()
        ids, w = W.moe_gate_topk(xt, k, bias=bt, **args)
        some = [W.moe_gate_topk(c.contiguous(), k, bias=bt, **args) for c in xt.split(500)]
        assert torch.equal(ids, torch.cat([s[0] for s in some]))
        np.testing.assert_allclose(w.cpu().numpy(), torch.cat([s[1] for s in some]).cpu().numpy(),
                                   rtol=64 * 2.0 ** -24, atol=0)
        rows = np.r_[0:40, T - 40:T]
        ri, rw = reference(xt.float().cpu().numpy()[rows], k, bias, scoring, n_group, topk_group, "top2", k % 2 == 0, 2.5)
        np.testing.assert_array_equal(ids.cpu().numpy()[rows], ri)
        np.testing.assert_allclose(w.cpu().numpy()[rows], rw, rtol=64 * 2.0 ** -24, atol=0)


@pytest.mark.parametrize("T,E,k,n_group,topk_group", [
    (16385, 128, 16, 16, 9), (16390, 100, 8, 1, 1), (16384, 72, 9, 1, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_more_tokens(T, E, k, n_group, topk_group, scoring):
    """The batches from which on 65 to 128 experts go to 16 lanes a token."""
    test_many_tokens(T, E, k, n_group, topk_group, scoring)


def test_empty_and_other_stream():
    ids, w = W.moe_gate_topk(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    x = torch.randn(300, 64, device="cuda")
    want = W.moe_gate_topk(x, 6)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = W.moe_gate_topk(x, 6)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(TypeError):
        W.moe_gate_topk(x.half(), 2)
    with pytest.raises(ValueError):
        W.moe_gate_topk(x.t(), 2)
    with pytest.raises(ValueError):
        W.moe_gate_topk(x, 2, scoring="relu")
    with pytest.raises(ValueError):
        W.moe_gate_topk(x, 2, group_score="mean")
    with pytest.raises(ValueError):
        W.moe_gate_topk(x, 9, n_group=8, topk_group=1)
    with pytest.raises(ValueError):
        W.moe_gate_topk(x, 2, bias=torch.zeros(63, device="cuda"))
    for bad in (dict(k=0), dict(k=33), dict(k=2, n_group=3), dict(k=2, n_group=4, topk_group=5),
                dict(k=2, n_group=64, topk_group=64), dict(k=2, routed_scale=float("nan"))):
        with pytest.raises(W.W8A8Error):
            W.moe_gate_topk(x, **bad)
