"""The norm's sum of squares is the exact sum rounded once to binary32, at every batch size: rows whose sum lies on or next
to the middle between two binary32 values, next to the end of their range, and far below eps' usual place."""
import math

import pytest
import torch

import w8a8_dynamic_quant_gb300 as W
from near_ties import near_tie_rows, rounded32, square_sum
from test_gpu_norm import FORMS, codes_reference, same_codes

pytestmark = pytest.mark.gpu


def norm_of(x, total, w, eps):
    """The norm in binary32 from the rows' sums of squares."""
    K = torch.full((), float(x.shape[1]), device="cuda")
    total = torch.tensor(total, dtype=torch.float32, device="cuda")[:, None]
    g = torch.rsqrt((total / K + torch.tensor(eps, device="cuda")).double()).float()
    return x.float() * g * w


def check(form, x, total, w, eps=1e-6):
    q, s, _, _ = FORMS[form](x, w, eps)
    rq, rs = codes_reference(norm_of(x, total, w, eps), form)
    assert torch.equal(s, rs), ("scales", int((s != rs).sum()), s.numel())
    assert same_codes(q, rq, form)


# (few, many): batches of one chunk a thread and of four; rows of one warp to 32, the last with eight chunks a thread
@pytest.mark.parametrize("K,many", [(256, 24), (512, 3000), (1024, 3000), (2048, 1500), (4096, 800), (8192, 400),
                                    (16384, 24), (32768, 12), (65536, 12)])
@pytest.mark.parametrize("form", list(FORMS))
def test_sums_next_to_a_tie(form, K, many):
    rows, total = near_tie_rows(K, 12 if K > 16384 else 24, K)
    w = torch.rand(K, generator=torch.Generator().manual_seed(K)).cuda() + 0.5
    x = rows.cuda()
    for n in (1, 3, 12, many):
        pick = [i % len(total) for i in range(n)]
        check(form, x[pick].contiguous(), [total[i] for i in pick], w)


@pytest.mark.parametrize("lo", [-60, -120])
@pytest.mark.parametrize("K,many", [(512, 3000), (4096, 800), (65536, 6)])
def test_far_smaller_values_decide(K, many, lo):
    """Ties and their neighbours whose last places lie up to 250 below the first."""
    rows, total = near_tie_rows(K - lo, 6 if K > 16384 else 24, K, lo=lo)
    w, x = torch.ones(K, device="cuda"), rows.cuda()
    for n in (3, many):
        pick = [i % len(total) for i in range(n)]
        check("int8", x[pick].contiguous(), [total[i] for i in pick], w)


def test_sums_with_a_residual():
    rows, total = near_tie_rows(5, 24, 4096)
    r, w = rows.cuda(), torch.ones(4096, device="cuda")
    x = torch.where(torch.rand(24, 4096, generator=torch.Generator().manual_seed(1)).cuda() < 0.5, r, r * 0.5)
    residual = r - x  # halves of bf16 values: exact
    for into in (None, x, residual):
        a, b = x.clone(), residual.clone()
        out = {id(x): a, id(residual): b}.get(id(into))
        q, s, stream, _ = W.w8a8_rms_norm_quant(a, w, residual=b, residual_out=out)
        rq, rs = codes_reference(norm_of(r, total, w, 1e-6), "int8")
        assert torch.equal(stream, r) and torch.equal(s, rs) and torch.equal(q, rq)


@pytest.mark.parametrize("form", list(FORMS))
def test_sums_at_the_ends_of_the_range(form):
    """Sums around the largest binary32 value (above 2^128 - 2^103 they are infinite), and sums so small that they or
    their squares are no normal numbers, under an eps that lets them count."""
    # 255 * 2^120 and a few values more or less than what is missing to 2^128 - 2^103
    missing, fill = 2 ** 120 - 2 ** 103, []
    while missing:
        r = math.isqrt(missing)
        r = r >> max(0, r.bit_length() - 8) << max(0, r.bit_length() - 8)
        missing -= r * r
        fill.append(float(r))
    assert len(fill) < 200
    tails = [fill, fill[:-1], fill[:-1] + [fill[-1] * 2], fill[:12], fill + [1.0], [], [2.0 ** 60]]
    for K, ones, value in ((512, 255, 2.0 ** 60), (2048, 1020, 2.0 ** 59)):
        rows = [[value] * ones + t for t in tails]
        rows = [r + [0.0] * (K - len(r)) for r in rows]
        x = torch.tensor(rows, dtype=torch.float64)
        assert torch.equal(x.to(torch.bfloat16).double(), x)
        total = [rounded32(*square_sum(r)) for r in rows]
        assert total[0] == total[2] == math.inf and total[1] == total[3] == 2.0 ** 128 - 2.0 ** 104
        check(form, x.to(torch.bfloat16).cuda(), total, torch.full((K,), 2.0 ** 20, device="cuda"))
    g = torch.Generator().manual_seed(2)
    for scale, eps in ((2.0 ** -66, 1e-38), (2.0 ** -70, 1e-42), (2.0 ** -74, 1e-44), (2.0 ** -76, 1e-45), (2.0 ** -50, 1e-30),
                       (2.0 ** -46, 1e-20), (2.0 ** -74, 1e-6)):
        x = (torch.randn(6, 1024, generator=g) * scale).to(torch.bfloat16)
        x[5] = 0.0
        total = [rounded32(*square_sum(r)) for r in x.double().tolist()]
        check(form, x.cuda(), total, torch.ones(1024, device="cuda"), eps)
