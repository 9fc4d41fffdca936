"""Every launch shape of the norm, chunks a thread x warps a row, against the formula bit for bit."""
import os

import pytest
import torch

from test_gpu_norm import FORMS, check, gen

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def arm(M, K, sms):
    """(chunks a thread, warps a row) as csrc/norm.cu chooses them."""
    n = K // 8
    if n <= 32:
        return 1, 1
    if n <= 1024 and M * -(-n // 128) < 16 * sms:
        return 1, next(g for g in (2, 4, 8, 16, 32) if n <= 32 * g)
    return next(((4, g) for g in (1, 2, 4, 8, 16, 32) if n <= 128 * g), (8, 32))


# (chunks, warps) -> (rows, values): rows that fill the last chunk, end inside it, or leave threads without one
ARMS = {
    (1, 1): [(5, 256), (2437, 32), (3001, 160)],
    (1, 2): [(5, 288), (2431, 512)],
    (1, 4): [(9, 544), (2431, 1024)],
    (1, 8): [(9, 1056), (1215, 2048)],
    (1, 16): [(9, 2080), (607, 4096)],
    (1, 32): [(9, 4128), (303, 8192)],
    (4, 1): [(2432, 1024), (2501, 288), (2600, 992)],
    (4, 2): [(1216, 2048), (1300, 1056), (1300, 2016)],
    (4, 4): [(608, 4096), (900, 2080), (900, 4064)],
    (4, 8): [(304, 8192), (500, 4128), (500, 7168)],
    (4, 16): [(3, 16384), (200, 8224)],
    (4, 32): [(3, 32768), (100, 16416)],
    (8, 32): [(2, 65536), (60, 32800)],
}
CASES = [(*a, *size) for a, sizes in ARMS.items() for size in sizes]


def test_the_cases_are_every_arm():
    for ch, g, M, K in CASES:
        assert arm(M, K, 152) == (ch, g), (ch, g, M, K)
    assert {arm(M, K, 152) for M in (1, 300, 700, 1300, 2600) for K in range(32, 65537, 32)} == set(ARMS)
    with open(os.path.join(ROOT, "w8a8_dynamic_quant_gb300", "csrc", "norm.cu")) as f:
        source = f.read()
    # the rules that arm() repeats
    for line in ("nchunk <= 32) return go<FORM, 1, 1>", "nchunk <= 1024 && a.M * ((nchunk + 127) / 128) < 16 * num_sms",
                 *(f"nchunk <= {32 * g}) return go<FORM, 1, {g}>" for g in (2, 4, 8, 16)), "return go<FORM, 1, 32>",
                 *(f"nchunk <= {128 * g}) return go<FORM, 4, {g}>" for g in (1, 2, 4, 8, 16, 32)), "return go<FORM, 8, 32>"):
        assert line in source, line


@pytest.mark.gpu
@pytest.mark.parametrize("ch,g,M,K", CASES)
@pytest.mark.parametrize("form", list(FORMS))
def test_every_arm(form, ch, g, M, K):
    assert arm(M, K, torch.cuda.get_device_properties(0).multi_processor_count) == (ch, g)
    r = gen(M + K)
    x = torch.randn(M, K, generator=r, device="cuda")
    x[:, ::97] *= 30.0
    x = x.to(torch.bfloat16)
    size = torch.exp2(torch.randint(-20, 20, (M, 1), generator=r, device="cuda").float())
    res = (torch.randn(M, K, generator=r, device="cuda") * size).to(torch.bfloat16)
    w = 1.0 + 0.3 * torch.randn(K, generator=r, device="cuda")
    check(form, x, w, residual=res, want_y=True)
    check(form, x, w.to(torch.bfloat16), residual=res)
    check(form, x, w.to(torch.bfloat16), want_y=True)
    x[M // 2, K - 1] = float("nan")
    x[M - 1, 3] = float("inf")
    x[0] = 0.0
    check(form, x, w)
