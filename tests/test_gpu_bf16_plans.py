"""Every way in which the bf16 products are tiled, whole, with K shared by a cluster's pairs, or cut, each against 64 bits:
the ways are derived by the plan as written out in bf16_plan.py, so a case that a changed plan takes elsewhere fails."""
import random

import pytest
import torch

import w8a8_dynamic_quant_gb300 as W
from bf16_plan import grouped_tile, plan
from test_gpu_bf16 import close, grouped_reference, inputs, reference

# tile, gated, way -> sizes: rows of y on 16-byte boundaries and not, K that ends inside a stage, ragged last blocks
WAYS = {
    (32, False, "whole"): [(23, 2312, 208), (336, 11, 64)],
    (32, False, "split"): [(17, 264, 1040), (31, 250, 4512)],
    (32, False, "cut"): [(6, 22595, 1904), (30, 20000, 1616)],
    (32, True, "whole"): [(29, 2312, 208), (336, 11, 64)],
    (32, True, "split"): [(19, 264, 1040), (31, 113, 4512)],
    (32, True, "cut"): [(9, 12550, 1520), (9, 20784, 1616), (27, 10504, 2000)],
    (64, False, "whole"): [(2899, 114, 16), (574, 1400, 48), (47, 20001, 80), (300, 3801, 5664)],
    (64, False, "split"): [(1070, 110, 416), (60, 1096, 2064)],
    (64, False, "cut"): [(37, 26482, 3600), (45, 20480, 2064), (51, 26358, 5584)],
    (64, True, "whole"): [(2439, 9, 16), (3555, 112, 48), (43, 10250, 80)],
    (64, True, "split"): [(585, 61, 864), (140, 408, 2064)],
    (64, True, "cut"): [(38, 10467, 1520), (33, 13560, 5824)],
    (128, False, "whole"): [(1528, 1108, 64), (356, 14312, 16), (77, 18000, 144), (1159, 1283, 5360)],
    (128, False, "split"): [(214, 1063, 784), (569, 16, 720)],
    (128, False, "cut"): [(66, 20332, 2048), (68, 26699, 4304), (100, 21744, 4000)],
    (128, True, "whole"): [(356, 7153, 16), (354, 5960, 32)],
    (128, True, "split"): [(1973, 185, 560), (1220, 112, 864)],
    (128, True, "cut"): [(83, 12482, 3024), (65, 10168, 2272), (99, 12742, 4288)],
    (256, False, "whole"): [(5117, 1947, 128), (4890, 328, 32)],
    (256, False, "cut"): [(129, 20397, 3344), (1062, 3976, 5344)],
    (256, True, "whole"): [(5185, 140, 16), (2919, 1521, 32), (504, 2926, 5424)],
    (256, True, "cut"): [(141, 9761, 3472), (1398, 1728, 6048)],
}
CASES = [(*way, *size) for way, sizes in WAYS.items() for size in sizes]


def way_of(M, N, K, gated):
    nt, _, split, cut = plan(M, N, K, "swiglu" if gated else "none")
    return nt, gated, "cut" if cut else "split" if split > 1 else "whole"


def test_the_cases_are_every_way():
    for case in CASES:
        assert way_of(*case[3:], case[1]) == case[:3], (case, plan(*case[3:], "swiglu" if case[1] else "none"))
    rng = random.Random(3)
    for _ in range(20000):
        M, N, K = int(2.0 ** rng.uniform(0, 14)), int(2.0 ** rng.uniform(3, 16)), 16 * int(2.0 ** rng.uniform(0, 10))
        assert way_of(M, N, K, rng.random() < 0.5) in WAYS


def test_the_plan_is_the_librarys():
    """As far as its size tells: whether a product is cut, and its tile then."""
    from w8a8_dynamic_quant_gb300 import _capi, build
    build.build()
    call = _capi.lib().w8a8_bf16_matmul_call_bytes
    rng, cut = random.Random(4), 0
    sizes = [(*c[3:], c[1]) for c in CASES]
    sizes += [(int(2.0 ** rng.uniform(0, 12)), int(2.0 ** rng.uniform(8, 16)), 16 * int(2.0 ** rng.uniform(3, 10)),
               rng.random() < 0.5) for _ in range(30000)]
    for M, N, K, gated in sizes:
        nt, _, _, is_cut = plan(M, N, K, "swiglu" if gated else "none")
        want = 5120 + 76 * 4 * 128 * nt * 4 if is_cut else 256
        assert call(M, N, K, 5 if gated else 2) == want, (M, N, K, gated)
        cut += is_cut
    assert cut > 500


@pytest.mark.gpu
@pytest.mark.parametrize("nt,gated,way,M,N,K", CASES)
def test_every_way(nt, gated, way, M, N, K):
    act = "swiglu" if gated else ("gelu", "none", "silu", "gelu_tanh", "relu")[(M + N) % 5]
    x, w, b, r = inputs(M, N, K, act, True, True, M + N + K)
    v, err = reference(x, w, b, act, None)
    half = 2.0 ** -24 * (v + r.double()).abs()  # of the residual's sum
    ws = W.workspace(W.bf16_matmul_workspace_bytes(M, N, K))
    for out in (torch.bfloat16, torch.float32):
        y = W.w8a8_bf16_matmul(x, w, b, act, r, out, ws=ws)
        close(y, v + r.double(), err + half)
        assert torch.equal(W.w8a8_bf16_matmul(x, w, b, act, r, out), y)  # a workspace of its own, the same bits
    close(W.w8a8_bf16_matmul(x, w, b, act, None, torch.float32, ws=ws), v, err)
    stream = r.clone()
    W.w8a8_bf16_matmul(x, w, b, act, stream, ws=ws, y=stream)
    assert torch.equal(stream, W.w8a8_bf16_matmul(x, w, b, act, r, ws=ws))
    assert W.read_device_status(ws) == 0 and not bool(ws[:5120].any())


# tile -> rows of every expert: groups that end inside a tile, its half and a token box; empty ones; several tiles
GROUPS = {
    32: [[5, 0, 16, 17, 1, 33, 32, 15], [9] * 76 + [0] * 20],
    64: [[24, 0, 48, 33, 16, 40, 9, 30], [17] * 90, [0, 130, 0, 0, 2, 65, 0, 20], [64, 1, 49, 14]],
    128: [[60, 0, 113, 50, 16, 129, 34, 96], [33, 64, 157, 0]],
    256: [[300, 5, 0, 241, 129, 256, 0, 97], [3, 700]],
}


def test_the_groups_take_every_tile():
    for nt, lists in GROUPS.items():
        for counts in lists:
            assert grouped_tile(len(counts), sum(counts)) == nt, counts


@pytest.mark.gpu
@pytest.mark.parametrize("nt,i", [(nt, i) for nt, lists in GROUPS.items() for i in range(len(lists))])
@pytest.mark.parametrize("act,N,K", [("none", 264, 1040), ("swiglu", 200, 1040), ("relu", 145, 528), ("swiglu", 67, 528)])
def test_every_group_tile(nt, i, act, N, K):
    counts = GROUPS[nt][i]
    E, R = len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(R + N)
    rows = 2 * N if act == "swiglu" else N
    x = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(E, rows, K, generator=g, device="cuda") * 2 * K ** -0.5).to(torch.bfloat16)
    b = torch.randn(E, rows, generator=g, device="cuda").to(torch.bfloat16)
    gl = torch.tensor(counts, dtype=torch.int64, device="cuda")
    ws = W.workspace(W.bf16_grouped_matmul_workspace_bytes(E, R, N, K))
    v, err = grouped_reference(x, counts, w, b, act)
    for out in (torch.bfloat16, torch.float32):
        y = W.w8a8_bf16_grouped_matmul(x, gl, w, b, act, out, ws=ws)
        close(y, v, err)
        assert torch.equal(W.w8a8_bf16_grouped_matmul(x, gl, w, b, act, out, ws=ws), y)
    assert W.read_device_status(ws) == 0
