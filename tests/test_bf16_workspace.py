"""The size of the bf16 products' workspace: one for the largest product serves every smaller one."""
import random

import pytest
import torch

import w8a8_dynamic_quant_gb300 as W


@pytest.fixture(scope="module")
def lib():
    from w8a8_dynamic_quant_gb300 import _capi, build
    build.build()
    return _capi.lib()


def log(rng, lo, hi):
    return int(round(2.0 ** rng.uniform(lo, hi)))


def test_one_size_serves_what_is_smaller(lib):
    rng = random.Random(1)
    cut = 0
    for _ in range(20000):
        M, N, K = log(rng, 0, 16), log(rng, 0, 16), 16 * log(rng, 0, 12)
        most = lib.w8a8_bf16_matmul_workspace_bytes(M, N, K)
        m, n, k, act = rng.choice([M, log(rng, 0, 16)]), rng.choice([N, log(rng, 0, 16)]), 16 * log(rng, 0, 12), rng.randrange(6)
        m, n = min(M, m), min(N, n)
        call = lib.w8a8_bf16_matmul_call_bytes(m, n, k, act)
        assert 256 <= call <= most, (m, n, k, act, call, M, N, most)
        assert lib.w8a8_bf16_matmul_workspace_bytes(m, n, k) <= most
        cut += call > 256
    assert cut > 500  # of the calls some need room


def test_the_sizes_that_were_too_small(lib):
    for most, small in (((8192, 14336, 4096), (64, 14336, 4096)), ((2048, 20480, 7168), (512, 20480, 7168))):
        assert lib.w8a8_bf16_matmul_workspace_bytes(*most) >= max(lib.w8a8_bf16_matmul_call_bytes(*small, a) for a in range(6))
    assert lib.w8a8_bf16_matmul_workspace_bytes(1 << 40, 1 << 40, 128) <= 5120 + 76 * 4 * 128 * 256 * 4


def test_call_bytes(lib):
    f = lib.w8a8_bf16_matmul_call_bytes
    assert f(64, 2048, 7168, 0) == 256 and f(0, 8, 128, 0) == 256
    assert f(64, 20480, 7168, 0) == 5120 + 76 * 4 * 128 * 64 * 4
    for bad in ((-1, 8, 128, 0), (4, 0, 128, 0), (4, 8, 0, 0), (4, 8, 65552, 0), (4, 8, 128, 6), (4, 8, 128, -1),
                ((1 << 31) - 256, 8, 128, 0), (4, 1 << 31, 128, 0)):
        assert f(*bad) == 0, bad


@pytest.mark.gpu
def test_smaller_products_on_a_large_workspace():
    """A workspace for 8192 rows through batches of which some are cut, and calls that bring their own: the same bits."""
    N, K = 20480, 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    w = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    ws = W.workspace(W.bf16_matmul_workspace_bytes(8192, N, K))
    for M in (1, 16, 64, 200, 512, 2048, 64, 16):
        for act, rows in (("none", N), ("swiglu", N)):
            x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
            want = W.w8a8_bf16_matmul(x, w[:rows], activation=act, ws=ws)
            junk = torch.full((48 << 20,), 255, dtype=torch.uint8, device="cuda")  # what the next allocation finds
            del junk
            assert torch.equal(W.w8a8_bf16_matmul(x, w[:rows], activation=act), want)
    assert W.read_device_status(ws) == 0 and not bool(ws[:5120].any())


@pytest.mark.gpu
def test_graphs_of_calls_without_a_workspace():
    """A captured call without a workspace zeroes its own at every replay; two such graphs share the capture's memory."""
    g = torch.Generator(device="cuda").manual_seed(2)
    pool, graphs = None, []
    for M, N, K, act in ((64, 20480, 1024, "none"), (33, 10200, 1040, "swiglu")):
        x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
        w = (torch.randn(2 * N if act == "swiglu" else N, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        W.w8a8_bf16_matmul(x, w, activation=act, y=y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            W.w8a8_bf16_matmul(x, w, activation=act, y=y)
            W.w8a8_bf16_matmul(x, w, activation=act, y=y)
        pool = pool or graph.pool()
        graphs.append((graph, x, w, act, y))
    for _ in range(5):
        for graph, x, w, act, y in graphs:
            x.mul_(1.25)
            y.zero_()
            graph.replay()
            assert torch.equal(y, W.w8a8_bf16_matmul(x, w, activation=act))
