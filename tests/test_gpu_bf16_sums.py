"""fp32 outputs whose sums over chunks of K stay in tensor memory from one chunk to the next, where a CTA pair's units have
different numbers of tokens in turn: the two halves of the epilogue are not in step with each other then."""
import pytest
import torch

import w8a8_dynamic_quant_gb300 as W
from bf16_plan import grouped_tile, plan
from test_gpu_bf16 import close, gen, grouped_reference, inputs, reference


# a ragged last block among the pairs' units, more than one chunk of K; stores that take long (rows on no 16-byte boundary)
DENSE = [(522, 6429, 1056, "none", 128), (304, 9970, 1296, "relu", 128), (295, 5929, 784, "swiglu", 128),
         (573, 6796, 736, "none", 128)]
# groups of every number of tokens up to the tile's
GROUPED = [([128, 17, 96, 40, 112, 64, 10, 33] * 8, 1025, 1040, "none", 128),
           ([128, 17, 96, 40, 112, 64, 10, 33, 20] * 4, 1025, 1040, "swiglu", 128),
           ([64, 17, 48, 9, 30, 0, 33, 20] * 16, 515, 1040, "none", 64), ([64, 3, 48, 9, 30, 0, 33, 20] * 12, 515, 2064, "swiglu", 64)]


def test_the_cases_are_what_they_say():
    for M, N, K, act, nt in DENSE:
        tile, per, split, cut = plan(M, N, K, act)
        units = -(-M // per) * -(-N // (128 if act == "swiglu" else 256))
        assert (tile, split, cut) == (nt, 1, 0) and M % per and units > 76 and K > 512
    for counts, _, K, _, nt in GROUPED:
        assert grouped_tile(len(counts), sum(counts)) == nt and K > 512


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,act,nt", DENSE)
def test_ragged_blocks(M, N, K, act, nt):
    x, w, b, r = inputs(M, N, K, act, True, True, M)
    ws = W.workspace(256)
    y = W.w8a8_bf16_matmul(x, w, b, act, r, torch.float32, ws=ws)
    close(y, *reference(x, w, b, act, r))
    for _ in range(150):
        assert torch.equal(W.w8a8_bf16_matmul(x, w, b, act, r, torch.float32, ws=ws), y)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K,act,nt", GROUPED, ids=[str(i) for i in range(len(GROUPED))])
def test_ragged_groups(counts, N, K, act, nt):
    E, R, rows, g = len(counts), sum(counts), 2 * N if act == "swiglu" else N, gen(N)
    x = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(E, rows, K, generator=g, device="cuda") * 2 * K ** -0.5).to(torch.bfloat16)
    gl, ws = torch.tensor(counts, device="cuda"), W.workspace(256)
    y = W.w8a8_bf16_grouped_matmul(x, gl, w, None, act, torch.float32, ws=ws)
    close(y, *grouped_reference(x, counts, w, None, act))
    for _ in range(150):
        assert torch.equal(W.w8a8_bf16_grouped_matmul(x, gl, w, None, act, torch.float32, ws=ws), y)
