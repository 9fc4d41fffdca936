"""bf16 rows whose exact sum of squares lies on, or next to, the middle between two binary32 values; plain integers."""
import math
import random

import torch


def square_sum(row):
    """Sum of squares of finite bf16 values as (integer, exponent of two), exact."""
    total = 0
    for v in row:
        m, e = math.frexp(v)
        total += int(m * 256) ** 2 << (2 * (e + 140))
    return total, -2 * 148


def rounded32(total, exp):
    """total * 2^exp rounded once to binary32, ties to even, as a float; infinity above its range."""
    if total == 0:
        return 0.0
    lsb = max(total.bit_length() - 24 + exp, -149)
    shift = lsb - exp
    if shift > 0:
        q, rest = total >> shift, total & ((1 << shift) - 1)
        half = 1 << (shift - 1)
        q += rest > half or (rest == half and q & 1)
    else:
        q = total << -shift
    return math.inf if q.bit_length() + lsb > 128 else math.ldexp(q, lsb)


def near_tie_row(rng, K, lo, hi, off):
    """K values of magnitudes 2^lo .. 2^hi with both signs, whose squares' sum is a tie plus `off` times the square of
    2^(lo - 7): a few places, kept free, take what is missing, the largest square first."""
    free = 24 + (hi - lo) // 2
    while True:
        row = [math.ldexp(rng.randint(128, 255), rng.randint(lo, hi) - 7) for _ in range(K - free)]
        have = sum(int(math.ldexp(v, 7 - lo)) ** 2 for v in row)
        grid = have.bit_length() - 24  # a tie: an odd multiple of 2^(grid - 1)
        assert grid >= 1
        missing = (((have >> grid) + rng.randint(2, 5)) << grid) + (1 << (grid - 1)) + off - have
        fill = []
        while missing > 0 and len(fill) < free:
            r = math.isqrt(missing)
            cut = max(0, r.bit_length() - 8)
            r = r >> cut << cut
            missing -= r * r
            fill.append(math.ldexp(r, lo - 7))
        if missing == 0:
            row += fill + [0.0] * (free - len(fill))
            rng.shuffle(row)
            return [v if rng.random() < 0.5 else -v for v in row]


def near_tie_rows(seed, count, K, lo=-14, hi=4):
    """[count, K] bf16 and the rows' sums of squares, each rounded once: ties, and sums just below and above one."""
    rng = random.Random(seed)
    rows = [near_tie_row(rng, K, lo, hi, (0, -1, 1)[i % 3]) for i in range(count)]
    x = torch.tensor(rows, dtype=torch.float64)
    assert torch.equal(x.to(torch.bfloat16).double(), x)
    return x.to(torch.bfloat16), [rounded32(*square_sum(r)) for r in rows]
