"""The choice of tiles, parts and cuts of the bf16 products, written out again: the tests take their sizes by it."""
MOST = 76  # CTA pairs
FIT = [0, 76, 36, 23, 15, 13, 8, 7, 7]


def tile(per):
    return 32 if per <= 32 else 64 if per <= 64 else 128 if per <= 128 else 256


def block_cost(n):
    return max(2 * n, (128 + n // 2) * 128 // 58)


def plan(M, N, K, act):
    """(tile, tokens a block, parts of K, cut)"""
    width = 128 if act == "swiglu" else 256
    channel_blocks, KB = -(-N // width), -(-K // 64)
    best, out = None, None
    for per in range(min(256, (M + 15) // 16 * 16), 15, -16):
        units = -(-M // per) * channel_blocks
        waves = -(-units // MOST)
        takes = [(waves * (KB * block_cost(per) + 300) + 8 * per, 1, 0)]
        if MOST < units < 4 * MOST and units % MOST:
            takes.append((-(-units * KB // MOST) * block_cost(per) + (waves + 1) * 300 + 2000 + 100 * per, 1, 1))
        takes += [(-(-KB // ks) * block_cost(per) + 1200 + 6 * per, ks, 0) for ks in range(2, 9)
                  if units <= FIT[ks] and 2 * ks <= KB and per <= 128]
        for cost, ks, cut in takes:
            if best is None or cost < best:
                best, out = cost, (tile(per), per, ks, cut)
    return out


def grouped_tile(E, R):
    want = 2 * -(-R // E)
    return 32 if want <= 32 else 64 if want <= 64 else 128 if want <= 128 else 256
