"""How chunk attention shares its work among thread blocks (csrc/attention_chunk.cu), modelled
on the CPU over random batches: every KV tile of every item is one block's, the pieces of
an item are consecutive blocks', those that the kernel counts, and each block shares at
most one item with the blocks before it and one with those after it (its two slots for
partial results)."""
import random

import pytest

LONE, PAIR, START, QUOTA = 5, 6, 10, 10
NEAR = {LONE: LONE, PAIR: 8 * PAIR}


def items(seqs, heads, tpc, window):
    """(KV tiles, units each) of every item in order."""
    for n, ctx in seqs:
        for _ in range(heads):
            for f in range(0, n, 2 * tpc):
                e = min(n, f + 2 * tpc)
                lo = max(0, ctx - n + f - window + 1) // 128 if window else 0
                yield (ctx - n + e - 1) // 128 + 1 - lo, PAIR if f + tpc < e else LONE


def ceil_div(a, b):
    return -(-a // b)


def pieces_of(block, quota, total, work):
    """(item, from, to, first block, last block) as the kernel's scheduler walks them."""
    c0, c1 = block * quota, min(total, (block + 1) * quota)
    base = 0
    out = []
    if c0 >= c1:
        return out
    for i, (tiles, each) in enumerate(work):
        near = NEAR[each]
        first = base + START
        end = first + tiles * each
        if end <= c0:  # the plan starts at the item that holds unit c0
            base = end
            continue
        if base >= c1:
            break
        a, b = 0, tiles
        if c0 > first + near:
            a = tiles if end - c0 <= near else ceil_div(c0 - first, each)
        if c1 < end:
            if c1 <= first + near:
                b = 0
            elif end - c1 > near:
                b = ceil_div(c1 - first, each)
        if a < b:
            cut = b - a != tiles
            out.append((i, a, b, (first + near) // quota if cut else block,
                        (end - near - 1) // quota if cut else block, cut))
        base = end
    return out


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once(seed):
    rng = random.Random(seed)
    kind = seed % 4
    B = rng.choice([1, 1, 2, 5, 40])
    top = rng.choice([1, 3, 70, 700])
    seqs = []
    for _ in range(B):
        n = 1 if kind == 0 else rng.randint(0, top)
        seqs.append((n, max(n, 1) + rng.choice([0, rng.randint(0, 500), rng.randint(0, 30000)])))
    work = list(items(seqs, rng.choice([1, 2, 8]), rng.choice([1, 18, 32, 128]),
                      rng.choice([0, 0, 100, 1000])))
    grid = rng.choice([1, 7, 152])
    total = sum(START + t * e for t, e in work)
    quota = max(ceil_div(total, grid), QUOTA)
    seen = [[] for _ in work]
    for block in range(grid):
        before = after = 0
        mine = pieces_of(block, quota, total, work)
        assert [p[0] for p in mine] == sorted({p[0] for p in mine})
        for i, a, b, lo, hi, cut in mine:
            seen[i].append((block, a, b, lo, hi))
            if cut:
                assert lo <= block <= hi < grid
                if block == lo:
                    after += 1
                else:
                    before += 1
        assert before <= 1 and after <= 1
    for (tiles, _), got in zip(work, seen):
        at = 0
        for block, a, b, lo, hi in got:
            assert a == at and b > a
            at = b
            assert (lo, hi) == (got[0][0], got[-1][0])
        assert at == tiles
        assert [g[0] for g in got] == list(range(got[0][0], got[-1][0] + 1))
