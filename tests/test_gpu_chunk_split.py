"""GPU attention of chunks whose items of two row tiles are shared by several thread blocks:
with windows, in both types and head sizes."""
import pytest
import torch

import test_chunk_partition as model
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def cut_pairs(seqs, N, K, window):
    """Items of two row tiles that the kernel's partition cuts (G = N / K <= 128)."""
    grid = torch.cuda.get_device_properties(0).multi_processor_count
    work = list(model.items(seqs, K, 128 // (N // K), window))
    total = sum(model.START + t * e for t, e in work)
    quota = max(model.ceil_div(total, grid), model.QUOTA)
    return {p[0] for b in range(grid) for p in model.pieces_of(b, quota, total, work)
            if p[5] and work[p[0]][1] == model.PAIR}


def check(gpu, seqs, N, K, H, dtype, window, seed):
    assert cut_pairs(seqs, N, K, window)
    c = Case(seqs, N, K, H, dtype, seed=seed)
    for b, (n, ctx) in enumerate(seqs):  # below the earliest token's window: nobody's
        low = max(0, ctx - n - window + 1) if window else 0
        for j in range(low // 16):
            c.kc[c.tables[b, j].long()] = float("nan")
            c.tables[b, j] = -5
        if low % 16:
            c.kc[c.tables[b, low // 16].long(), :low % 16] = float("nan")
            c.vc[c.tables[b, low // 16].long(), :low % 16] = float("nan")
    got = c.run(gpu, window=window)
    assert c.status == 0
    assert torch.equal(got, c.run(gpu, window=window))  # whichever CTA folds
    # (the plain form multiplies what a row does not see by 0: finite numbers there)
    c.kc, c.vc = (torch.nan_to_num(x, nan=0.0, posinf=0.0) for x in (c.kc, c.vc))
    c.tables = c.tables.clamp(min=0)
    c.check(got, window=window)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("window", [0, 5000, 20001])
@pytest.mark.parametrize("n,N,K", [(64, 8, 2), (33, 4, 1), (256, 2, 2), (129, 1, 1)])
def test_shared_pairs(gpu, dtype, H, window, n, N, K):
    """Up to 235 KV tiles; the second row tile whole, or one row of it; with one head per KV
    head the tiles' windows start and end in different KV tiles."""
    check(gpu, [(n, 30000)], N, K, H, dtype, window, n)


@pytest.mark.parametrize("dtype,H", [(F16, 64), (BF16, 128)])
@pytest.mark.parametrize("window", [0, 3000])
def test_shared_pairs_among_other_items(gpu, dtype, H, window):
    check(gpu, [(1, 7000), (200, 9000), (3, 3), (70, 6000), (0, 5), (300, 300), (1, 1)], 14, 2, H,
          dtype, window, 7)


@pytest.mark.parametrize("ctx", [2300, 2500, 4200])
@pytest.mark.parametrize("dtype,H", [(F16, 128), (BF16, 64)])
def test_pairs_just_long_enough_to_be_shared(gpu, ctx, dtype, H):
    """Few KV tiles more than the two ends at which no boundary cuts."""
    check(gpu, [(40, ctx)], 16, 4, H, dtype, 0, ctx)
