"""GPU choice of blocks whose bounds were never made: a scale that is no number, or minus
infinity, ranks its block behind all others."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from chunk_ref import choose
from test_gpu_select import make_select

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("what", [float("nan"), float("-inf")])
@pytest.mark.parametrize("N,K,lens", [(8, 2, [900, 5000, 333]), (4, 1, [9700 * 16])])
@pytest.mark.parametrize("negative", [False, True])
def test_blocks_without_bounds_rank_last(gpu, what, N, K, lens, negative):
    q, codes, scale, tables, ctx = make_select(len(lens), N, K, 64, BF16, lens, seed=len(lens))
    if negative:
        codes = -codes.abs()  # every score below zero
        q[:, :, ::2] = q[:, :, ::2].abs()
    q[0, 0, 0] = 0  # a query whose scores are all 0
    g = torch.Generator().manual_seed(1)
    gone = torch.rand(scale.shape, generator=g) < 0.3
    scale = torch.where(gone, torch.tensor(what), scale)
    ref = torch.where(gone, torch.tensor(float("nan")), scale)  # (the plain form puts NaN last)
    for keep in (5, 15, 250):  # the last: more than the rest
        got = gq.select_blocks(*(x.to(gpu) for x in (q, codes, scale, tables, ctx)), keep, first=1,
                               recent=1)
        want = choose(q[:, 0], codes.numpy(), ref.numpy(), tables, ctx, keep, 1, 1)
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)


def test_never_made_behind_a_bad_block(gpu):
    """A bad block id scores minus infinity, which is a number; blocks without bounds come
    after it, the lower one first; an infinite scale counts as fp32's largest number."""
    q, codes, scale, tables, ctx = make_select(1, 4, 1, 64, F16, [40 * 16], seed=3)
    scale[tables[0, 20:30].long()] = float("nan")
    tables[0, 10] = -4
    codes[tables[0, 7].long()] = 0
    codes[tables[0, 7].long(), :, 0] = 1
    scale[tables[0, 7].long()] = float("inf")
    q[:] = q.abs()
    for keep in (2, 3, 29, 30, 31, 32):
        got = gq.select_blocks(*(x.to(gpu) for x in (q, codes, scale, tables, ctx)), keep, first=0,
                               recent=1)
        order = got.blocks[0, 0].tolist()
        assert (7 in order) and (10 in order) == (keep >= 30)
        assert [i for i in order if 20 <= i < 30] == list(range(20, 20 + max(0, keep - 30)))
