"""GPU attention of chunks whose scores are so large that neighbouring fp32 numbers are further
apart than what a probability may hold."""
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from chunk_ref import chunk, chunk_bound
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def whole_scores(c, values, gen):
    """Keys that score whole numbers of `values` for every query, exactly."""
    c.q = torch.zeros_like(c.q)
    c.q[..., 3] = 1
    k = torch.zeros(c.kc.shape)
    k[..., 3] = values[torch.randint(len(values), c.kc.shape[:3], generator=gen)]
    c.kc = torch.where(c.kc.isnan(), c.kc, k.to(c.dtype))
    return c


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("power", [18, 22, 23, 24, 25, 27, 28, 29, 31, 36, 60, 110])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(gpu, dtype, H, power, sign):
    """Multiples of 2^power, above or below zero: the largest ones share a row alone, whatever
    order they come in; rows of one CTA's items and of shared ones."""
    g = torch.Generator().manual_seed(power)
    c = Case([(33, 900), (1, 9000), (128, 128), (3, 3)], 8, 2, H, dtype, seed=power)
    whole_scores(c, sign * torch.arange(1.0, 8.0), g)
    got = c.run(gpu, scale=2.0 ** power)
    assert c.status == 0
    c.check(got, scale=2.0 ** power)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("power", [0, 4, 8])
def test_large_and_small_scores_in_one_batch(gpu, dtype, power):
    """Ordinary rows beside rows whose scores grow along the context, to 2^27 and 2^35."""
    g = torch.Generator().manual_seed(power)
    c = Case([(40, 2000), (7, 700)], 8, 2, 128, dtype, seed=power)
    ordinary, k = c.q * 2.0 ** (-3 - power), torch.nan_to_num(c.kc)
    whole_scores(c, torch.arange(1.0, 8.0), g)
    c.q[1::3] *= 2.0 ** 12
    c.q[::3] = ordinary[::3]
    c.q[::3, :, :8] = 0
    for b, (_, n) in enumerate(c.seqs):
        for i in range(-(-n // 16)):
            blk = c.tables[b, i].long()
            c.kc[blk, ..., 3] *= 2.0 ** min(12, i // 4)
    c.kc[..., 8:] = torch.where(c.kc[..., 8:].isnan(), c.kc[..., 8:], k[..., 8:])
    got = c.run(gpu, scale=2.0 ** power)
    assert c.status == 0
    c.check(got, scale=2.0 ** power)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sparse_scores_of_any_size(gpu, dtype):
    for power in (22, 24, 28, 31, 60):
        g = torch.Generator().manual_seed(power)
        c = Case([(1, 9000), (1, 700)], 8, 2, 128, dtype, seed=power)
        whole_scores(c, torch.arange(-5.0, 6.0), g)
        want = c.run(gpu, scale=2.0 ** power)
        c.check(want, scale=2.0 ** power)
        got = gq.sparse_decode_attention(c.q[:, None].to(gpu), c.kc.to(gpu), c.vc.to(gpu),
                                         c.tables[:, None].repeat(1, 2, 1).to(gpu),
                                         c.ctx.to(gpu), scale=2.0 ** power)
        c.check(got[:, 0], scale=2.0 ** power)


@pytest.mark.parametrize("dtype,H", [(F16, 128), (BF16, 64)])
@pytest.mark.parametrize("window", [1, 17, 128, 300, 5000])
@pytest.mark.parametrize("power", [26, 36])
def test_windows_of_large_scores(gpu, dtype, H, window, power):
    g = torch.Generator().manual_seed(window)
    c = Case([(33, 900), (1, 9000), (300, 300), (3, 3), (64, 30000)], 8, 2, H, dtype, seed=window)
    whole_scores(c, torch.arange(-3.0, 4.0), g)
    got = c.run(gpu, scale=2.0 ** power, window=window)
    assert c.status == 0
    # (the plain form multiplies what a row does not see by 0: finite numbers there)
    c.kc, c.vc = (torch.nan_to_num(x, nan=0.0, posinf=0.0) for x in (c.kc, c.vc))
    c.check(got, window=window, scale=2.0 ** power)
