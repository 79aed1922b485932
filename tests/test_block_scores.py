"""What a block's score says about its keys: <q, k> passes it by no more than what rounding
the query to 8 bits takes away."""
import numpy as np
import pytest
import torch

from chunk_ref import bounds, finite


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("kind", ["normal", "outliers"])
def test_score_and_slack_bound_every_key(dtype, H, kind):
    """With c = rn(q / t) every q_d is within t / 2 of t c_d, and the codes of the largest and
    smallest key are rounded outwards: <q, k> <= score + t / 2 sum_d |k_d|.  In fp32 the
    quotients (2^-24 of at most 127 steps of t, of the scale), the scale and the two products
    are off by less than 2^-20 of sum_d |q_d| max |k|."""
    g = torch.Generator().manual_seed(H)
    NB, K, G = 60, 2, 4
    kc = torch.randn(NB, 16, K, H, generator=g)
    q = torch.randn(K * G, H, generator=g)
    if kind == "outliers":  # one element many times the others: coarse steps for those
        kc[..., 3] *= 30
        q[:, 5] *= 40
    kc, q = kc.to(dtype), q.to(dtype)
    tables = torch.arange(NB, dtype=torch.int32)[None]
    codes, scale = bounds(kc, tables, [NB * 16], [0, NB * 16], np.zeros((NB, K, 2, H), np.int8),
                          np.zeros((NB, K), np.float32))
    for h in range(K):
        x = finite(q[h * G:(h + 1) * G])
        t = np.abs(x).max(1) / np.float32(127)
        c = np.rint(x / t[:, None]).astype(np.int64)
        dot = np.maximum(c, 0) @ codes[:, h, 0].astype(np.int64).T
        dot += np.minimum(c, 0) @ codes[:, h, 1].astype(np.int64).T
        score = (t[:, None] * scale[None, :, h]).astype(np.float64) * dot  # [G, NB]
        k = kc[:, :, h].double().numpy()
        s = np.einsum("gd,brd->gbr", x.astype(np.float64), k)
        slack = (t[:, None, None] / 2 * np.abs(k).sum(-1)[None]
                 + 2.0 ** -20 * np.abs(x).sum(-1)[:, None, None] * np.abs(k).max((1, 2))[None, :, None])
        assert (s <= score[..., None] + slack).all()


def test_a_key_may_pass_the_score_itself():
    """t = 1, s = 1 / 127: the score is 127, <q, k> is 127 + 63 / 4; the slack covers it."""
    kc = torch.ones(1, 16, 1, 64).half()
    codes, scale = bounds(kc, torch.zeros(1, 1, dtype=torch.int32), [16], [0, 16],
                          np.zeros((1, 1, 2, 64), np.int8), np.zeros((1, 1), np.float32))
    q = np.full(64, 0.25)
    q[0] = 127.0
    c = np.rint(q)
    score = float(scale[0, 0]) * (np.maximum(c, 0) @ codes[0, 0, 0] + np.minimum(c, 0) @ codes[0, 0, 1])
    dot = float(q @ np.ones(64))
    assert abs(score - 127) < 1e-3 and dot == 127 + 63 / 4
    assert score < dot <= score + 64 / 2 + 1e-3
