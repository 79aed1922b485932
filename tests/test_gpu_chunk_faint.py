"""GPU attention of chunks and over chosen blocks where one key outweighs each of tens of
thousands of others by some 17 nats (an attention sink), so that what the others weigh
together has to survive each one's rounding to 16 bits."""
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def bound(out, mag, total, dtype):
    """As chunk_bound: with u half a step of the type, each probability is rounded once
    (u mag in the products) and the result once (u |out|, or half a step of the smallest
    numbers); scores, exp2 and sums in fp32 are off by less than 2^-12 of each probability.
    Below f16's normal numbers a probability is off by up to 2^-25 instead, where the largest
    one is 2^7 or more and so is their sum: 2^-32 of every |v| together (`total`)."""
    fi = torch.finfo(dtype)
    tiny = 2.0 ** -25 if dtype == F16 else fi.tiny * fi.eps
    u = fi.eps / 2
    return ((u + 2 ** -12) * mag + (u + 2 ** -12) * out.abs() + torch.clamp(u * out.abs(), min=tiny)
            + (2.0 ** -32 * total if dtype == F16 else 0.0))


class Sinks:
    """B sequences over the same `ctx` cached tokens: a score of `d` for position 0, whose V is
    0, and 0 for all others, whose V is 0.5 .. 1.5."""

    def __init__(self, dev, ctx, d, K, H, dtype):
        g = torch.Generator(device=dev).manual_seed(ctx)
        NB = -(-ctx // 16)
        self.order = torch.randperm(NB, generator=g, device=dev).to(torch.int32)
        rows = torch.zeros(NB * 16, K, H, device=dev)
        rows[0, :, 0] = d
        self.v = (0.5 + torch.rand(NB * 16, K, H, generator=g, device=dev)).to(dtype)
        self.v[0] = 0
        self.kc, self.vc = (torch.empty(NB, 16, K, H, dtype=dtype, device=dev) for _ in range(2))
        self.kc[self.order.long()] = rows.to(dtype).view(NB, 16, K, H)
        self.vc[self.order.long()] = self.v.view(NB, 16, K, H)
        assert float(rows.to(dtype)[0, 0, 0]) == d
        self.ctx, self.d, self.dtype = ctx, d, dtype

    def queries(self, *shape):
        q = torch.zeros(*shape, dtype=self.dtype, device=self.kc.device)
        q[..., 0] = 1
        return q

    def check(self, got, n):
        """got [n,N,H] of the last n tokens, in 64 bits from the formula."""
        v = self.v.double()[:self.ctx]
        w = torch.full((self.ctx, 1, 1), torch.exp(torch.tensor(-self.d, dtype=torch.float64)).item(),
                       dtype=torch.float64, device=v.device)
        w[0] = 1
        sums = torch.cumsum(w * v, 0)[-n:]  # (v >= 0: |v| sums alike)
        want = sums / torch.cumsum(w, 0)[-n:]
        total = torch.cumsum(v, 0)[-n:]
        G = got.shape[1] // v.shape[1]
        over = ((got.double() - want.repeat_interleave(G, 1)).abs()
                - bound(want, want, total, self.dtype).repeat_interleave(G, 1))
        assert float(over.max()) <= 0, f"{float(over.max())} over, of {float(want.max())}"


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("ctx,d", [(20000, 17.25), (131072, 17.375), (40000, 9.5)])
@pytest.mark.parametrize("B,n", [(19, 1), (19, 40), (1, 1)])
def test_many_faint_keys_behind_a_sink(gpu, dtype, H, ctx, d, B, n):
    """19 sequences of 8 KV heads: as many items as SMs, most of them one CTA's alone."""
    s = Sinks(gpu, ctx, d, 8, H, dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    got = gq.chunk_attention(s.queries(B * n, 32, H), s.kc, s.vc, s.order[None].repeat(B, 1),
                             i32([ctx] * B), i32([n * b for b in range(B + 1)]), scale=1.0)
    for b in range(B):
        s.check(got[n * b:n * b + n], n)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("ctx,d,B", [(20000, 17.25, 19), (32768, 17.375, 19), (32768, 17.375, 1)])
def test_many_faint_keys_in_chosen_blocks(gpu, dtype, ctx, d, B):
    s = Sinks(gpu, ctx, d, 8, 128, dtype)
    got = gq.sparse_decode_attention(s.queries(B, 1, 32, 128), s.kc, s.vc,
                                     s.order[None, None].repeat(B, 8, 1),
                                     torch.full((B,), ctx, dtype=torch.int32, device=gpu), scale=1.0)
    for b in range(B):
        s.check(got[b], 1)
