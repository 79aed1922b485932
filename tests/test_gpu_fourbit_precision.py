"""GPU attention over a 4-bit cache where its arithmetic is put to the test.

Caches are made of codes and scales directly, the exact outputs in fp64 from the values
c * s.  Notation of the bounds: ref the exact output, A = sum p |V| with the exact
probabilities p, HALF the output type's half step relative to the value (2^-25 the
smallest f16 half step), P what the products with V leave of a probability, relative to
it.  Errors of the scores cost 2^-13 of A where sum |q k| scale log2(e) <= 40 (at most
H/16 + 4 roundings of 2^-23 of that: 2^-14 of a probability; numerator and sum).
"""
import numpy as np
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from oracle import fourbit as f4
from test_gpu_fourbit import HALF, t

pytestmark = pytest.mark.gpu
P = {"f16": 2.0 ** -22, "bf16": 2.0 ** -11}  # of a probability, in the products with V
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
GRID = f4.scale_values()


def byte(s):
    """The scale byte of a value on the grid."""
    (i,) = np.flatnonzero(GRID[:226] == s)
    return int(i)


class Cache:
    """One KV head of one sequence of n positions: codes [n, H] in -7..7 and scale
    bytes [n, H/32] of keys and values, in shuffled blocks."""

    def __init__(self, kc, ks, vc, vs, seed=0):
        n, H = kc.shape
        self.n, self.H, nb = n, H, (n + 15) // 16
        self.perm = np.random.default_rng(seed).permutation(nb + 2)[:nb].astype(np.int32)
        self.parts = []
        for c, s in ((kc, ks), (vc, vs)):
            nib = np.zeros((nb * 16, H), np.uint8)
            nib[:n] = (c + 8).astype(np.uint8)
            codes = np.full((nb + 2, 1, 16, H // 2), 0xFF, np.uint8)
            scale = np.full((nb + 2, 1, 16, H // 32), 0xFF, np.uint8)
            codes[self.perm, 0] = (nib[:, 0::2] | (nib[:, 1::2] << 4)).reshape(nb, 16, -1)
            pad = np.full((nb * 16, H // 32), 0xFF, np.uint8)
            pad[:n] = s
            scale[self.perm, 0] = pad.reshape(nb, 16, -1)
            self.parts.append((codes, scale))
        self.k = kc * np.repeat(GRID[ks], 32, 1)
        self.v = vc * np.repeat(GRID[vs], 32, 1)

    def attend(self, q, dtype, dev, *, B=1, scale=None):
        """q [N, H] (exact in dtype) for B sequences that share the blocks: [B, N, H]."""
        (kc, ks), (vc, vs) = ([t(x, dev) for x in p] for p in self.parts)
        qd = torch.from_numpy(q).to(DT[dtype])
        assert (qd.double().numpy() == q).all()
        qd = qd.to(dev)[None, None].expand(B, 1, -1, -1).contiguous()
        tables = t(self.perm[None], dev).expand(B, -1).contiguous()
        lens = torch.full((B,), self.n, dtype=torch.int32, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        out = gq.decode_attention_quant(qd, kc, vc, ks, vs, tables, lens, kv="int4", scale=scale,
                                        status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return out[:, 0].double().cpu().numpy()

    def exact(self, q, scale=None):
        """(ref, A, sum of exp(s - max s)) of every row."""
        s = q @ self.k.T * (scale or self.H ** -0.5)
        p = np.exp(s - s.max(-1, keepdims=True))
        L = p.sum(-1, keepdims=True)
        return p @ self.v / L, p @ np.abs(self.v) / L, L


def check(out, ref, lim):
    assert np.isfinite(out).all()
    worst = np.abs(out - ref) / lim
    assert (worst <= 1).all(), (int((worst > 1).sum()), float(worst.max()))


@pytest.mark.parametrize("N,H,dtype", [(4, 64, "f16"), (4, 128, "bf16"), (16, 128, "f16"),
                                       (24, 64, "bf16")])
@pytest.mark.parametrize("gap", [16, 18, 20])
def test_a_long_tail_behind_dominant_positions(gpu, N, H, dtype, gap):
    """A few positions lead by `gap` nats and have no value (attention sinks): the
    output is the tail's, whose probabilities are near 2^-23 .. 2^-29 of the
    sinks'.  Probabilities enter the products as f16 against a reference that
    leaves the largest at 2^7 at least: each of the tail is off by at most 2^-25 of
    that, 2^-32 of a sink's.  320 segments: four warps each, sinks in the share of
    every one."""
    n, rng = 100_003, np.random.default_rng(gap)
    kc = np.zeros((n, H), np.int64)
    kc[:, 0] = rng.integers(-7, 8, n)
    ks = np.full((n, H // 32), byte(2.0 ** -4))
    vc, vs = rng.integers(1, 8, (n, H)), np.full((n, H // 32), byte(0.25))
    vc *= rng.choice([-1, 1], H)
    sinks = np.array([f * n // 4 // 128 * 128 + 32 * w for f in range(4) for w in range(4)])
    kc[sinks], ks[sinks], vc[sinks] = 0, byte(gap / 8.0), 0
    kc[sinks, 0] = 7
    q = np.zeros((N, H))
    q[:, 0] = 8.0
    scale = 1.0 / 7  # a sink scores gap, the tail -0.5 .. 0.5
    c = Cache(kc, ks, vc, vs)
    ref, A, L = c.exact(q, scale)
    assert (L < 20).all() and (np.abs(ref) > 5e-6).all()
    lost = n * 2.0 ** -32 / L
    inner = A * (2.0 ** -11 + 2.0 ** -13) + lost * (np.abs(c.v).max() + np.abs(ref))
    lim = inner + HALF[dtype] * (np.abs(ref) + inner) + 2.0 ** -25
    out = c.attend(q, dtype, gpu, B=320, scale=scale)
    check(out, ref, lim)


@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 27, 2.0 ** 28, 2.0 ** 40, 2.0 ** 80, 2.0 ** 110])
@pytest.mark.parametrize("N,H", [(4, 128), (16, 64)])
def test_scores_of_any_size(gpu, N, H, size):
    """Scores of millions and more, of both signs: the largest takes the row, whatever
    the spacing of fp32 numbers near it.  (The best and the next key differ by a
    quarter of the best's score, far above any rounding.)"""
    n, rng = 700, np.random.default_rng(3)
    kc = np.zeros((n, H), np.int64)
    kc[:, 0] = rng.integers(1, 6, n)
    ks, vs = np.full((n, H // 32), byte(1.0)), np.full((n, H // 32), byte(0.5))
    vc = rng.integers(-7, 8, (n, H))
    kc[413, 0], kc[77, 0] = 7, -7
    q = np.zeros((N, H))
    q[:, 0] = size
    c = Cache(kc, ks, vc, vs)
    out = c.attend(q, "bf16", gpu, B=3)
    check(out, c.v[413][None], 2.0 ** -8 * np.abs(c.v[413]) + 2.0 ** -30)
    kc[:, 0] = rng.integers(2, 7, n)  # every score far below zero
    kc[413, 0], kc[77, 0], q[:, 0] = 1, 7, -size
    c = Cache(kc, ks, vc, vs)
    out = c.attend(q, "bf16", gpu, B=3)
    check(out, c.v[413][None], 2.0 ** -8 * np.abs(c.v[413]) + 2.0 ** -30)


@pytest.mark.parametrize("N,H", [(4, 64), (4, 128), (16, 64), (16, 128), (24, 128)])
def test_f16_outputs_keep_the_probabilities(gpu, N, H):
    """f16 outputs: what rounding a probability to f16 leaves is a second term of the
    products, so 2^-22 of A remains of it and values that nearly cancel come out
    within the output's own half step."""
    rng = np.random.default_rng(N + H)
    for n in (2, 3, 5, 16, 17, 33, 295):
        codes = lambda: rng.integers(-7, 8, (n, H))  # noqa: E731
        sb = lambda lo, hi: rng.integers(lo, hi, (n, H // 32))  # noqa: E731
        vc = codes()
        if n <= 3:
            vc[1:] = -vc[:1]
        c = Cache(codes(), sb(byte(2.0 ** -4), byte(2.0 ** -3)), vc, sb(byte(0.25), byte(0.5)))
        q = torch.from_numpy(rng.standard_normal((N, H))).half().double().numpy()
        ref, A, L = c.exact(q)
        inner = A * (2.0 ** -13 + 2.0 ** -15 + 2.0 ** -22)
        inner = inner + n * 2.0 ** -32 / L * 2 * np.abs(c.v).max()
        out = c.attend(q, "f16", gpu)[0]
        check(out, ref, inner + HALF["f16"] * (np.abs(ref) + inner) + 2.0 ** -25)


@pytest.mark.parametrize("N,H,dtype", [(3, 64, "bf16"), (4, 128, "f16"), (24, 128, "bf16")])
def test_every_piece_of_a_split_segment_counts(gpu, N, H, dtype):
    """Values that are waves along the sequence and average to almost nothing: leaving
    out (or doubling) any stretch of 300 positions would move the output by several
    times the bound, which is checked first."""
    n, rng = 90_005, np.random.default_rng(N)
    j, d = np.arange(n)[:, None], np.arange(H)[None]
    wave = np.cos(2 * np.pi * (j * (1 + d // 2) / n + 0.25 * (d % 2)))
    vc, vs = np.rint(7 * wave).astype(np.int64), np.full((n, H // 32), byte(0.125))
    kc, ks = rng.integers(-7, 8, (n, H)), np.full((n, H // 32), byte(2.0 ** -6))
    q = torch.from_numpy(rng.standard_normal((N, H))).to(DT[dtype]).double().numpy()
    c = Cache(kc, ks, vc, vs)
    ref, A, L = c.exact(q)
    steps = n / 16 / 16 * 2.0 ** -21  # at least 16 warps share it
    inner = A * (P[dtype] + 2.0 ** -13 + steps) + n * 2.0 ** -32 / L
    lim = inner + HALF[dtype] * (np.abs(ref) + inner) + 2.0 ** -25
    s = q @ c.k.T * H ** -0.5
    p = np.exp(s - s.max(-1, keepdims=True))
    for lo in range(0, n - 300, 300):
        part, v = p[:, lo:lo + 300], c.v[lo:lo + 300]
        moved = np.abs(part @ v - ref * part.sum(-1, keepdims=True)) / L
        assert (moved / lim).max() > 3
    check(c.attend(q, dtype, gpu)[0], ref, lim)


@pytest.mark.parametrize("N,H", [(4, 128), (4, 64), (16, 128), (24, 64)])
def test_thousands_of_positions_in_one_warp(gpu, N, H):
    """320 long segments: four warps each, so one adds up 10^4 positions and more.  Values
    that nearly cancel, a group with one large channel (the others' codes 0 and +-1)
    and a channel of zeros.  Scores are one product each (2^-22 of |score| <= 1 with
    its scale factor, ex2 2^-22, P: 2^-20 of A, numerator and sum).  A product step
    truncates each of 17 addends at 2^-23 of the largest with two bits to spare:
    2^-21 of a partial sum at most, and partial sums stay within the range of the
    cumulative sums of a warp's share (pairs of tiles, every fourth)."""
    n, rng = 113_000, np.random.default_rng(H + N)
    kc = np.zeros((n, H), np.int64)
    kc[:, 0] = rng.integers(-7, 8, n)
    ks = np.full((n, H // 32), byte(2.0 ** -4))
    vc = rng.integers(-1, 2, (n, H))
    vc[:, 32:] = rng.integers(-7, 8, (n, H - 32))
    vc[:, 5] = rng.choice([-7, 7], n)
    vc[:, 9] = 0
    vs = np.full((n, H // 32), byte(0.25))
    q = np.zeros((N, H))
    q[:, 0] = rng.choice([-8.0, 8.0], N)
    scale = 1.0 / 7
    c = Cache(kc, ks, vc, vs)
    ref, A, L = c.exact(q, scale)
    out = c.attend(q, "f16", gpu, B=320, scale=scale)
    share = np.arange(n) // 32 % 4
    R = np.zeros((N, H))
    for r in range(N):
        s = c.k @ q[r] * scale
        pv = np.exp(s - s.max())[:, None] * c.v
        for w in range(4):
            cum = np.cumsum(pv[share == w], 0)
            R[r] = np.maximum(R[r], np.maximum(cum.max(0), 0) - np.minimum(cum.min(0), 0))
    steps = n / 16 * 2.0 ** -21  # all warps'; the sum of p meets a warp's
    inner = A * 2.0 ** -20 + steps * R / L + np.abs(ref) * steps / 4 + n * 2.0 ** -32 / L * 1.75
    check(out, ref, inner + HALF["f16"] * (np.abs(ref) + inner) + 2.0 ** -25)
