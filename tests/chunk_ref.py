"""Plain 64-bit forms of the chunk, rotation and block-choice calls, for the tests (torch on
the CPU; written from the formulas, no library code)."""
import math

import numpy as np
import torch


def rows_of(cache, table, n):
    """[n,K,H] float64 rows of a sequence."""
    pos = torch.arange(n)
    return cache[table[pos // 16].long(), pos % 16].double()


def chunk(q, kc, vc, tables, ctx, cu, window=0, scale=None, skip=()):
    """(out, weight) float64 [M,N,H]: the attention, and sum_j p_j |v_j| that its roundings
    scale with.  Sequences in `skip` are left out (zeros)."""
    M, N, H = q.shape
    K = kc.shape[2]
    G = N // K
    scale = scale or 1.0 / math.sqrt(H)
    out, mag = torch.zeros(2, M, N, H, dtype=torch.float64)
    for b in range(len(ctx)):
        n, c = int(cu[b + 1] - cu[b]), int(ctx[b])
        if n <= 0 or b in skip:
            continue
        lo = max(0, c - n - window + 1) // 16 * 16 if window else 0
        t = tables[b].clone()
        t[:lo // 16] = t[lo // 16]
        k, v = rows_of(kc, t, c)[lo:], rows_of(vc, t, c)[lo:]
        mine = torch.arange(c - n, c)[:, None]
        pos = torch.arange(lo, c)[None]
        seen = pos <= mine
        if window:
            seen &= pos > mine - window
        rows = slice(int(cu[b]), int(cu[b + 1]))
        low = int((c - n) - window + 1 - lo) if window else 0
        v = v.clone()
        if low > 0:
            v[:low] = 0  # seen by no token
        for h in range(K):
            s = torch.einsum("tgd,jd->gtj", q[rows, h * G:(h + 1) * G].double(), k[:, h]) * scale
            p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
            out[rows, h * G:(h + 1) * G] = torch.einsum("gtj,jd->tgd", p, v[:, h])
            mag[rows, h * G:(h + 1) * G] = torch.einsum("gtj,jd->tgd", p, v[:, h].abs())
    return out, mag


def chunk_bound(out, mag, dtype):
    """How far a result may be off: with u half a step of the type, each probability is
    rounded once (u, in the products and in the sum alike: u (mag + |out|)) and the result
    once (u |out|); scores and sums in fp32, exp2 by the hardware: scores are off by less
    than 128 * 2^-24 of sum |q k| scale (below 16 in these tests) plus 2^-23 of their size,
    together below 2^-12 of each probability; values below the smallest normal number are
    off by half a step of that."""
    u = torch.finfo(dtype).eps / 2
    return (u + 2 ** -12) * mag + (2 * u + 2 ** -12) * out.abs() + torch.finfo(dtype).tiny


def turn(x, table, pos, interleaved):
    """fp32 [M,X,H] turned by the formula (each operation rounded in fp32 on its own)."""
    x = x.float().numpy()
    half = table.shape[1] // 2
    c, s = (table.numpy()[pos][:, None, i * half:(i + 1) * half] for i in (0, 1))
    y = x.copy()
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return torch.from_numpy(y)


def finite(x):
    """float32 of a 16-bit tensor; NaN 0, infinities the type's largest numbers."""
    big = torch.finfo(x.dtype).max
    return torch.nan_to_num(x.float(), nan=0.0, posinf=big, neginf=-big).numpy()


def bounds(kc, tables, ctx, cu, codes, scale):
    """codes int8 [NB,K,2,H] and scale fp32 [NB,K] (numpy), brought up to date."""
    for b in range(len(ctx)):
        n, c = int(cu[b + 1] - cu[b]), int(ctx[b])
        for i in range((c - n) // 16, -(-c // 16)) if n > 0 else ():
            blk = int(tables[b, i])
            k = finite(kc[blk, :min(16, c - 16 * i)])
            s = np.abs(k).max((0, 2)) / np.float32(127)
            one = np.where(s > 0, s, np.float32(1))[:, None]
            codes[blk, :, 0] = np.clip(np.ceil(k.max(0) / one), -127, 127)
            codes[blk, :, 1] = np.clip(np.floor(k.min(0) / one), -127, 127)
            codes[blk][s == 0] = 0
            scale[blk] = s
    return codes, scale


def choose(q, codes, scale, tables, ctx, keep, first, recent):
    """(tables, lens, blocks) of q [B,N,H]; codes int8 and scale fp32, numpy."""
    B, N, H = q.shape
    K = codes.shape[1]
    G = N // K
    out = np.full((2, B, K, keep), -1, np.int64)
    lens = np.zeros(B, np.int64)
    for b in range(B):
        nb = -(-int(ctx[b]) // 16)
        held = min(nb, keep)
        lens[b] = (held - 1) * 16 + int(ctx[b]) - (nb - 1) * 16
        ids = tables[b, :nb].numpy()
        for h in range(K):
            if nb <= keep:
                pick = np.arange(nb)
            else:
                x = finite(q[b, h * G:(h + 1) * G])
                t = np.abs(x).max(1) / np.float32(127)
                c = np.where(t[:, None] > 0, np.rint(x / np.where(t > 0, t, 1)[:, None]), 0)
                c = np.clip(c, -127, 127).astype(np.int64)
                ok = (ids >= 0) & (ids < codes.shape[0])
                top, low = (codes[np.where(ok, ids, 0), h, i].astype(np.int64) for i in (0, 1))
                dot = np.maximum(c, 0) @ top.T + np.minimum(c, 0) @ low.T
                with np.errstate(over="ignore"):
                    u = np.minimum(t[:, None] * scale[np.where(ok, ids, 0), h][None],
                                   np.finfo(np.float32).max).astype(np.float32)
                    score = (u * dot.astype(np.float32)).max(0)
                score[~ok] = -np.inf
                i = np.arange(nb)
                always = (i < first) | (i >= nb - recent)
                pick = np.sort(np.lexsort((i, -score, ~always))[:keep])
            out[0, b, h, :held] = ids[pick]
            out[1, b, h, :held] = pick
    return out[0], lens, out[1]
