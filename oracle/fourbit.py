"""The 4-bit cached row and the block planner, restated in numpy (float64 and
Python integers) from their definitions.

Groups of 32 elements: scale s = a / 7 (a the largest magnitude) on the ue5m3
grid (byte b: the f16 number with bits b << 7), nearest even, at most 9216; codes
x / s rounded to nearest even within [-7, 7], stored as c + 8, two a byte (even
element low).  "جعل inference رخيصًا: KV cache وbatching والتكميم", quantization
section, at 4 bits and with a scale per group; block addressing of CS336 lecture
10 §"PagedAttention".
"""
from __future__ import annotations

import numpy as np

GROUP = 32
MAX_SCALE_CODE = 225  # 9216


def scale_values() -> np.ndarray:
    """float64 [256]: the ue5m3 value of every byte (inf / NaN from 248 on)."""
    b = np.arange(256)
    e, m = b >> 3, b & 7
    v = np.where(e > 0, 2.0 ** (e - 15.0) * (1 + m / 8.0), m * 2.0 ** -17)
    v[248] = np.inf
    v[249:] = np.nan
    return v


_GRID = scale_values()[: MAX_SCALE_CODE + 1]


def scale_code(a) -> np.ndarray:
    """Nearest grid code (ties to the even code) of a / 7, saturating."""
    y = np.asarray(a, np.float64) / 7.0
    y = np.minimum(y, _GRID[-1])
    hi = np.clip(np.searchsorted(_GRID, y), 1, MAX_SCALE_CODE)
    lo = hi - 1
    dl, dh = y - _GRID[lo], _GRID[hi] - y
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8)


def quantize(x) -> tuple:
    """x [..., H] -> codes uint8 [..., H/2], scales uint8 [..., H/32]."""
    x = np.asarray(x, np.float64)
    H = x.shape[-1]
    g = x.reshape(*x.shape[:-1], H // GROUP, GROUP)
    a = np.nanmax(np.where(np.isnan(g), 0.0, np.abs(g)), axis=-1)
    sc = scale_code(a)
    s = _GRID[sc][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, g / s, 0.0)
    c = np.rint(np.clip(np.where(np.isnan(y), 0.0, y), -7, 7)).astype(np.int64)
    n = (c + 8).reshape(*x.shape[:-1], H // 2, 2)
    return (n[..., 0] | (n[..., 1] << 4)).astype(np.uint8), sc


def dequantize(codes, scales) -> np.ndarray:
    """float64 [..., H] values of codes [..., H/2] and scales [..., H/32]."""
    codes = np.asarray(codes, np.int64)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1) - 8
    s = np.repeat(scale_values()[np.asarray(scales)], GROUP, axis=-1)
    return c * s


def quantize_cache(cache) -> tuple:
    """A 16-bit cache [NB,16,K,H] (torch) as 4-bit: codes [NB,K,16,H/2], scales
    [NB,K,16,H/32].  NaN slots read as zeros."""
    x = cache.double().permute(0, 2, 1, 3).numpy()
    return quantize(x)


def cache_values(codes, scales) -> np.ndarray:
    """float64 [NB,16,K,H] values of a 4-bit cache."""
    return np.ascontiguousarray(np.swapaxes(dequantize(codes, scales), 1, 2))


def plan_blocks(context_lens, new_lens, block_tables, held, free_ring, ring_state, max_tokens):
    """One step of the planner, sequence by sequence.  Returns a dict of the
    outputs, tables and ring included, and the set of reported errors (7: a
    length, 8: a block id, 12: no blocks or token entries, or the ring)."""
    ctx, held = [int(x) for x in context_lens], [int(x) for x in held]
    new = [int(x) for x in new_lens]
    tables, ring = np.array(block_tables), np.array(free_ring)
    mb, C = tables.shape[1], len(ring)
    head, count = (int(x) for x in ring_state)
    ok = 0 <= head < C and 0 <= count <= C
    errors = set() if ok else {12}
    h0, n0 = (head, count) if ok else (0, 0)
    asked_ids = asked_tokens = taken = 0
    cu, slots, pos = [0], [], []
    grants = []
    for b in range(len(ctx)):
        target = ctx[b] + new[b] if new[b] >= 0 else 0
        bad = (ctx[b] < 0 or new[b] < -1 or held[b] < 0 or held[b] > mb
               or held[b] * 16 < ctx[b] or target > 16 * mb)
        if bad:
            errors.add(7)
            cu.append(cu[-1])
            continue
        need, add = -(-target // 16), max(new[b], 0)
        more = max(0, need - held[b])
        asked_ids, asked_tokens = asked_ids + more, asked_tokens + add
        if ((more and asked_ids > n0) or (add and 0 <= max_tokens < asked_tokens)
                or (not ok and need < held[b])):
            errors.add(12)
            cu.append(cu[-1])
            continue
        grants.append((b, target, need))
        for j in range(held[b], need):
            tables[b, j] = ring[(h0 + taken) % C]
            if not 0 <= tables[b, j] < C:
                errors.add(8)
            taken += 1
        for t in range(add):
            p = ctx[b] + t
            blk = int(tables[b, p // 16])
            slots.append(blk * 16 + p % 16 if 0 <= blk < C else -1)
            pos.append(p)
        cu.append(cu[-1] + add)
    back = [int(tables[b, j]) for b, _, need in grants for j in range(need, held[b])]
    full = n0 + len(back) > C
    if full:
        errors.add(12)
    for b, target, need in grants:
        ctx[b] = target
        if not (full and need < held[b]):
            held[b] = need
    if not full:
        for i, blk in enumerate(back):
            ring[(h0 + n0 + i) % C] = blk
    state = ([(h0 + taken) % C, n0 - taken + (0 if full else len(back))] if ok
             else [head, count])
    if max_tokens >= 0:
        slots = slots + [-1] * (max_tokens - len(slots))
        pos = pos + [-1] * (max_tokens - len(pos))
    i32 = lambda x: np.asarray(x, np.int64).astype(np.int32)  # noqa: E731
    return dict(context_lens=i32(ctx), held=i32(held), ring_state=i32(state), cu_new=i32(cu),
                slots=i32(slots), positions=i32(pos), block_tables=i32(tables),
                free_ring=i32(ring)), errors
