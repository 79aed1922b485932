"""Pins of the oracle's 4-bit row and block planner: the scale grid against torch's
f16, the rounding rules against exact fractions, and the planner's invariants."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fourbit as f4


def test_scale_grid_is_f16_without_its_low_bits():
    bits = torch.arange(256, dtype=torch.int32) << 7
    ref = bits.to(torch.int16).view(torch.float16).double().numpy()
    np.testing.assert_array_equal(f4.scale_values(), ref)
    assert f4.scale_values()[f4.MAX_SCALE_CODE] == 9216.0


def _nearest(y: Fraction):
    """Nearest grid code of an exact y, ties to the even code."""
    best = None
    for c in range(f4.MAX_SCALE_CODE + 1):
        d = abs(Fraction(float(f4.scale_values()[c])) - y)
        if best is None or d < best[0] or (d == best[0] and c % 2 == 0):
            best = (d, c)
    return best[1]


def test_scale_rounding_against_fractions():
    rng = np.random.default_rng(0)
    grid = f4.scale_values()[: f4.MAX_SCALE_CODE + 1]
    mids = (grid[1:] + grid[:-1]) / 2
    pick = np.concatenate([mids[::9], np.exp(rng.uniform(-12, 11, 60)), [0.0, 1e-7, 70000.0]])
    for y in pick:
        a = float(np.float32(7 * y))
        assert f4.scale_code(a) == _nearest(Fraction(a) / 7), y


def test_codes_of_ties_ends_and_special_elements():
    x = np.zeros(32)
    x[:8] = [7.0, 0.5, 1.5, -0.5, -2.5, 3.49, -7.0, np.nan]  # scale 1
    codes, sc = f4.quantize(x)
    assert f4.scale_values()[sc[0]] == 1.0
    got = f4.dequantize(codes, sc)[:8]
    np.testing.assert_array_equal(got, [7, 0, 2, 0, -2, 3, -7, 0])
    x[:3] = [np.inf, -1e6, 64512.0]
    codes, sc = f4.quantize(x)
    np.testing.assert_array_equal(f4.dequantize(codes, sc)[:3], [64512.0, -64512.0, 64512.0])
    codes, sc = f4.quantize(np.full(32, 7 * 2.0 ** -18))  # a tie with zero: the even code
    assert sc[0] == 0 and (f4.dequantize(codes, sc) == 0).all()


@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
def test_error_is_at_most_half_a_step(size):
    """|x - c s| <= s / 2: rounding the scale down never costs more (the largest
    element has |x / s| <= 7 * 16 / 15 < 7.5)."""
    x = size * np.random.default_rng(1).normal(size=(500, 128))
    codes, sc = f4.quantize(x)
    s = np.repeat(f4.scale_values()[sc], 32, axis=-1)
    assert (np.abs(x - f4.dequantize(codes, sc)) <= s / 2).all()


def test_values_are_exact_in_both_16_bit_types():
    c = np.arange(-7, 8)[:, None] * f4.scale_values()[: f4.MAX_SCALE_CODE + 1][None]
    for dt in (torch.float16, torch.bfloat16):
        np.testing.assert_array_equal(torch.from_numpy(c).to(dt).double().numpy(), c)


def test_planner_conserves_blocks():
    """Over random steps every block is in one table's used part or in the ring."""
    rng = np.random.default_rng(5)
    B, mb, NB = 9, 20, 60
    ctx, held = np.zeros(B, int), np.zeros(B, int)
    tables, ring, state = np.full((B, mb), -1), rng.permutation(NB), np.array([7, NB])
    for _ in range(200):
        new = rng.integers(-1, 40, size=B)
        new[new > 20] = 1
        new = np.minimum(new, 16 * mb - ctx)
        got, err = f4.plan_blocks(ctx, new, tables, held, ring, state, 100)
        assert err <= {12}
        ctx, held, tables, ring, state = (got[k] for k in ("context_lens", "held", "block_tables",
                                                           "free_ring", "ring_state"))
        used = [tables[b, j] for b in range(B) for j in range(held[b])]
        free = [ring[(state[0] + i) % NB] for i in range(state[1])]
        assert sorted(used + free) == list(range(NB))
        assert (held * 16 >= ctx).all()
        live = got["slots"][got["slots"] >= 0]
        assert len(set(live.tolist())) == len(live) == got["cu_new"][-1]
        cut = rng.random(B) < 0.3  # a rejection shortens some sequences
        ctx = np.where(cut, np.maximum(0, ctx - rng.integers(0, 5, size=B)), ctx)
