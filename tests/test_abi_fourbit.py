"""CPU checks of the 4-bit, slot and planner entry points: every refusal is host
logic and happens before any launch."""
import ctypes

import pytest

from gqa_decode_attention_02_gb300 import _lib

FAKE, ODD = ctypes.c_void_p(16), ctypes.c_void_p(18)


def shape(**kw):
    d = dict(B=2, T=1, N=8, K=2, H=128, block_size=16, num_blocks=10, max_blocks_per_seq=4,
             dtype=1, scale=0.0, kv_dtype=3)
    d.update(kw)
    return _lib.Shape(**d)


def args(n, **kw):
    a = [FAKE] * n
    for i, v in kw.items():
        a[int(i[1:])] = v
    return a


def test_other_entry_points_refuse_a_four_bit_shape(cuda_lib):
    s = ctypes.byref(shape())
    assert cuda_lib.gqa_kv_append(s, *args(6), None, None) == 3
    assert cuda_lib.gqa_decode_attention(s, *args(7), 1 << 30, None, None) == 3
    assert cuda_lib.gqa_decode_attention_quant(s, *args(9), 1 << 30, None, None) == 3
    assert cuda_lib.gqa_kv_append_quant(s, *args(8), None, None) == 3
    assert cuda_lib.gqa_kv_compact(ctypes.byref(shape(T=4)), *args(8), None, None) == 3


@pytest.mark.parametrize("kw,code", [
    (dict(kv_dtype=0), 3), (dict(kv_dtype=1), 3), (dict(kv_dtype=4), 3), (dict(dtype=7), 3),
    (dict(H=96), 2), (dict(N=7), 2), (dict(block_size=32), 2), (dict(T=0), 2),
    (dict(window=-1), 2), (dict(flags=4), 2), (dict(flags=8), 2), (dict(flags=16), 2),
])
def test_attention_and_append_refuse_bad_shapes(cuda_lib, kw, code):
    s = ctypes.byref(shape(**kw))
    assert cuda_lib.gqa_attention_fourbit(s, *args(7), None, FAKE, FAKE, 1 << 30, None,
                                          None) == code
    assert cuda_lib.gqa_append_attention_fourbit(s, *args(9), None, FAKE, FAKE, 1 << 30, None,
                                                 None) == code
    assert cuda_lib.gqa_kv_append_fourbit(s, *args(8), None, None) == code
    assert cuda_lib.gqa_attention_engine(s) == 0 or kw.get("kv_dtype") in (0, 1)
    if "kv_dtype" not in kw:
        assert cuda_lib.gqa_attention_workspace_size(s) == 0


def test_attention_refuses_missing_misaligned_and_combined(cuda_lib):
    f = cuda_lib.gqa_attention_fourbit
    s = ctypes.byref(shape())

    def call(a, mask=None, out=FAKE, ws=FAKE, sh=s):
        return f(sh, *a, mask, out, ws, 1 << 30, None, None)

    for i in range(7):
        assert call(args(7, **{f"_{i}": None})) == 1
    for i in range(5):
        assert call(args(7, **{f"_{i}": ODD})) == 4
    assert call(args(7), out=None) == 1 and call(args(7), out=ODD) == 4
    # a tree mask with a window, with more than 64 tokens, misaligned
    assert call(args(7), mask=FAKE, sh=ctypes.byref(shape(T=4, window=8))) == 2
    assert call(args(7), mask=FAKE, sh=ctypes.byref(shape(T=65))) == 2
    assert call(args(7), mask=ctypes.c_void_p(20), sh=ctypes.byref(shape(T=4))) == 4
    assert call([None] * 7, out=None, ws=None, sh=ctypes.byref(shape(B=0))) == 0
    assert cuda_lib.gqa_attention_fourbit(None, *args(7), None, FAKE, FAKE, 0, None, None) == 1
    assert cuda_lib.gqa_attention_engine(s) == 4


def test_slot_calls_refuse(cuda_lib):
    put, take = cuda_lib.gqa_kv_append_slots, cuda_lib.gqa_kv_gather_slots
    for kv in (0, 1, 2, 3):
        s = ctypes.byref(shape(B=0, kv_dtype=kv))
        sc = None if kv == 0 else FAKE
        good = [FAKE, FAKE, FAKE, FAKE, sc, sc, FAKE]
        back = [FAKE, FAKE, sc, sc, FAKE, FAKE, FAKE]
        assert put(s, -1, *good, None, None) == 2 and take(s, 1 << 31, *back, None, None) == 2
        assert put(s, 0, *[None] * 7, None, None) == 0
        assert take(s, 0, *[None] * 7, None, None) == 0
        for i in (0, 1, 2, 3, 6):
            a = list(good)
            a[i] = None
            assert put(s, 4, *a, None, None) == 1
            if i < 4:
                a[i] = ODD
                assert put(s, 4, *a, None, None) == 4
        if kv:
            assert put(s, 4, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, None) == 1
            assert put(s, 4, FAKE, FAKE, FAKE, FAKE, ODD, FAKE, FAKE, None, None) == 4
        else:
            assert put(s, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None) == 3
    assert put(ctypes.byref(shape(kv_dtype=9)), 4, *args(7), None, None) == 3
    assert put(ctypes.byref(shape(H=32)), 4, *args(7), None, None) == 2


def test_planner_refuses(cuda_lib):
    f = cuda_lib.gqa_plan_blocks
    good = args(12)
    assert f(16385, 4, 10, 8, *good, 0, None, None) == 2
    assert f(-1, 4, 10, 8, *good, 0, None, None) == 2
    assert f(2, 0, 10, 8, *good, 0, None, None) == 2
    assert f(2, 4, 0, 8, *good, 0, None, None) == 2
    assert f(2, 4, 10, -2, *good, 0, None, None) == 2
    assert f(16384, 1 << 18, 10, 8, *good, 0, None, None) == 2
    assert f(2, 4, 1 << 27, 8, *good, 0, None, None) == 2
    for i in range(11):
        a = list(good)
        a[i] = None
        assert f(2, 4, 10, 8, *a, 0, None, None) == 1, i
    assert f(2, 4, 10, -1, *good, 0, None, None) == 1  # a slot map without entries
    a = list(good)
    a[10] = None  # positions without slots
    assert f(2, 4, 10, -1, *a, 0, None, None) == 1


def test_compaction_refuses(cuda_lib):
    f = cuda_lib.gqa_kv_compact_fourbit
    assert f(ctypes.byref(shape(T=65)), *args(8), None, None) == 2
    assert f(ctypes.byref(shape(T=4, kv_dtype=0)), *args(8), None, None) == 3
    assert f(ctypes.byref(shape(T=4)), *args(8, _2=None), None, None) == 1
    assert f(ctypes.byref(shape(T=4)), *args(8, _0=ODD), None, None) == 4
    assert f(ctypes.byref(shape(T=1)), *[None] * 8, None, None) == 0


def test_status_string_of_the_planner_error():
    assert "free" in _lib.status_string(12) and _lib.Status.ERR_BLOCKS == 12
