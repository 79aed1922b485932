"""CPU checks of the chunk, rotation and block-choice entry points: every refusal is host
logic and happens before any launch."""
import ctypes

import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from gqa_decode_attention_02_gb300 import _lib

FAKE, ODD = ctypes.c_void_p(16), ctypes.c_void_p(18)


def shape(**kw):
    d = dict(B=2, T=1, N=8, K=2, H=128, block_size=16, num_blocks=10, max_blocks_per_seq=4,
             dtype=1, scale=0.0, kv_dtype=0)
    d.update(kw)
    return ctypes.byref(_lib.Shape(**d))


def calls(L, s):
    """Every entry point that looks at a shape, with arguments that are otherwise fine."""
    return (L.gqa_chunk_attention(s, 4, FAKE, 1024, *[FAKE] * 7, 1 << 30, None, None),
            L.gqa_sparse_decode_attention(s, *[FAKE] * 7, 1 << 30, None, None),
            L.gqa_kv_block_bounds(s, *[FAKE] * 6, None, None),
            L.gqa_select_blocks(s, 2, 0, 1, *[FAKE] * 9, 1 << 30, None, None))


@pytest.mark.parametrize("kw,code", [
    (dict(kv_dtype=1), 3), (dict(kv_dtype=3), 3), (dict(dtype=7), 3), (dict(H=96), 2),
    (dict(N=7), 2), (dict(block_size=32), 2), (dict(T=0), 2), (dict(window=-1), 2),
    (dict(flags=4), 2), (dict(flags=8), 2), (dict(flags=16), 2), (dict(B=16385), 2),
    (dict(N=2 * 8193), 2), (dict(num_blocks=1 << 27), 2), (dict(num_blocks=0), 2),
])
def test_bad_shapes(cuda_lib, kw, code):
    assert calls(cuda_lib, shape(**kw)) == (code,) * 4
    assert cuda_lib.gqa_chunk_workspace_size(shape(**kw)) == 0
    assert cuda_lib.gqa_select_workspace_size(shape(**kw)) == 0


def test_no_shape(cuda_lib):
    assert calls(cuda_lib, None) == (1,) * 4


def test_chunk_refuses(cuda_lib):
    f = cuda_lib.gqa_chunk_attention

    def call(s=shape(), rows=4, stride=1024, a=None, n=1 << 30):
        a = a or [FAKE] * 8
        return f(s, rows, a[0], stride, *a[1:], n, None, None)

    assert call(rows=-1) == 2 and call(rows=1 << 31) == 2
    assert call(stride=1016) == 2 and call(stride=1028) == 2 and call(stride=1 << 39) == 2
    assert call(rows=0, a=[None] * 8) == 0 and call(s=shape(B=0), a=[None] * 8) == 0
    for i in range(7):
        a = [FAKE] * 8
        a[i] = None
        assert call(a=a) == 1
    for i in (0, 1, 2, 6):
        a = [FAKE] * 8
        a[i] = ODD
        assert call(a=a) == 4


def test_sparse_refuses(cuda_lib):
    f = cuda_lib.gqa_sparse_decode_attention
    assert f(shape(T=2), *[FAKE] * 7, 1 << 30, None, None) == 2
    assert f(shape(window=4), *[FAKE] * 7, 1 << 30, None, None) == 2
    assert f(shape(B=0), *[None] * 7, 0, None, None) == 0
    for i in range(6):
        a = [FAKE] * 7
        a[i] = None
        assert f(shape(), *a, 1 << 30, None, None) == 1


def test_rotary_refuses(cuda_lib):
    f = cuda_lib.gqa_kv_append_rotary

    def call(s=None, rows=4, p=None, strides=(1024, 256, 256), table=(8, 128), inter=0):
        p = p or [FAKE] * 10
        return f(s or shape(), rows, *p[:3], *strides, p[3], p[4], None, None, *p[5:8], *table,
                 inter, p[8], None, None)

    for i in range(9):
        p = [FAKE] * 10
        p[i] = None
        assert call(p=p) == 1, i
    for i in (0, 1, 2, 3, 4, 7, 8):
        p = [FAKE] * 10
        p[i] = ODD
        assert call(p=p) == 4, i
    for strides in ((1016, 256, 256), (1028, 256, 256), (1024, 248, 256), (1024, 256, 260)):
        assert call(strides=strides) == 2
    for table in ((0, 128), (8, 8), (8, 120), (8, 144), (8, 0), (-1, 128)):
        assert call(table=table) == 2
    assert call(rows=-1) == 2 and call(rows=0, p=[None] * 10) == 0
    assert call(s=shape(kv_dtype=9)) == 3 and call(s=shape(kv_dtype=1)) == 1  # no scales
    assert call(s=shape(H=64)) == 2  # the table turns more than a row has


def test_bounds_and_choice_refuse(cuda_lib):
    f = cuda_lib.gqa_kv_block_bounds
    for i in range(6):
        a = [FAKE] * 6
        a[i] = None
        assert f(shape(), *a, None, None) == 1
    assert f(shape(), ODD, *[FAKE] * 5, None, None) == 4
    assert f(shape(B=0), *[None] * 6, None, None) == 0
    g = cuda_lib.gqa_select_blocks
    for keep, first, recent in ((0, 0, 1), (4, 0, 0), (4, -1, 1), (4, 3, 2), (1 << 27, 0, 1),
                                (2 ** 31 - 1, 2 ** 31 - 1, 1)):
        assert g(shape(), keep, first, recent, *[FAKE] * 9, 1 << 30, None, None) == 2
    assert g(shape(T=2), 4, 0, 1, *[FAKE] * 9, 1 << 30, None, None) == 2
    assert g(shape(N=2 * 129), 4, 0, 1, *[FAKE] * 9, 1 << 30, None, None) == 2
    for i in range(8):
        a = [FAKE] * 9
        a[i] = None
        assert g(shape(), 4, 0, 1, *a, 1 << 30, None, None) == 1
    for i, want in ((0, 4), (1, 4), (8, 4)):
        a = [FAKE] * 9
        a[i] = ODD
        assert g(shape(), 4, 0, 1, *a, 1 << 30, None, None) == want
    need = cuda_lib.gqa_select_workspace_size(shape())
    assert need == 2 * 2 * 4 * 4
    assert g(shape(), 4, 0, 1, *[FAKE] * 9, need - 1, None, None) == 5
    assert g(shape(), 4, 0, 1, *[FAKE] * 8, None, need, None, None) == 5


def test_host_tensors_are_refused(cuda_lib):
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c, i = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    b, s = torch.zeros(1, 2, 2, 64, dtype=torch.int8), torch.zeros(1, 2)
    for f in (lambda: gq.kv_append_rotary(q, q, q, c, c, i, i, torch.zeros(4, 64)),
              lambda: gq.chunk_attention(q, c, c, i[:1, None], i[:1], i),
              lambda: gq.kv_block_bounds(c, i[:1, None], i[:1], i, b, s),
              lambda: gq.select_blocks(q[:1, None], b, s, i[:1, None], i[:1], 4),
              lambda: gq.sparse_decode_attention(q[:1, None], c, c, i.view(1, 2, 1), i[:1])):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            f()
