"""CPU checks of the binding of the 4-bit, slot and planner calls: what it refuses
before a GPU is asked for, and the host logic of sizes and kernels."""
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq


def test_tensors_of_the_host_are_refused():
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for f in (lambda: gq.kv_append_slots(k, k, c, c, s), lambda: gq.kv_gather_slots(c, c, s),
              lambda: gq.plan_blocks(s, s, s[:, None], s, s, s)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            f()


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5])
def test_more_tokens_than_an_int_counts_are_refused(n):
    """Not taken modulo 2^32."""
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_tokens"):
        gq.plan_blocks(s, s, s[:, None], s, s, s, max_tokens=n)


@pytest.mark.parametrize("H", [64, 128])
def test_engine_of_a_four_bit_cache(cuda_lib, H):
    q = torch.zeros(2, 5, 8, H, dtype=torch.float16)
    c = torch.zeros(4, 2, 16, H // 2, dtype=torch.uint8)
    bt = torch.zeros(2, 4, dtype=torch.int32)
    assert gq.attention_engine(q, c, bt, kv="int4") == "fourbit"
    assert gq.attention_engine(q, c, bt, kv="int4", window=8) == "fourbit"
    for engine in ("warp", "direct", "tmem"):
        with pytest.raises(gq.GqaError):
            gq.attention_engine(q, c, bt, kv="int4", engine=engine)
    with pytest.raises(ValueError, match="kv"):
        gq.attention_engine(q, c, bt, kv="nibble")
    if H == 128:  # what one-byte caches have
        one = torch.zeros(4, 16, 2, H, dtype=torch.uint8)
        assert gq.attention_engine(q, one, bt, kv="int8") == "warp"
        assert gq.attention_engine(q, one.half(), bt) == gq.attention_engine(q, one.half(), bt,
                                                                             kv="same")
