"""CPU checks of the binding of the 4-bit, slot and planner calls: what it refuses
before a GPU is asked for, and the host logic of sizes and kernels."""
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq


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
