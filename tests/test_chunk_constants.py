"""The model of chunk attention's work shares (test_chunk_partition.py) has the kernel's own
constants."""
import os
import re

import test_chunk_partition as model

SRC = os.path.join(os.path.dirname(__file__), "..", "gqa_decode_attention_02_gb300", "csrc",
                   "attention_chunk.cu")


def constants():
    """Every `constexpr int` of the source that is made of numbers and earlier ones."""
    found = {}
    for line in re.findall(r"^constexpr int ([^;]*);", open(SRC, encoding="utf-8").read(), re.M):
        for one in line.split(","):
            name, value = (x.strip() for x in one.split("="))
            if re.fullmatch(r"[\w\s*/+<-]+", value):
                try:
                    found[name] = eval(value, {}, dict(found))
                except NameError:
                    pass
    return found


def test_constants_are_the_kernels():
    c = constants()
    assert (c["kLone"], c["kPair"], c["kStart"], c["kQuota"]) == (model.LONE, model.PAIR,
                                                                  model.START, model.QUOTA)
    assert (c["kNearLone"], c["kNearPair"]) == (model.NEAR[model.LONE], model.NEAR[model.PAIR])
    assert c["kStep"] == c["kRows"] == 128
