"""The planner's launch at the sizes where its shared memory changes, alone in a
process of its own and from two threads at once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, threading
sys.path[:0] = [{tests!r}, {root!r}]
import torch
import gqa_decode_attention_02_gb300 as gq
from test_gpu_slots import check_plan, plan_inputs, t
dev = torch.device("cuda:0")
"""


def run(body):
    code = PROGRAM.format(tests=os.path.join(ROOT, "tests"), root=ROOT) + body
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_every_batch_size_launches_first_in_a_process(gpu):
    """Static and dynamic shared memory together pass 48 KB from 2,016 sequences on; the
    lengths stay in shared memory up to 4,096."""
    run("""
for B in (2015, 2016, 2031, 2047, 2048, 4095, 4096, 4097, 16384):
    for in_place in (False, True):
        a, tokens = plan_inputs(B, B, top=7)
        check_plan(a, tokens + 5, dev, in_place=in_place)
""")


def test_two_threads_plan_batches_of_different_sizes(gpu):
    """Neither call's shared memory takes the other's away."""
    run("""
errors = []
def work(B):
    try:
        a, tokens = plan_inputs(B, B, top=3)
        d = [t(x, dev) for x in a]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(400):
                e = [x.clone() for x in d]
                gq.plan_blocks(*e, max_tokens=tokens)
            torch.cuda.synchronize()
    except Exception as e:
        errors.append((B, repr(e)))
threads = [threading.Thread(target=work, args=(B,)) for B in (16384, 4097, 3000, 2016)]
[x.start() for x in threads]
[x.join() for x in threads]
assert not errors, errors
""")
