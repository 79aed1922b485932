"""A launch that the runtime refuses is reported by the call that made it and by no
later one.  (The refusal: a stream whose capture has been invalidated by waiting for
it; nothing runs on the GPU.)"""
import ctypes

import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from gqa_decode_attention_02_gb300 import _lib
from helpers import small, to
from test_gpu_fourbit import four, t
from test_gpu_slots import plan_inputs

pytestmark = pytest.mark.gpu
RELAXED, UNSUPPORTED, INVALIDATED = 2, 900, 901  # capture mode; driver results

NAMES = ("plan", "append_slots", "gather_slots", "append_int4", "attention_int4", "compact",
         "append", "append_int8", "attention_warp", "attention_direct", "attention_tmem",
         "accept", "accept_cluster", "accept_sampled", "clear", "noalloc")


def calls(dev):
    """name -> a call that takes the stream, with every buffer made beforehand."""
    w = small(B=2, T=2, N=8, K=2, H=64, dtype="bf16", ctx=(40, 17), append=True, vocab=33)
    wd = to(w, dev)
    c = [t(x, dev) for x in four(w)]
    q, bt, cl, kn, vn = wd.q[0], wd.block_tables, wd.context_lens, wd.k_new[0], wd.v_new[0]
    kc, vc = wd.k_cache[0], wd.v_cache[0]
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=dev)  # noqa: E731
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    codes = [torch.zeros(kc.shape, dtype=torch.uint8, device=dev) for _ in range(2)]
    sc = [torch.zeros(kc.shape[0], 2, 16, device=dev) for _ in range(2)]
    a, tokens = plan_inputs(4, 1)
    p = [t(x, dev) for x in a]
    po = dict(context_lens_out=i32(4), held_out=i32(4), ring_state_out=i32(2), cu_new=i32(5),
              slots=i32(tokens), positions=i32(tokens))
    rows, slots = kn.reshape(4, 2, 64), torch.arange(4, dtype=torch.int32, device=dev)
    back = dict(k_out=torch.empty_like(rows), v_out=torch.empty_like(rows))
    q32 = torch.cat([q] * 8, 2)  # 32 rows of 2 tokens per KV head
    att = dict(out=torch.empty_like(q), workspace=ws)
    tmem = dict(out=torch.empty_like(q32), workspace=ws)
    path, got = i32(2, 1) + 1, dict(accepted=i32(2), next_token=i32(2))
    f4 = dict(k_scale=c[2], v_scale=c[3], kv="int4")
    probs, uni = torch.full((2, 2, 33), 1 / 33, device=dev), torch.zeros(2, 2, device=dev).double()
    dprobs = probs[:, :1].contiguous()
    table = {
        "plan": lambda s: gq.plan_blocks(*p, stream=s, **po),
        "append_slots": lambda s: gq.kv_append_slots(rows, rows, c[0], c[1], slots, stream=s, **f4),
        "gather_slots": lambda s: gq.kv_gather_slots(c[0], c[1], slots, stream=s, **back, **f4),
        "append_int4": lambda s: gq.kv_append_quant(kn, vn, *c, bt, cl, kv="int4", stream=s),
        "attention_int4": lambda s: gq.verify_attention_quant(q, *c, bt, cl, kv="int4", stream=s,
                                                              **att),
        "compact": lambda s: gq.kv_compact(c[0], c[1], bt, cl, path, i32_acc, stream=s, **f4),
        "append": lambda s: gq.kv_append(kn, vn, kc, vc, bt, cl, stream=s),
        "append_int8": lambda s: gq.kv_append_quant(kn, vn, *codes, *sc, bt, cl, stream=s),
        "attention_warp": lambda s: gq.verify_attention(q, kc, vc, bt, cl, engine="warp", stream=s,
                                                        **att),
        "attention_direct": lambda s: gq.verify_attention(q, kc, vc, bt, cl, engine="direct",
                                                          stream=s, **att),
        "attention_tmem": lambda s: gq.verify_attention(q32, kc, vc, bt, cl, engine="tmem",
                                                        stream=s, **tmem),
        "accept": lambda s: gq.accept_prefix(wd.logits, wd.draft, workspace=ws, stream=s, **got),
        "accept_cluster": lambda s: gq.accept_prefix(wd.logits, wd.draft, cluster=True, stream=s,
                                                     **got),
        "accept_sampled": lambda s: gq.accept_sampled(probs, dprobs, wd.draft, uni, stream=s, **got),
    }
    i32_acc = i32(2)

    def raw(name, *args):
        def call(s):
            stream = ctypes.c_void_p((s or torch.cuda.current_stream()).cuda_stream)
            rc = getattr(lib, name)(*args, stream)
            if rc:
                raise gq.GqaError(name, rc)
        return call

    lib, ptr = _lib.lib(), lambda x: ctypes.c_void_p(x.data_ptr())
    q1, o1 = q[:, :1].contiguous(), q[:, :1].contiguous()
    keep = (q1, o1, _lib.make_shape(q1, kc, bt, None))
    table["clear"] = raw("gqa_workspace_clear", ptr(ws), 1 << 16)
    table["noalloc"] = raw("gqa_decode_attention_noalloc", ctypes.byref(keep[2]), ptr(q1), ptr(kc),
                           ptr(vc), ptr(bt), ptr(cl), ptr(o1), None)
    table["noalloc"].keep = (keep, wd, kc, vc, bt, cl)
    table["clear"].keep = ws
    assert set(table) == set(NAMES)
    return table


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_launch_is_reported_once(gpu, name):
    table, cuda = calls(gpu), ctypes.CDLL("libcuda.so.1")
    call = table[name]
    call(None)  # attributes, occupancy and the like are asked for here
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert cuda.cuStreamBeginCapture_v2(handle, RELAXED) == 0
    try:
        assert cuda.cuStreamSynchronize(handle) == UNSUPPORTED
        with pytest.raises(gq.GqaError) as e:
            call(side)
        assert e.value.status == gq.Status.ERR_CUDA
    finally:
        assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) == INVALIDATED
    table["append"](None)  # another one, then the same, now accepted
    call(side)
    torch.cuda.synchronize()
