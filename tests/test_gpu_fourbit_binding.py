"""GPU checks of the binding of the 4-bit, slot and planner calls: a caller's own
workspace, and tensors of the host after calls of the same sizes on the GPU."""
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from helpers import small, to
from test_gpu_attention import as_i64, random_trees
from test_gpu_fourbit import four, t
from test_gpu_slots import plan_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,N,H,ctx", [(1, 1, 4, 64, (20,)), (3, 2, 8, 128, (9000, 40, 800)),
                                         (40, 1, 8, 64, (3000,) * 40)])
def test_a_workspace_of_the_size_asked_for(gpu, B, T, N, H, ctx):
    """Cleared once, then used by every call, in graphs too: the same bits as with the
    binding's own; a byte less is refused."""
    w = small(B=B, T=T, N=N, K=2, H=H, dtype="f16", ctx=ctx, seed=B)
    wd, c = to(w, gpu), [t(x, gpu) for x in four(w)]
    q, bt, cl = wd.q[0], wd.block_tables, wd.context_lens
    n = gq.attention_workspace_size(q, c[0], bt, kv="int4")
    ws, out = torch.zeros(n, dtype=torch.uint8, device=gpu), torch.empty_like(q)
    call = lambda **kw: gq.verify_attention_quant(q, *c, bt, cl, kv="int4", **kw)  # noqa: E731
    want = call()
    for _ in range(2):
        assert torch.equal(call(workspace=ws), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    with pytest.raises(gq.GqaError) as e:
        call(workspace=ws[: n - 1])
    assert e.value.status == gq.Status.ERR_WORKSPACE


def test_workspace_size_of_one_byte_caches(gpu):
    w = small(B=2, T=1, N=8, K=2, H=128, dtype="f16", ctx=(40, 17))
    q, bt = w.q[0].to(gpu), w.block_tables.to(gpu)
    kc = torch.zeros(w.k_cache[0].shape, dtype=torch.uint8, device=gpu)
    sc = torch.ones(kc.shape[0], 2, 16, device=gpu)
    ws = torch.zeros(gq.attention_workspace_size(q, kc, bt, kv="int8"), dtype=torch.uint8,
                     device=gpu)
    a = gq.decode_attention_quant(q, kc, kc, sc, sc, bt, w.context_lens.to(gpu), workspace=ws)
    b = gq.decode_attention_quant(q, kc, kc, sc, sc, bt, w.context_lens.to(gpu))
    assert torch.equal(a, b)


def test_tensors_of_the_host_after_a_call_on_the_gpu(gpu):
    """The same sizes and types, checked before: refused all the same."""
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.arange(3, dtype=torch.int32)
    a, tokens = plan_inputs(4, 1)
    host = [torch.from_numpy(x) for x in a]
    put = lambda *x: gq.kv_append_slots(x[0], x[0], x[1], x[1].clone(), x[2])  # noqa: E731
    put(k.to(gpu), c.to(gpu), s.to(gpu))
    gq.plan_blocks(*[x.to(gpu) for x in host], max_tokens=tokens)
    for f in (lambda: put(k, c, s), lambda: gq.kv_gather_slots(c, c, s),
              lambda: gq.plan_blocks(*host, max_tokens=tokens),
              lambda: put(k, c.to(gpu), s.to(gpu)), lambda: put(k.to(gpu), c.to(gpu), s)):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("T,N,K,H,dtype", [(6, 16, 2, 128, "bf16"), (26, 8, 2, 64, "f16")])
def test_append_and_tree_verification_in_one_call(gpu, T, N, K, H, dtype):
    """gqa_append_attention_fourbit with a tree mask: the bits of the two calls, caches
    included, eagerly and from a graph."""
    ctx = (T, T + 1, 300, 1029)
    w = small(B=4, T=T, N=N, K=K, H=H, dtype=dtype, ctx=ctx, seed=T, append=True)
    wd, c = to(w, gpu), four(w)
    mask = as_i64(random_trees(4, T, seed=T)).to(gpu)
    q, kn, vn, bt, cl = wd.q[0], wd.k_new[0], wd.v_new[0], wd.block_tables, wd.context_lens
    two, one, cap = ([t(x, gpu) for x in c] for _ in range(3))
    gq.kv_append_quant(kn, vn, *two, bt, cl, kv="int4")
    want = gq.verify_attention_quant(q, *two, bt, cl, kv="int4", tree_mask=mask)
    chain = gq.verify_attention_quant(q, *two, bt, cl, kv="int4")
    assert not torch.equal(want, chain)
    fused = lambda c, **kw: gq.append_verify_attention_quant(  # noqa: E731
        q, kn, vn, *c, bt, cl, kv="int4", tree_mask=mask, **kw)
    assert torch.equal(fused(one, pdl=True), want)
    out, graph = torch.empty_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fused(cap, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for a, b, d in zip(two, one, cap):
        assert torch.equal(a, b) and torch.equal(a, d)
    with pytest.raises(ValueError, match="tree_mask"):
        gq.append_verify_attention_quant(q, kn, vn, *two, bt, cl, kv="int8", tree_mask=mask)
    with pytest.raises(gq.GqaError):  # not with a window
        fused(one, window=8)
