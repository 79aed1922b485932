"""GPU 4-bit cache: the append bit for bit, attention within a bound derived from
its roundings, compaction, and the calls together.

The bound on |out - exact|, exact being fp64 attention over the cached values c * s
(exact numbers of either 16-bit type, so the fp64 oracle reads the same cache):
  * the output's rounding, half a step: 2^-11 (f16) or 2^-8 (bf16) of |out|;
  * probabilities rounded to f16 before the product with V: 2^-11 of
    A = sum p |V|, and 2^-25 * max|V| for each of the n positions below f16's normal
    range (the row's largest exponent reference itself contributes a 1 to the sum);
  * scores: fp32 sums of H exact products in at most H/16 + 4 roundings of 2^-23,
    with sum |q k| * scale * log2(e) <= 40 for these inputs: below 2^-15 of the
    probability, taken twice (numerator and sum), plus ex2.approx (2^-22) and
    the fp32 accumulation of at most 2^13 terms, 2^-11 / 16 of A together.
"""
import numpy as np
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
import oracle
from helpers import small, to
from oracle import fourbit as f4
from test_gpu_attention import as_i64, random_trees

pytestmark = pytest.mark.gpu
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def t(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def four(w):
    """(k codes, v codes, k scales, v scales) of a workload's 16-bit caches."""
    kc, ks = f4.quantize_cache(w.k_cache[0])
    vc, vs = f4.quantize_cache(w.v_cache[0])
    return kc, vc, ks, vs


def exact(w, c, **kw):
    """(fp64 out, bound on the error) over a 4-bit cache c."""
    kc, vc, ks, vs = c
    dt = w.torch_dtype
    bits = lambda x: torch.from_numpy(x).to(dt)  # noqa: E731  exact
    k, v = f4.cache_values(kc, ks), f4.cache_values(vc, vs)
    k, v = np.nan_to_num(k, posinf=0, neginf=0), np.nan_to_num(v, posinf=0, neginf=0)
    tables = kw.pop("tables", w.block_tables)
    ref, err = oracle.attention(w.q[0], bits(k), bits(v), tables, w.context_lens, w.dtype, **kw)
    A, _ = oracle.attention(w.q[0], bits(k), bits(np.abs(v)), tables, w.context_lens, w.dtype,
                            **kw)
    assert (err == 0).all()
    n = int(w.context_lens.max())
    inner = A * (2.0 ** -11 * 17 / 16 + 2.0 ** -14) + n * 2.0 ** -25 * np.abs(v).max()
    return ref, inner + HALF[w.dtype] * (np.abs(ref) + inner) + 2.0 ** -24


def check(out, ref, lim, what=""):
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bad = np.abs(got - ref) > lim
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - ref) / lim).max()))


def attend(w, c, dev, *, window=0, mask=None, tables=None, **kw):
    wd = to(w, dev)
    fn = gq.decode_attention_quant if w.T == 1 else gq.verify_attention_quant
    if mask is not None:
        kw["tree_mask"] = as_i64(mask).to(dev)
        fn = gq.verify_attention_quant
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    out = fn(wd.q[0], *(t(x, dev) for x in c),
             wd.block_tables if tables is None else t(tables, dev), wd.context_lens, kv="int4",
             window=window, status=st, **kw)
    torch.cuda.synchronize()
    return out, int(st.item())


@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 5])
def test_append_is_bit_exact(gpu, H, dtype, T):
    ctx = tuple(max(c, T) for c in (1, 3, 16, 17, 32, 33, 500))
    w = small(B=len(ctx), T=T, N=6, K=3, H=H, dtype=dtype, ctx=ctx, seed=H + T, append=True)
    row = torch.zeros(H)
    row[:8] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -3.5, 6.5, -7.0])  # ties at scale 1
    row[32:40] = torch.tensor([1e-5, -2e-5, 3e-7, 0, 0, 0, 0, 0])        # below the grid
    w.k_new[0][0, 0, 0] = row.to(w.torch_dtype)
    row[32:36] = torch.tensor([60000.0, -65000.0, float("inf"), 3.0])    # saturation
    w.v_new[0][-1, T - 1, 2] = row.to(w.torch_dtype)
    w.k_new[0][1, 0, 1] = 0.0
    w.v_new[0][2, 0, 1, 5] = float("nan")
    # every scale binade: rows of one size each
    w.k_new[0][3, 0] *= 2.0 ** -9
    w.v_new[0][3, 0] *= 300.0
    rng = np.random.default_rng(0)
    NB, K = w.num_blocks, w.K
    want = [rng.integers(0, 256, s, dtype=np.uint8) for s in
            ((NB, K, 16, H // 2),) * 2 + ((NB, K, 16, H // 32),) * 2]
    kc, vc, ks, vs = (t(x, gpu) for x in want)
    for b, c in enumerate(ctx):
        for i in range(T):
            pos = c - T + i
            blk, r = int(w.block_tables[b, pos // 16]), pos % 16
            for new, codes, sc in ((w.k_new[0], want[0], want[2]), (w.v_new[0], want[1], want[3])):
                codes[blk, :, r], sc[blk, :, r] = f4.quantize(new[b, i].double().numpy())
    wd = to(w, gpu)
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    gq.kv_append_quant(wd.k_new[0], wd.v_new[0], kc, vc, ks, vs, wd.block_tables,
                       wd.context_lens, kv="int4", status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for got, ref in zip((kc, vc, ks, vs), want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("T,N,K,H,dtype", [
    (1, 14, 2, 64, "f16"), (1, 32, 8, 128, "bf16"), (1, 3, 3, 128, "f16"), (1, 16, 1, 128, "bf16"),
    (1, 9, 1, 64, "bf16"), (5, 64, 8, 128, "bf16"), (3, 16, 2, 64, "f16"), (2, 8, 1, 128, "f16"),
    (8, 16, 4, 64, "bf16"), (7, 20, 4, 128, "f16")])
def test_attention_matches_oracle(gpu, T, N, K, H, dtype):
    """Lengths of one token to several thousand, pages that end inside a tile,
    1 to 48 query rows per KV head (one to three row chunks)."""
    ctx = tuple(max(c, T) for c in (1, 2, 15, 16, 17, 31, 33, 295, 1029, 4097))
    w = small(B=len(ctx), T=T, N=N, K=K, H=H, dtype=dtype, ctx=ctx, seed=N + T + K + H)
    c = four(w)
    ref, lim = exact(w, c)
    out, st = attend(w, c, gpu)
    assert st == 0
    check(out, ref, lim)
    again, _ = attend(w, c, gpu)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # deterministic


@pytest.mark.parametrize("B,N,K,ctx", [(300, 4, 2, 40), (700, 2, 1, 7), (1, 8, 8, 20000),
                                       (2, 4, 1, 16384), (40, 16, 8, 1000)])
def test_attention_over_many_and_long_segments(gpu, B, N, K, ctx):
    """More segments than thread blocks; segments cut into many pieces."""
    rng = np.random.default_rng(B)
    lens = tuple(int(x) for x in rng.integers(max(1, ctx - 9), ctx + 1, size=B))
    w = small(B=B, T=1, N=N, K=K, H=64, dtype="bf16", ctx=lens, seed=B + ctx)
    c = four(w)
    ref, lim = exact(w, c)
    out, st = attend(w, c, gpu)
    assert st == 0
    check(out, ref, lim)


@pytest.mark.parametrize("T,N,H", [(1, 3, 64), (1, 4, 128), (2, 8, 64), (3, 8, 64), (3, 8, 128)])
def test_one_segment_over_the_whole_gpu(gpu, T, N, H):
    """One KV head of one sequence: more pieces than a warp has lanes, 3 to 24 rows
    each.  A page that no cache has, in one piece only, gives zeros."""
    w = small(B=1, T=T, N=N, K=1, H=H, dtype="bf16", ctx=(90005,), seed=T * N + H)
    c = four(w)
    ref, lim = exact(w, c)
    out, st = attend(w, c, gpu)
    assert st == 0
    check(out, ref, lim)
    tables = w.block_tables.numpy().copy()
    tables[0, 3500] = w.num_blocks
    out, st = attend(w, c, gpu, tables=tables)
    assert st == 8 and not out.any()


@pytest.mark.parametrize("T,N,K,H,dtype", [(1, 32, 8, 128, "bf16"), (5, 40, 4, 64, "f16"),
                                           (3, 16, 2, 128, "f16")])
@pytest.mark.parametrize("W", [1, 15, 17, 100, 1024])
def test_windows_ignore_what_lies_outside(gpu, T, N, K, H, dtype, W):
    """Below the windows and past the lengths: any code, NaN scales, and table
    entries of freed blocks."""
    ctx = tuple(max(c, T) for c in (1, 2, 16, 17, 31, 295, 1029, 4097))
    w = small(B=len(ctx), T=T, N=N, K=K, H=H, dtype=dtype, ctx=ctx, seed=W + 7 * T + N)
    c = [x.copy() for x in four(w)]
    ref, lim = exact(w, c, window=W)
    tables = w.block_tables.numpy().copy()
    rng = np.random.default_rng(W)
    for b, n in enumerate(ctx):
        first = max(0, n - T - W + 1)
        for pos in list(range(first)) + list(range(n, (n + 15) // 16 * 16)):
            blk, r = tables[b, pos // 16], pos % 16
            c[0][blk, :, r] = rng.integers(0, 256, c[0][blk, :, r].shape)
            c[1][blk, :, r] = rng.integers(0, 256, c[1][blk, :, r].shape)
            c[2][blk, :, r], c[3][blk, :, r] = 255, 255
        tables[b, : first // 16] = 2**31 - 1
    out, st = attend(w, c, gpu, window=W, tables=tables)
    assert st == 0
    check(out, ref, lim)


@pytest.mark.parametrize("T,N,K,H,dtype", [(6, 64, 8, 128, "bf16"), (26, 64, 8, 128, "bf16"),
                                           (4, 14, 2, 64, "f16"), (64, 4, 4, 64, "f16")])
def test_trees_match_oracle(gpu, T, N, K, H, dtype):
    ctx = (T, T + 1, 16 + T, 300, 1029)
    w = small(B=len(ctx), T=T, N=N, K=K, H=H, dtype=dtype, ctx=ctx, seed=11 * T + N)
    c = four(w)
    m = random_trees(len(ctx), T, seed=T + 2)
    ref, lim = exact(w, c, tree_mask=m)
    out, st = attend(w, c, gpu, mask=m)
    assert st == 0
    check(out, ref, lim)
    chain = np.array([[(1 << i) - 1 for i in range(T)]] * len(ctx), dtype=np.uint64)
    a, _ = attend(w, c, gpu, mask=chain)
    b, _ = attend(w, c, gpu)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 1.0, 2.0 ** 20, 2.0 ** 100])
def test_queries_of_any_size(gpu, size):
    """bf16 queries far outside f16's range, with a score scale that undoes it."""
    w = small(B=3, T=1, N=8, K=2, H=128, dtype="bf16", ctx=(5, 40, 333), seed=5)
    w.q[0] = (w.q[0].double() * size).to(torch.bfloat16)
    w.q[0][1, 0, 3] = 0.0
    scale = float(128 ** -0.5 / size)
    c = four(w)
    ref, lim = exact(w, c, scale=scale)
    out, st = attend(w, c, gpu, scale=scale)
    assert st == 0
    check(out, ref, lim, size)


def test_large_scales_and_growing_scores(gpu):
    """Rows near the end of the cached range, and scores that keep growing along
    the sequence (the running maximum is raised again and again)."""
    w = small(B=2, T=1, N=4, K=2, H=64, dtype="f16", ctx=(900, 901), seed=6)
    for b in range(2):
        for pos in range(900):
            blk, r = int(w.block_tables[b, pos // 16]), pos % 16
            w.k_cache[0][blk, r] = (w.q[0][b, 0, ::2] * (0.02 * pos)).to(torch.float16)
            w.v_cache[0][blk, r] *= 12000.0
    c = four(w)
    assert (c[3] >= 210).any()
    ref, lim = exact(w, c)
    # scores reach 0.02 * 900 * |q|^2 / 8 * log2(e) < 500: 12 times the bound's 40
    out, st = attend(w, c, gpu)
    check(out, ref, lim * 2)


@pytest.mark.parametrize("T,N,K,H,dtype", [(1, 32, 8, 128, "bf16"), (4, 14, 2, 64, "f16")])
def test_append_and_attention_in_one_call(gpu, T, N, K, H, dtype):
    """The same bits as the two calls, with and without dependent launch, on a
    stream of its own and replayed from a graph."""
    ctx = tuple(max(c, T) for c in (1, 16, 17, 33, 300, 2049))
    w = small(B=len(ctx), T=T, N=N, K=K, H=H, dtype=dtype, ctx=ctx, seed=T + N, append=True)
    c = four(w)
    wd = to(w, gpu)
    fused = gq.append_decode_attention_quant if T == 1 else gq.append_verify_attention_quant
    plain = gq.decode_attention_quant if T == 1 else gq.verify_attention_quant
    pair = [t(x, gpu) for x in c]
    gq.kv_append_quant(wd.k_new[0], wd.v_new[0], *pair, wd.block_tables, wd.context_lens,
                       kv="int4")
    want = plain(wd.q[0], *pair, wd.block_tables, wd.context_lens, kv="int4")
    torch.cuda.synchronize()
    ref, lim = exact(w, [x.cpu().numpy() for x in pair])
    check(want, ref, lim)
    side = torch.cuda.Stream()
    for kw in (dict(), dict(pdl=True, early_kv=True), dict(stream=side)):
        one = [t(x, gpu) for x in c]
        torch.cuda.synchronize()
        got = fused(wd.q[0], wd.k_new[0], wd.v_new[0], *one, wd.block_tables, wd.context_lens,
                    kv="int4", **kw)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for a, b in zip(one, pair):
            assert torch.equal(a, b)
    one = [t(x, gpu) for x in c]
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fused(wd.q[0], wd.k_new[0], wd.v_new[0], *one, wd.block_tables, wd.context_lens,
              kv="int4", out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_graphs_captured_on_one_stream_replay_together(gpu):
    """Each graph owns its workspace: replayed at the same time on two streams,
    long enough to overlap, neither disturbs the other's split segments."""
    ws, outs, graphs, wants = [], [], [], []
    for i in range(2):
        w = small(B=4, T=1, N=8, K=2, H=64, dtype="bf16", ctx=(9000, 8000, 5000, 4000), seed=i)
        wd, c = to(w, gpu), [t(x, gpu) for x in four(w)]
        wants.append(gq.decode_attention_quant(wd.q[0], *c, wd.block_tables, wd.context_lens,
                                               kv="int4"))
        ws.append((wd, c))
        outs.append(torch.empty_like(wants[-1]))
    torch.cuda.synchronize()
    cap = torch.cuda.Stream()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        wd, c = ws[i]
        with torch.cuda.graph(g, stream=cap):
            for _ in range(20):
                gq.decode_attention_quant(wd.q[0], *c, wd.block_tables, wd.context_lens,
                                          kv="int4", out=outs[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 5])
def test_blocks_whose_bytes_lie_beyond_32_bits(gpu, T):
    """Block ids so high that code offsets pass 2^32: the same bits as the same rows
    in a small cache, for attention, append and rows by slot."""
    w = small(B=2, T=T, N=8, K=8, H=128, dtype="bf16", ctx=(700, 41), seed=21, append=True)
    c, wd = four(w), to(w, gpu)
    NB, high = w.num_blocks, 600_000
    big = [torch.empty((high,) + x.shape[1:], dtype=torch.uint8, device=gpu) for x in c]
    assert high * 8 * 1024 > 2 ** 32
    for x, y in zip(big, c):
        x[high - NB:] = t(y, gpu)
    lowc = [t(x, gpu) for x in c]
    used = torch.arange(w.max_blocks, device=gpu)[None] < (wd.context_lens[:, None] + 15) // 16
    tables = torch.where(used, wd.block_tables + (high - NB), wd.block_tables)
    fn = gq.append_decode_attention_quant if T == 1 else gq.append_verify_attention_quant
    args = (wd.q[0], wd.k_new[0], wd.v_new[0])
    a = fn(*args, *lowc, wd.block_tables, wd.context_lens, kv="int4")
    b = fn(*args, *big, tables, wd.context_lens, kv="int4")
    assert torch.equal(a, b)
    for x, y in zip(big, lowc):
        assert torch.equal(x[high - NB:], y)
    slots = torch.arange((high - NB) * 16, high * 16, device=gpu, dtype=torch.int32)
    sc = lambda z: dict(k_scale=z[2], v_scale=z[3], kv="int4")  # noqa: E731
    rows = gq.kv_gather_slots(big[0], big[1], slots, **sc(big))
    want = gq.kv_gather_slots(lowc[0], lowc[1], slots - (high - NB) * 16, **sc(lowc))
    assert torch.equal(rows[0], want[0]) and torch.equal(rows[1], want[1])
    gq.kv_append_slots(rows[1], rows[0], big[0], big[1], slots, **sc(big))
    gq.kv_append_slots(want[1], want[0], lowc[0], lowc[1], slots - (high - NB) * 16, **sc(lowc))
    for x, y in zip(big, lowc):
        assert torch.equal(x[high - NB:], y)


def test_device_errors_zero_the_sequence_and_leave_the_others(gpu):
    w = small(B=4, T=2, N=8, K=2, H=128, dtype="bf16", ctx=(40, 700, 33, 5), seed=8)
    c = four(w)
    good, _ = attend(w, c, gpu)
    w.block_tables[1, 20] = 10 ** 6
    out, st = attend(w, c, gpu)
    assert st == 8 and (out[1] == 0).all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[2:], good[2:])
    w.block_tables[1, 20] = -3
    assert attend(w, c, gpu)[1] == 8
    w.context_lens[2], w.context_lens[3] = 1, 16 * w.max_blocks + 1
    out, st = attend(w, c, gpu)
    assert st in (7, 8) and (out[1:] == 0).all() and torch.equal(out[0], good[0])
    assert attend(w, c, gpu)[1] in (7, 8)  # the workspace is in order after it


def test_workspace_is_left_zero_and_shared_with_the_other_kernels(gpu):
    w = small(B=2, T=1, N=8, K=2, H=128, dtype="bf16", ctx=(3000, 2000), seed=9)
    c, wd = four(w), to(w, gpu)
    q, bt, cl = wd.q[0], wd.block_tables, wd.context_lens
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=gpu)
    a = gq.decode_attention(q, wd.k_cache[0], wd.v_cache[0], bt, cl, workspace=ws, engine="warp")
    out, _ = attend(w, c, gpu, workspace=ws)
    b = gq.decode_attention(q, wd.k_cache[0], wd.v_cache[0], bt, cl, workspace=ws, engine="warp")
    out2, _ = attend(w, c, gpu, workspace=ws)
    assert torch.equal(a, b) and torch.equal(out, out2)
    assert not ws[: 1 << 18].any()
    with pytest.raises(gq.GqaError) as e:
        attend(w, c, gpu, workspace=ws[:1024])
    assert e.value.status == gq.Status.ERR_WORKSPACE


@pytest.mark.parametrize("H", [64, 128])
def test_compaction_moves_the_branch(gpu, H):
    T, ctx = 6, (6, 40, 17, 300)
    w = small(B=4, T=T, N=4, K=2, H=H, dtype="f16", ctx=ctx, seed=12)
    c = four(w)
    path = np.array([[1, 3, 5, -1, -1], [2, 4, -1, -1, -1], [-1] * 5, [1, 2, 3, 4, 5]], np.int32)
    acc = np.array([3, 2, 0, 5], np.int32)
    cl = np.array([n - (T - 1 - a) for n, a in zip(ctx, acc)], np.int32)
    want = [x.copy() for x in c]
    for b in range(4):
        base = int(cl[b]) - 1 - int(acc[b])
        place = lambda p: (int(w.block_tables[b, p // 16]), p % 16)  # noqa: E731
        for x, src in zip(want, c):
            for j in range(acc[b]):
                (db, dr), (sb, sr) = place(base + 1 + j), place(base + int(path[b, j]))
                x[db, :, dr] = src[sb, :, sr]
    kc, vc, ks, vs = (t(x, gpu) for x in c)
    gq.kv_compact(kc, vc, w.block_tables.to(gpu), t(cl, gpu), t(path, gpu), t(acc, gpu),
                  k_scale=ks, v_scale=vs, kv="int4")
    torch.cuda.synchronize()
    for got, ref in zip((kc, vc, ks, vs), want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)


def test_scale_given_as_a_tensor(gpu):
    """Its value at each call counts, also after it changed in place."""
    w = small(B=2, T=1, N=4, K=2, H=64, dtype="f16", ctx=(40, 17), seed=3)
    wd, c = to(w, gpu), [t(x, gpu) for x in four(w)]
    f = lambda s: gq.decode_attention_quant(wd.q[0], *c, wd.block_tables,  # noqa: E731
                                            wd.context_lens, kv="int4", scale=s)
    x = torch.tensor(0.25)
    assert torch.equal(f(x), f(0.25))
    x.fill_(0.5)
    assert torch.equal(f(x), f(0.5)) and not torch.equal(f(0.5), f(0.25))


def test_binding_refuses(gpu):
    w = small(B=2, T=1, N=8, K=2, H=128, dtype="bf16", ctx=(5, 40), seed=13)
    kc, vc, ks, vs = (t(x, gpu) for x in four(w))
    wd = to(w, gpu)
    q, bt, cl = wd.q[0], wd.block_tables, wd.context_lens

    def call(q=q, kc=kc, vc=vc, ks=ks, vs=vs, bt=bt, cl=cl, **kw):
        return gq.decode_attention_quant(q, kc, vc, ks, vs, bt, cl, kv="int4", **kw)

    for kw in (dict(q=q.float()), dict(q=q[..., :64].contiguous()), dict(ks=ks.float()),
               dict(ks=ks[..., :2].contiguous()), dict(vc=vc[:3].contiguous()),
               dict(cl=cl[:1].contiguous()), dict(bt=bt[:1].contiguous()),
               dict(kc=kc.transpose(1, 2)), dict(q=q.cpu()), dict(out=torch.empty_like(q[:1]))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(gq.GqaError):  # decode is one token
        call(q=torch.cat([q, q], 1))
