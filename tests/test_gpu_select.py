"""GPU bounds of cache blocks, the choice by them and decoding over what was chosen."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from chunk_ref import bounds, choose, chunk, chunk_bound
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def run_bounds(c, dev, codes, scale):
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    gq.kv_block_bounds(c.kc.to(dev), c.tables.to(dev), c.ctx.to(dev), c.cu.to(dev), codes, scale,
                       status=st)
    return int(st.item())


def buffers(NB, K, H, dev):
    return (torch.full((NB, K, 2, H), 99, dtype=torch.int8, device=dev),
            torch.full((NB, K), -1.0, device=dev))


SEQS = [(1, 1), (0, 9), (3, 3), (16, 16), (1, 17), (17, 40), (2, 17), (40, 100), (1, 640), (33, 33)]


@pytest.mark.parametrize("dtype,H,K", [(BF16, 128, 8), (F16, 64, 3), (F16, 128, 1), (BF16, 64, 2)])
def test_bounds_of_touched_blocks(gpu, dtype, H, K):
    c = Case(SEQS, K, K, H, dtype, seed=K)
    # what a block's own rows may hold
    blk = c.tables[7, 5].long()
    c.kc[blk, 1] = 0.0
    c.kc[c.tables[3, 0].long(), 2, 0, 5] = float("nan")
    c.kc[c.tables[5, 2].long(), 0, 0, 1] = float("-inf")
    c.kc[c.tables[2, 0].long(), :3] = 0.0
    c.kc[c.tables[9, 1].long(), 0] *= 1e-3
    codes, scale = buffers(c.kc.shape[0], K, H, gpu)
    assert run_bounds(c, gpu, codes, scale) == 0
    wc, ws = (x.cpu().numpy() for x in buffers(c.kc.shape[0], K, H, "cpu"))
    wc, ws = bounds(c.kc, c.tables, c.ctx, c.cu, wc, ws)
    assert np.array_equal(codes.cpu().numpy(), wc)
    assert np.array_equal(scale.cpu().numpy(), ws)


@pytest.mark.parametrize("B", [33, 700, 16384])
def test_bounds_of_many_sequences(gpu, B):
    rng = np.random.default_rng(B)
    seqs = [(int(rng.integers(0, 4)), int(rng.integers(4, 40))) for _ in range(B)]
    c = Case(seqs, 1, 1, 64, F16, seed=B)
    codes, scale = buffers(c.kc.shape[0], 1, 64, gpu)
    assert run_bounds(c, gpu, codes, scale) == 0
    wc, ws = (x.cpu().numpy() for x in buffers(c.kc.shape[0], 1, 64, "cpu"))
    wc, ws = bounds(c.kc, c.tables, c.ctx, c.cu, wc, ws)
    assert np.array_equal(codes.cpu().numpy(), wc) and np.array_equal(scale.cpu().numpy(), ws)


def test_bounds_bad_lengths_and_blocks(gpu):
    for change, code in ((lambda c: c.ctx.__setitem__(1, 2), 7), (lambda c: c.ctx.__setitem__(1, 1 << 30), 7),
                         (lambda c: c.tables.__setitem__((1, 1), -4), 8),
                         (lambda c: c.tables.__setitem__((1, 1), c.kc.shape[0]), 8)):
        c = Case([(3, 20), (20, 30), (5, 5)], 2, 2, 64, F16, seed=2)
        old = c.tables.clone()
        change(c)
        codes, scale = buffers(c.kc.shape[0], 2, 64, gpu)
        assert run_bounds(c, gpu, codes, scale) == code
        assert (scale[old[1, 1].long()] == -1).all()
        for b, i in ((0, 1), (2, 0)):
            assert (scale[old[b, i].long()] > 0).all()


def test_bounds_hold_for_every_key(gpu):
    """sum_d max(q max, q min) of the values the codes stand for >= <q, k>: the codes round
    outwards, off by their division's and product's rounding at most."""
    c = Case([(200, 200)], 2, 2, 128, BF16, seed=3)
    codes, scale = buffers(c.kc.shape[0], 2, 128, gpu)
    run_bounds(c, gpu, codes, scale)
    val = codes.cpu().double() * scale.cpu().double()[:, :, None, None]
    for i in range(12):
        blk = c.tables[0, i].long()
        k = c.kc[blk].double()
        slack = 2 ** -22 * k.abs().amax((0, 2))[:, None]
        assert (val[blk, :, 0] + slack >= k.amax(0)).all()
        assert (val[blk, :, 1] - slack <= k.amin(0)).all()


def make_select(B, N, K, H, dtype, lens, seed=0, ties=False, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    nblk = [-(-max(n, 0) // 16) for n in lens]
    NB = sum(nblk) + 2
    ids = torch.randperm(NB, generator=g).to(torch.int32)
    tables = torch.full((B, max(nblk + [1])), 2 ** 31 - 1, dtype=torch.int32)
    off = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = ids[off:off + n]
        off += n
    codes = torch.randint(-127, 128, (NB, K, 2, H), generator=g).to(torch.int8)
    codes = torch.stack([codes.amax(2), codes.amin(2)], 2)
    scale = torch.rand(NB, K, generator=g) * 0.1
    if ties:
        codes, scale = (codes.float() / 64).round().to(torch.int8), torch.full((NB, K), 0.125)
    q = torch.randn(B, 1, N, H, generator=g).to(dtype)
    if ties:
        q = q.sign()
    return q, codes, scale, tables, torch.tensor(lens, dtype=torch.int32)


def check_select(gpu, args, keep, first, recent, **kw):
    q, codes, scale, tables, ctx = args
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    got = gq.select_blocks(*(x.to(gpu) for x in args), keep, first=first, recent=recent, status=st,
                           **kw)
    want = choose(q[:, 0], codes.numpy(), scale.numpy(), tables, ctx, keep, first, recent)
    for a, b, n in zip(got, want, ("tables", "lens", "blocks")):
        assert np.array_equal(a.cpu().numpy(), b), n
    return int(st.item()), got


LENS = [1, 16, 17, 100, 159, 160, 161, 400, 1000, 4000]


@pytest.mark.parametrize("dtype,H", [(BF16, 128), (F16, 64), (F16, 128), (BF16, 64)])
@pytest.mark.parametrize("N,K", [(1, 1), (32, 8), (14, 2), (27, 3), (40, 2), (128, 1)])
def test_choice(gpu, dtype, H, N, K):
    for keep, first, recent in ((1, 0, 1), (10, 1, 2), (10, 8, 2), (10, 0, 1), (64, 3, 5)):
        args = make_select(len(LENS), N, K, H, dtype, LENS, seed=keep + N)
        assert check_select(gpu, args, keep, first, recent)[0] == 0


@pytest.mark.parametrize("keep", [5, 33, 200])
def test_ties_go_to_the_lowest_block(gpu, keep):
    args = make_select(4, 8, 2, 64, F16, [3000, 4000, 333, 16 * 201], seed=keep, ties=True)
    check_select(gpu, args, keep, 1, 1)
    q, codes, scale, tables, ctx = args
    check_select(gpu, (torch.zeros_like(q), codes, scale, tables, ctx), keep, 0, 1)
    check_select(gpu, (q, codes, torch.zeros_like(scale), tables, ctx), keep, 0, 1)
    check_select(gpu, (q, -codes.abs(), scale, tables, ctx), keep, 0, 1)  # scores below zero


@pytest.mark.parametrize("n", [9599 * 16, 9600 * 16 + 48, 30000 * 16])
def test_more_blocks_than_shared_memory_holds(gpu, n):
    args = make_select(1, 4, 1, 64, BF16, [n], seed=1)
    check_select(gpu, args, 300, 1, 2)


def test_special_queries_and_scales(gpu):
    q, codes, scale, tables, ctx = make_select(3, 4, 2, 64, BF16, [900, 800, 700], seed=4)
    q[0, 0, 0, 3] = float("nan")
    q[0, 0, 1, 4] = float("inf")
    q[1] = 3e38
    q[2, 0, 1] = 0.0
    scale[5:40] = 3e36
    check_select(gpu, (q, codes, scale, tables, ctx), 12, 1, 1)


def test_choice_bad_lengths_and_blocks(gpu):
    for bad in (0, -1, 10 ** 8):
        args = make_select(3, 4, 2, 64, F16, [900, 500, 700], seed=5)
        args[4][1] = bad
        st = torch.zeros(1, dtype=torch.int32, device=gpu)
        got = gq.select_blocks(*(x.to(gpu) for x in args), 8, status=st)
        assert int(st.item()) == 7 and int(got.lens[1]) == 0
        assert (got.tables[1] == -1).all() and (got.blocks[1] == -1).all()
        args[4][1] = 500
        want = choose(args[0][:, 0], args[1].numpy(), args[2].numpy(), args[3], args[4], 8, 1, 2)
        for b in (0, 2):
            assert np.array_equal(got.tables[b].cpu().numpy(), want[0][b])
    args = make_select(2, 4, 2, 64, F16, [900, 500], seed=6)
    args[3][0, 20], args[3][0, 21] = -3, 10 ** 6
    assert check_select(gpu, args, 8, 1, 2)[0] == 8
    assert check_select(gpu, args, 56, 1, 2)[0] == 8  # all but one: a bad one is chosen


def test_select_refusals(gpu):
    args = [x.to(gpu) for x in make_select(2, 4, 2, 64, F16, [900, 500])]
    for keep, first, recent in ((0, 0, 1), (8, 0, 0), (8, -1, 1), (8, 6, 3)):
        with pytest.raises(gq.GqaError):
            gq.select_blocks(*args, keep, first=first, recent=recent)
    q, codes, scale, tables, ctx = args
    for bad in ((q.float(), codes, scale, tables, ctx), (q, codes.float(), scale, tables, ctx),
                (q, codes, scale[:-1], tables, ctx), (q, codes, scale, tables.long(), ctx),
                (q, codes, scale, tables, ctx[:1]), (q, codes[..., :32], scale, tables, ctx),
                (q.cpu(), codes, scale, tables, ctx)):
        with pytest.raises((ValueError, TypeError)):
            gq.select_blocks(*bad, 8)
    with pytest.raises(gq.GqaError):
        gq.select_blocks(q.repeat(1, 2, 1, 1), codes, scale, tables, ctx, 8)
    with pytest.raises((ValueError, TypeError)):
        gq.select_blocks(*args, 8, tables=torch.zeros(2, 2, 9, dtype=torch.int32, device=gpu))
    with pytest.raises(gq.GqaError):
        gq.select_blocks(*args, 8, workspace=torch.zeros(16, dtype=torch.uint8, device=gpu))


@pytest.mark.parametrize("dtype,H", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("N,K", [(1, 1), (32, 8), (14, 2), (150, 1)])
@pytest.mark.parametrize("S", [1, 7, 40, 700])
def test_sparse_decode(gpu, dtype, H, N, K, S):
    """Every KV head against the plain form over its own table."""
    lens = [1, 16 * S, 16 * S - 15, max(1, 16 * (S // 2) - 3), 5]
    B, NB = len(lens), 5 * S + 3
    g = torch.Generator().manual_seed(S + N)
    kc, vc = (torch.randn(NB, 16, K, H, generator=g).to(dtype) for _ in range(2))
    kc[NB - 1], vc[NB - 1] = float("nan"), float("inf")
    tables = torch.full((B, K, S), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(K):
            tables[b, h, :-(-n // 16)] = torch.randperm(NB - 1, generator=g)[:-(-n // 16)].to(torch.int32)
    q = torch.randn(B, 1, N, H, generator=g).to(dtype)
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    got = gq.sparse_decode_attention(q.to(gpu), kc.to(gpu), vc.to(gpu), tables.to(gpu),
                                     torch.tensor(lens, dtype=torch.int32, device=gpu), status=st)
    assert int(st.item()) == 0 and got.shape == q.shape
    G = N // K
    for h in range(K):
        heads = slice(h * G, (h + 1) * G)
        want, mag = chunk(q[:, 0, heads], kc[:, :, h:h + 1], vc[:, :, h:h + 1],
                          tables[:, h].clamp(min=0), lens, list(range(B + 1)))
        over = (got[:, 0, heads].cpu().double() - want).abs() - chunk_bound(want, mag, dtype)
        assert float(over.max()) <= 0


def test_sparse_bad_tables_and_refusals(gpu):
    q = torch.ones(3, 1, 4, 64, dtype=F16, device=gpu)
    kc = torch.ones(5, 16, 2, 64, dtype=F16, device=gpu)
    tables = torch.tensor([[[0, 1], [2, 3]], [[4, -1], [1, 0]], [[1, 1], [0, 2]]],
                          dtype=torch.int32, device=gpu)
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    lens = torch.tensor([20, 20, 33], dtype=torch.int32, device=gpu)
    got = gq.sparse_decode_attention(q, kc, kc, tables, lens, status=st)[:, 0]
    assert int(st.item()) in (7, 8)  # whichever came first
    assert (got[0] == 1).all() and (got[1, :2] == 0).all() and (got[1, 2:] == 1).all()
    assert (got[2] == 0).all()
    for a in ((q, kc, kc, tables[:2], lens), (q, kc, kc, tables[:, :1].contiguous(), lens),
              (q, kc, kc, tables, lens[:2]), (q, kc, kc, tables.long(), lens),
              (q.bfloat16(), kc, kc, tables, lens), (q, kc, kc.cpu(), tables, lens)):
        with pytest.raises((ValueError, TypeError)):
            gq.sparse_decode_attention(*a)
    with pytest.raises(gq.GqaError):
        gq.sparse_decode_attention(q.view(1, 3, 4, 64), kc, kc, tables, lens)


def test_choosing_every_block_is_decode_attention(gpu):
    c = Case([(1, 333), (1, 70), (1, 1)], 8, 2, 128, BF16, seed=3)
    codes, scale = buffers(c.kc.shape[0], 2, 128, gpu)
    d = [x.to(gpu) for x in (c.kc, c.vc, c.tables, c.ctx)]
    q = c.q[:, None].to(gpu)
    ch = gq.select_blocks(q, codes, scale, *d[2:], 30)
    assert torch.equal(ch.lens, d[3])
    got = gq.sparse_decode_attention(q, d[0], d[1], ch.tables, ch.lens)
    want, mag = chunk(c.q, c.kc, c.vc, c.tables, c.ctx, c.cu)
    assert ((got[:, 0].cpu().double() - want).abs() <= chunk_bound(want, mag, BF16)).all()


def test_a_serving_run(gpu):
    """Prompts in two chunks, then decode steps over chosen blocks: plan, rotated append,
    bounds, chunk attention, choice, sparse attention -- eager, then the decode step
    captured and replayed; against the plain forms on the same caches."""
    N, K, H, NB, mb, B = 8, 2, 128, 80, 30, 3
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(1)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    tables, ring = i([[-1] * mb] * B), i(rng.permutation(NB).tolist())
    held, state, ctx = i([0] * B), i([0, NB]), i([0] * B)
    kc = torch.zeros(NB, 16, K, H, dtype=BF16, device=gpu)
    vc = torch.zeros_like(kc)
    codes = torch.zeros(NB, K, 2, H, dtype=torch.int8, device=gpu)
    scale = torch.zeros(NB, K, device=gpu)
    table = torch.from_numpy(np.concatenate([f(np.arange(600)[:, None] * 1e4 ** (-np.arange(64) / 64))
                                             for f in (np.cos, np.sin)], 1)).float().to(gpu)
    st = torch.zeros(1, dtype=torch.int32, device=gpu)

    def admit(x, new, M):
        plan = gq.plan_blocks(ctx, new, tables, held, ring, state, max_tokens=M, in_place=True,
                              status=st)
        q = gq.kv_append_rotary(x[:, :N], x[:, N:N + K], x[:, N + K:], kc, vc, plan.slots,
                                plan.positions, table, status=st)
        gq.kv_block_bounds(kc, tables, ctx, plan.cu_new, codes, scale, status=st)
        return q, plan

    def rows(M):
        return torch.randn(M, N + 2 * K, H, generator=g).bfloat16().to(gpu)

    for new in ([200, 1, 37], [130, 300, 0]):
        M = sum(new) + 4
        q, plan = admit(rows(M), i(new), M)
        out = gq.chunk_attention(q, kc, vc, tables, ctx, plan.cu_new, status=st)
        assert int(st.item()) == 0
        want, mag = chunk(q.cpu(), kc.cpu(), vc.cpu(), tables.cpu().clamp(min=0), ctx.cpu(),
                          plan.cu_new.cpu())
        assert ((out.cpu().double() - want).abs() <= chunk_bound(want, mag, BF16)).all()
    assert ctx.tolist() == [330, 301, 37]
    x, one = rows(B), i([1] * B)

    def step():
        q, plan = admit(x, one, B)
        ch = gq.select_blocks(q[:, None], codes, scale, tables, ctx, 8, status=st)
        return q, ch, gq.sparse_decode_attention(q[:, None], kc, vc, ch.tables, ch.lens, status=st)

    def check(q, ch, out):
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        tb = tables.cpu()
        want = choose(q.cpu(), codes.cpu().numpy(), scale.cpu().numpy(), tb, ctx.cpu(), 8, 1, 2)
        for a, b in zip(ch, want):
            assert np.array_equal(a.cpu().numpy(), b)
        wc, ws = bounds(kc.cpu(), tb, ctx.cpu(), [sum(ctx.tolist()[:b]) for b in range(B + 1)],
                        codes.cpu().numpy().copy(), scale.cpu().numpy().copy())
        assert np.array_equal(codes.cpu().numpy(), wc) and np.array_equal(scale.cpu().numpy(), ws)
        for h in range(K):
            s = slice(h * N // K, (h + 1) * N // K)
            w, m = chunk(q.cpu()[:, s], kc.cpu()[:, :, h:h + 1], vc.cpu()[:, :, h:h + 1],
                         ch.tables.cpu()[:, h].clamp(min=0), ch.lens.cpu(), list(range(B + 1)))
            assert ((out[:, 0, s].cpu().double() - w).abs() <= chunk_bound(w, m, BF16)).all()

    check(*step())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(20):
        x.copy_(rows(B))
        graph.replay()
        check(*captured)
    assert ctx.tolist() == [351, 322, 58]


def test_streams_graphs_and_dependent_launches(gpu):
    """Two graphs of bounds, choice and attention captured on one stream, replayed on two at
    once between eager calls; then the three as dependent launches."""
    cases = [Case([(1, 5000), (1, 900), (1, 16)], 8, 2, 128, BF16, seed=21),
             Case([(1, 12000), (1, 300)], 8, 2, 128, BF16, seed=22)]
    sets = []
    for c in cases:
        d = [x.to(gpu) for x in (c.kc, c.vc, c.tables, c.ctx, c.cu)]
        codes, scale = buffers(c.kc.shape[0], 2, 128, gpu)
        whole = torch.cumsum(torch.cat([c.ctx.new_zeros(1), c.ctx]), 0).to(torch.int32).to(gpu)
        gq.kv_block_bounds(d[0], d[2], d[3], whole, codes, scale)
        sets.append((c.q[:, None].to(gpu), d, codes, scale))

    def step(q, d, codes, scale, **kw):
        gq.kv_block_bounds(d[0], d[2], d[3], d[4], codes, scale, **kw)
        ch = gq.select_blocks(q, codes, scale, d[2], d[3], 40, **kw)
        return ch, gq.sparse_decode_attention(q, d[0], d[1], ch.tables, ch.lens, **kw)

    def same(a, b):
        return all(torch.equal(x, y) for x, y in zip((*a[0], a[1]), (*b[0], b[1])))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    side, graphs, held = torch.cuda.Stream(), [], []
    with torch.cuda.stream(side):
        for s in sets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                held.append(step(*s))
            graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        x = step(*sets[0])
    torch.cuda.synchronize()
    assert same(held[0], want[0]) and same(held[1], want[1]) and same(x, want[0])
    for _ in range(20):
        x = step(*sets[1], pdl=True)
    torch.cuda.synchronize()
    assert same(x, want[1])
    x = step(*sets[0], stream=streams[0])
    streams[0].synchronize()
    assert same(x, want[0])


def test_scratch_of_the_callers(gpu):
    args = [x.to(gpu) for x in make_select(2, 8, 2, 64, F16, [4000, 333])]
    want = gq.select_blocks(*args, 8)
    n = 2 * 2 * args[3].shape[1] * 4
    ws = torch.full((n + 256,), 77, dtype=torch.uint8, device=gpu)
    got = gq.select_blocks(*args, 8, workspace=ws[:n])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (ws[n:] == 77).all()
    with pytest.raises(gq.GqaError):
        gq.select_blocks(*args, 8, workspace=ws[:n - 4])


def test_more_places_than_the_table_is_wide(gpu):
    args = make_select(3, 8, 2, 64, F16, [400, 333, 1])
    check_select(gpu, args, args[3].shape[1] + 9, 4, 3)


@pytest.mark.parametrize("N,K,H", [(4, 1, 128), (128, 1, 128), (9, 1, 64)])
def test_scores_in_shared_memory_or_not(gpu, N, K, H):
    """Around the number of blocks whose scores fit behind the queries' codes."""
    most = (39 * 1024 - (N + 7) // 8 * 8 * (2 * H + 4)) // 4
    for nb in (most - 1, most, most + 1):
        args = make_select(1, N, K, H, BF16, [nb * 16 - 3], seed=nb)
        assert check_select(gpu, args, 70, 2, 3)[0] == 0
    args = make_select(3, N, K, H, BF16, [most * 16 + 16, most * 16, 900], seed=5)
    assert check_select(gpu, args, 33, 0, 1)[0] == 0
