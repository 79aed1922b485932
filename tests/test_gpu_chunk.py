"""GPU attention of chunks of new tokens against a plain 64-bit form, within a bound derived
from its roundings."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from chunk_ref import chunk, chunk_bound

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


class Case:
    """A batch: seqs = [(new tokens, length)], made on the CPU, tables shuffled; table
    entries past a sequence's blocks and cache rows past its tokens are garbage."""

    def __init__(self, seqs, N, K, H, dtype, seed=0, spare=0, extra=3, wide=0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.seqs = dtype, seqs
        nblk = [-(-c // 16) for _, c in seqs]
        NB = sum(nblk) + extra
        ids = torch.randperm(NB, generator=g).to(torch.int32)
        self.tables = torch.full((len(seqs), max(nblk + [1]) + wide), 2 ** 31 - 1,
                                 dtype=torch.int32)
        self.kc = torch.randn(NB, 16, K, H, generator=g).to(dtype)
        self.vc = torch.randn(NB, 16, K, H, generator=g).to(dtype)
        off = 0
        used = torch.zeros(NB, 16, dtype=torch.bool)
        for b, (n, (_, c)) in enumerate(zip(nblk, seqs)):
            self.tables[b, :n] = ids[off:off + n]
            pos = torch.arange(c)
            used[self.tables[b, pos // 16].long(), pos % 16] = True
            off += n
        self.kc[~used] = float("nan")
        self.vc[~used] = float("inf")
        self.cu = torch.tensor([0] + list(np.cumsum([n for n, _ in seqs])), dtype=torch.int32)
        self.ctx = torch.tensor([c for _, c in seqs], dtype=torch.int32)
        M = int(self.cu[-1]) + spare
        self.q = torch.randn(M, N, H, generator=g).to(dtype)

    def run(self, dev, out=None, strided=False, **kw):
        q = self.q.to(dev)
        if strided:
            wide = torch.full((q.shape[0], q.shape[1] + 3, q.shape[2]), float("nan"),
                              dtype=q.dtype, device=dev)
            wide[:, 1:-2] = q
            q = wide[:, 1:-2]
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        got = gq.chunk_attention(q, *(x.to(dev) for x in (self.kc, self.vc, self.tables, self.ctx,
                                                          self.cu)), out=out, status=st, **kw)
        torch.cuda.synchronize()
        self.status = int(st.item())
        return got

    def check(self, got, window=0, scale=None, skip=()):
        want, mag = chunk(self.q, self.kc, self.vc, self.tables, self.ctx, self.cu, window, scale,
                          skip)
        over = (got.cpu().double() - want).abs() - chunk_bound(want, mag, self.dtype)
        assert torch.isfinite(got).all()
        assert float(over.max()) <= 0, f"{float(over.max())} over the bound"


EDGES = [(1, 1), (0, 5), (3, 3), (15, 15), (16, 31), (17, 17), (1, 128), (1, 129), (127, 127),
         (128, 128), (129, 300), (0, 0), (2, 257), (64, 700), (65, 65)]


@pytest.mark.parametrize("dtype,H", [(BF16, 128), (F16, 64), (F16, 128), (BF16, 64)])
@pytest.mark.parametrize("N,K", [(4, 1), (14, 2), (3, 3), (32, 8)])
def test_length_edges(gpu, dtype, H, N, K):
    c = Case(EDGES, N, K, H, dtype, seed=N, spare=5, wide=3)
    out = torch.full((c.q.shape[0], N, H), 7.0, dtype=dtype, device=gpu)
    got = c.run(gpu, out=out)
    assert c.status == 0 and got is out
    assert (out[-5:] == 7).all()  # behind the last sequence
    out[-5:] = 0
    c.check(out)


@pytest.mark.parametrize("n,ctx", [(1, 1), (1, 20000), (7, 9001), (300, 300), (700, 3000),
                                   (64, 30000), (513, 513)])
@pytest.mark.parametrize("N,K", [(8, 2), (16, 1)])
def test_one_sequence_over_all_ctas(gpu, n, ctx, N, K):
    c = Case([(n, ctx)], N, K, 128, BF16, seed=n)
    got = c.run(gpu)
    assert c.status == 0
    c.check(got)
    assert torch.equal(got, c.run(gpu))  # whichever CTA folds


@pytest.mark.parametrize("G", [5, 7, 16, 33, 64, 65, 100, 127, 128, 129, 150, 300])
def test_any_number_of_heads_per_kv_head(gpu, G):
    c = Case([(5, 5), (1, 200), (40, 333)], G, 1, 64, F16, seed=G)
    c.check(c.run(gpu))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 129, 500, 5000])
@pytest.mark.parametrize("N,K,H", [(8, 2, 128), (4, 4, 64)])
def test_windows(gpu, window, N, K, H):
    seqs = [(1, 1), (5, 700), (300, 300), (200, 1000), (1, 129), (130, 2000)]
    c = Case(seqs, N, K, H, BF16, seed=window)
    # blocks wholly below the earliest token's window are nobody's; rows below it anything
    for b, (n, ctx) in enumerate(seqs):
        low = max(0, ctx - n - window + 1)
        for j in range(low // 16):
            c.kc[c.tables[b, j].long()] = float("nan")
            c.tables[b, j] = -5
        if low % 16:
            c.kc[c.tables[b, low // 16].long(), :low % 16] = float("nan")
            c.vc[c.tables[b, low // 16].long(), :low % 16] = float("nan")
    got = c.run(gpu, window=window)
    assert c.status == 0
    # (the plain form multiplies what a row does not see by 0: finite numbers there)
    c.kc, c.vc = (torch.nan_to_num(x, nan=0.0, posinf=0.0) for x in (c.kc, c.vc))
    c.tables = c.tables.clamp(min=0)
    c.check(got, window=window)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rising_scores_rescale(gpu, dtype):
    """Every KV tile holds larger scores than the ones before it, by more than the slack."""
    c = Case([(200, 2000), (70, 1500)], 4, 2, 128, dtype, seed=5)
    c.q = c.q.abs()
    for b, (_, ctx) in enumerate(c.seqs):
        for i in range(-(-ctx // 16)):
            c.kc[c.tables[b, i].long()] = (0.02 * (i // 8)) * (1 + 0.1 * torch.rand(16, 2, 128)).to(dtype)
    got = c.run(gpu)
    c.check(got)


def test_scores_of_one_sign_and_scale(gpu):
    c = Case([(33, 900), (128, 128)], 8, 2, 64, F16, seed=8)
    c.q = -c.q.abs()
    c.kc = c.kc.abs()
    got = c.run(gpu, scale=0.3)
    c.check(got, scale=0.3)


def test_strided_queries(gpu):
    c = Case([(100, 150), (1, 77)], 6, 2, 128, BF16, seed=3)
    assert torch.equal(c.run(gpu), c.run(gpu, strided=True))


@pytest.mark.parametrize("B", [1000, 16384])
def test_many_sequences(gpu, B):
    rng = np.random.default_rng(B)
    seqs = [(int(rng.integers(0, 3)), int(rng.integers(2, 40))) for _ in range(B)]
    c = Case(seqs, 2, 1, 64, F16, seed=B)
    c.check(c.run(gpu))


def test_more_sequences_are_refused(gpu):
    c = Case([(1, 1)], 2, 1, 64, F16)
    c.tables, c.ctx = c.tables.repeat(16385, 1), c.ctx.repeat(16385)
    c.cu = torch.zeros(16386, dtype=torch.int32)
    with pytest.raises(gq.GqaError):
        c.run(gpu)


def test_bad_lengths_and_rows(gpu):
    seqs = [(4, 40), (5, 60), (3, 30), (6, 90)]
    for b, ctx, code in ((1, 3, 7), (1, -1, 7), (2, 10 ** 6, 7), (3, 2 ** 31 - 1, 7), (0, 0, 7)):
        c = Case(seqs, 4, 2, 64, BF16, seed=b)
        c.ctx[b] = ctx
        out = torch.full((18, 4, 64), 7.0, dtype=BF16, device=gpu)
        got = c.run(gpu, out=out)
        assert c.status == code
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        assert (got[rows] == 0).all()
        c.ctx[b] = seqs[b][1]
        c.check(got, skip=(b,))
    # rows that are not there, or backwards: left out, everybody else served
    for cu in ([0, 4, 9, 12, 19], [0, 4, 9, 2 ** 31 - 1, 18], [0, 4, -1, 12, 18], [-3, 4, 9, 12, 18]):
        c = Case(seqs, 4, 2, 64, BF16, seed=9)
        good = c.cu.clone()
        c.cu = torch.tensor(cu, dtype=torch.int32)
        out = torch.full((18, 4, 64), 7.0, dtype=BF16, device=gpu)
        got = c.run(gpu, out=out)
        assert c.status == 7
        keep = [b for b in range(4) if cu[b] == int(good[b]) and cu[b + 1] == int(good[b + 1])]
        c.cu = good
        want, mag = chunk(c.q, c.kc, c.vc, c.tables, c.ctx, good)
        for b in range(4):
            rows = slice(int(good[b]), int(good[b + 1]))
            if b in keep:
                over = (got[rows].cpu().double() - want[rows]).abs()
                assert (over <= chunk_bound(want[rows], mag[rows], BF16)).all()
            elif cu[b] > 18 or cu[b] < 0 or cu[b + 1] < cu[b] or cu[b + 1] > 18:
                assert (got[rows] == 7).all()


@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
def test_bad_blocks_give_zeros(gpu, bad):
    c = Case([(4, 40), (300, 900), (3, 30)], 4, 2, 128, BF16, seed=1)
    c.tables[1, 50] = bad  # positions 800 .. 815: rows from there on read it
    got = c.run(gpu)
    assert c.status == 8
    assert (got[4 + 200:304] == 0).all()
    c.tables[1, 50] = 0
    want, mag = chunk(c.q, c.kc, c.vc, c.tables, c.ctx, c.cu)
    for rows in (slice(0, 4), slice(304, 307)):
        assert ((got[rows].cpu().double() - want[rows]).abs()
                <= chunk_bound(want[rows], mag[rows], BF16)).all()
    assert torch.isfinite(got).all()


def test_bad_block_of_a_split_item(gpu):
    c = Case([(2, 20000)], 4, 1, 128, BF16, seed=2)
    c.tables[0, 600] = -7
    assert (c.run(gpu) == 0).all() and c.status == 8
    c.tables[0, 600] = 3
    assert c.run(gpu).abs().sum() > 0 and c.status == 0  # nothing is left behind


def test_no_rows_and_no_sequences(gpu):
    c = Case([(0, 5), (0, 0)], 4, 2, 64, F16)
    assert c.run(gpu).shape == (0, 4, 64) and c.status == 0
    c.q = torch.ones(3, 4, 64, dtype=F16)
    out = torch.full((3, 4, 64), 7.0, dtype=F16, device=gpu)
    assert (c.run(gpu, out=out) == 7).all() and c.status == 0
    c.tables, c.ctx, c.cu = c.tables[:0], c.ctx[:0], torch.zeros(1, dtype=torch.int32)
    assert (c.run(gpu, out=out) == 7).all()


def test_offsets_past_32_bits(gpu):
    NB, K, H = 280000, 8, 128  # 4.6e9 elements a cache
    kc = torch.empty(NB, 16, K, H, dtype=BF16, device=gpu)
    vc = torch.empty(NB, 16, K, H, dtype=BF16, device=gpu)
    c = Case([(70, 500)], 16, K, H, BF16, seed=4)
    nb = -(-500 // 16)
    far = torch.arange(NB - nb, NB, dtype=torch.int32)
    src = c.tables[0, :nb].long()
    kc[NB - nb:] = c.kc[src].to(gpu)
    vc[NB - nb:] = c.vc[src].to(gpu)
    got = gq.chunk_attention(c.q.to(gpu), kc, vc, far[None].to(gpu), c.ctx.to(gpu), c.cu.to(gpu))
    assert torch.equal(got, c.run(gpu))


def test_streams_graphs_and_shared_workspace(gpu):
    """Two graphs captured on one stream and replayed on two at once, between eager calls of
    other attention kernels that use the same cached workspace."""
    a = Case([(1, 9000), (40, 4000)], 8, 2, 128, BF16, seed=6)
    b = Case([(300, 1200)], 8, 2, 128, BF16, seed=7)
    want = [a.run(gpu), b.run(gpu)]
    dev = [[x.to(gpu) for x in (c.q, c.kc, c.vc, c.tables, c.ctx, c.cu)] for c in (a, b)]
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for d, o in zip(dev, outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                gq.chunk_attention(*d, out=o)
            graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        x = gq.chunk_attention(*dev[0])
        gq.verify_attention(a.q[:8].reshape(2, 4, 8, 128).to(gpu), *dev[0][1:3], dev[0][3],
                            dev[0][4])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert torch.equal(x, want[0])
    y = gq.chunk_attention(*dev[1], stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(y, want[1])


def test_dependent_launches(gpu):
    c = Case([(1, 3000), (130, 700)], 8, 2, 128, BF16, seed=11)
    want = c.run(gpu)
    d = [x.to(gpu) for x in (c.q, c.kc, c.vc, c.tables, c.ctx, c.cu)]
    for _ in range(30):
        got = gq.chunk_attention(*d, pdl=True)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_agrees_with_verify(gpu):
    """The same tokens through both calls: each within its roundings of the other."""
    seqs = [(5, 700), (5, 16), (5, 5), (5, 1300)]
    c = Case(seqs, 16, 2, 128, BF16, seed=12)
    got = c.run(gpu)
    out = gq.verify_attention(c.q.view(4, 5, 16, 128).to(gpu), c.kc.to(gpu), c.vc.to(gpu),
                              c.tables.to(gpu), c.ctx.to(gpu))
    want, mag = chunk(c.q, c.kc, c.vc, c.tables, c.ctx, c.cu)
    bound = chunk_bound(want, mag, BF16)
    assert ((got - out.view(20, 16, 128)).abs().cpu().double() <= 2 * bound).all()


def test_binding_refuses(gpu):
    c = Case([(4, 40), (2, 20)], 4, 2, 64, F16)
    d = [x.to(gpu) for x in (c.q, c.kc, c.vc, c.tables, c.ctx, c.cu)]

    def but(i, x):
        return [x if j == i else y for j, y in enumerate(d)]

    for a, kw in ((but(0, d[0].float()), {}), (but(0, c.q), {}), (but(0, d[0][:, ::2]), {}),
                  (but(0, d[0][..., :32]), {}), (but(1, d[1].bfloat16()), {}),
                  (but(2, d[2][:-1]), {}), (but(3, d[3].long()), {}), (but(3, d[3][:1]), {}),
                  (but(4, d[4][:1]), {}), (but(5, d[5][:2]), {}), (but(5, d[5].long()), {}),
                  (d, dict(out=torch.empty(5, 4, 64, dtype=F16, device=gpu))),
                  (d, dict(out=torch.empty(6, 4, 64, dtype=BF16, device=gpu))),
                  (d, dict(out=torch.empty(6, 4, 64, dtype=F16))),
                  (d, dict(workspace=torch.zeros(4096, dtype=torch.float32, device=gpu)))):
        with pytest.raises((ValueError, TypeError)):
            gq.chunk_attention(*a, **kw)
    for kw in (dict(workspace=torch.zeros(4096, dtype=torch.uint8, device=gpu)),
               dict(window=-1)):
        with pytest.raises(gq.GqaError):
            gq.chunk_attention(*d, **kw)
    with pytest.raises(gq.GqaError):  # heads that do not divide
        gq.chunk_attention(d[0][:, :3].contiguous(), *d[1:])


@pytest.mark.parametrize("n,ctx", [(40, 400), (40, 20000), (1, 20000)])
@pytest.mark.parametrize("what", ["q", "k", "all", "inf"])
def test_nan_scores_give_nan_rows(gpu, n, ctx, what):
    """Of items that one CTA does and of shared ones; other rows and sequences as they were."""
    c = Case([(3, 33), (n, ctx), (2, 90)], 8, 2, 128, BF16, seed=n)
    want = c.run(gpu)
    nan = torch.zeros_like(want, dtype=torch.bool)
    at = ctx - n + n // 2  # a position; tokens from there on see it
    blk, row = c.tables[1, at // 16].long(), at % 16
    if what == "q":
        c.q[3 + n // 2, 4:6] = float("nan")
        nan[3 + n // 2, 4:6] = True
    elif what == "k":
        c.kc[blk, row, 1] = float("nan")
        nan[3 + n // 2:3 + n, 4:] = True
    elif what == "all":  # no score is a number
        for b in range(-(-ctx // 16)):
            c.kc[c.tables[1, b].long(), :, 0] = float("nan")
        nan[3:3 + n, :4] = True
    else:  # q . k = inf: inf - inf in the softmax
        c.kc[blk, row, 0] = float("inf")
        c.q[3:3 + n] = c.q[3:3 + n].abs()
    got = c.run(gpu)
    assert c.status == 0
    if what == "inf":
        assert torch.isnan(got[3 + n // 2:3 + n, :4]).all()
        assert not torch.isnan(got[:3 + n // 2]).any() and not torch.isnan(got[3 + n:]).any()
        return
    assert torch.isnan(got[nan]).all()
    assert torch.equal(got[~nan], want[~nan])


def test_a_workspace_of_the_callers(gpu):
    """Of the very size, with guards behind it; its tickets zero again after every call."""
    c = Case([(1, 9000), (40, 4000)], 8, 2, 128, BF16, seed=6)
    want = c.run(gpu)
    shape = gq.Shape(B=2, T=1, N=8, K=2, H=128, block_size=16, num_blocks=c.kc.shape[0],
                     max_blocks_per_seq=c.tables.shape[1], dtype=1, scale=0.0, flags=0,
                     window=0, kv_dtype=0)
    n = gq.chunk_workspace_size(shape)
    ws = torch.zeros(n + 4096, dtype=torch.uint8, device=gpu)
    ws[n:] = 77
    for _ in range(3):
        assert torch.equal(c.run(gpu, workspace=ws[:n]), want)
    assert (ws[n:] == 77).all() and (ws[:1 << 14] == 0).all()
    with pytest.raises(gq.GqaError):
        c.run(gpu, workspace=ws[:n - 16])
    with pytest.raises((ValueError, TypeError)):
        c.run(gpu, workspace=ws[:n].cpu())
