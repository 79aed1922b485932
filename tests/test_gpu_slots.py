"""GPU rows by slot: every cache kind, against the appends by block table and the
oracle's rows (bit for bit), and the planner against its restatement."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
import oracle
from helpers import small, to
from oracle import fourbit as f4
from test_gpu_fourbit import check, exact, t

pytestmark = pytest.mark.gpu


def caches(kv, NB, K, H, dtype, dev, fill=0x5A):
    if kv == "same":
        kc = torch.full((NB, 16, K, H), 3.0, dtype=dtype, device=dev)
        return [kc, kc.clone()], [None, None]
    if kv == "int4":
        kc = torch.full((NB, K, 16, H // 2), fill, dtype=torch.uint8, device=dev)
        ks = torch.full((NB, K, 16, H // 32), fill, dtype=torch.uint8, device=dev)
    else:
        kc = torch.full((NB, 16, K, H), fill, dtype=torch.uint8, device=dev)
        ks = torch.full((NB, K, 16), -1.0, dtype=torch.float32, device=dev)
    return [kc, kc.clone()], [ks, ks.clone()]


@pytest.mark.parametrize("kv", ["same", "int8", "e4m3", "int4"])
@pytest.mark.parametrize("H,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("M,K", [(1, 1), (37, 3), (1000, 8)])
def test_rows_land_where_the_block_table_append_puts_them(gpu, kv, H, dtype, M, K):
    NB = M // 16 + 2
    rng = np.random.default_rng(M + H)
    place = rng.permutation(NB * 16)[:M].astype(np.int32)
    g = torch.Generator().manual_seed(M)
    k = torch.randn(M, K, H, generator=g).to(dtype)
    v = (torch.randn(M, K, H, generator=g) * 5).to(dtype)
    k[0, 0] = 0.0
    slots = place.copy()
    slots[::5] = -1
    (kc, vc), (ks, vs) = caches(kv, NB, K, H, dtype, gpu)
    (wk, wv), (wks, wvs) = caches(kv, NB, K, H, dtype, gpu)
    # by block table: one sequence per row, its block the row's block, its length the place
    live = np.flatnonzero(slots >= 0)
    if len(live):
        rows = [x[live][:, None].contiguous().to(gpu) for x in (k, v)]
        bt = t((slots[live] // 16).astype(np.int32)[:, None], gpu)
        cl = t((slots[live] % 16 + 1).astype(np.int32), gpu)
        if kv == "same":
            gq.kv_append(*rows, wk, wv, bt, cl)
        else:
            gq.kv_append_quant(*rows, wk, wv, wks, wvs, bt, cl, kv=kv)
    kw = {} if kv == "same" else dict(k_scale=ks, v_scale=vs)
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    gq.kv_append_slots(k.to(gpu), v.to(gpu), kc, vc, t(slots, gpu), kv=kv, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for a, b in ((kc, wk), (vc, wv), (ks, wks), (vs, wvs)):
        assert a is None or torch.equal(a, b)
    # and back: the cached values, rounded once
    gk, gv = gq.kv_gather_slots(kc, vc, t(slots, gpu), kv=kv, dtype=dtype, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for got, x, codes, sc in ((gk, k, kc, ks), (gv, v, vc, vs)):
        if kv == "same":
            want = x.double().numpy().copy()
        elif kv == "int4":
            want = f4.dequantize(*f4.quantize(x.double().numpy()))
        else:
            want = np.zeros((M, K, H))
            for i in live:
                for h in range(K):
                    c = codes[slots[i] // 16, slots[i] % 16, h].cpu()
                    s = sc[slots[i] // 16, h, slots[i] % 16].item()
                    val = (c.view(torch.int8) if kv == "int8"
                           else c.view(torch.float8_e4m3fn)).float().numpy()
                    want[i, h] = (val * np.float32(s)).astype(np.float64)
        want[slots < 0] = 0.0
        np.testing.assert_array_equal(got.cpu().double().numpy(),
                                      torch.from_numpy(want).to(dtype).double().numpy())


def test_bad_slots_are_reported_and_skipped(gpu):
    k = torch.ones(4, 2, 64, dtype=torch.float16, device=gpu)
    for bad in (32, -2, 2**31 - 1, -2**31):
        (kc, vc), _ = caches("same", 2, 2, 64, torch.float16, gpu)
        st = torch.zeros(1, dtype=torch.int32, device=gpu)
        slots = t(np.array([0, bad, -1, 31], np.int32), gpu)
        gq.kv_append_slots(k, k, kc, vc, slots, status=st)
        assert int(st.item()) == 8
        st.zero_()
        gk, gv = gq.kv_gather_slots(kc, vc, slots, status=st)
        assert int(st.item()) == 8
        assert (gk[[0, 3]] == 1).all() and (gk[[1, 2]] == 0).all()
        assert int((kc == 3).sum()) == kc.numel() - 2 * 128
        assert torch.equal(gk, gv)


def test_no_rows(gpu):
    (kc, vc), (ks, vs) = caches("int4", 1, 2, 64, None, gpu)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=gpu)
    s = torch.empty(0, dtype=torch.int32, device=gpu)
    gq.kv_append_slots(e, e, kc, vc, s, k_scale=ks, v_scale=vs, kv="int4")
    gk, _ = gq.kv_gather_slots(kc, vc, s, k_scale=ks, v_scale=vs, kv="int4")
    assert gk.shape == (0, 2, 64) and bool((kc == 0x5A).all())


def test_slot_binding_refuses(gpu):
    (kc, vc), (ks, vs) = caches("int4", 4, 2, 64, None, gpu)
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=gpu)
    s = torch.zeros(3, dtype=torch.int32, device=gpu)
    kw = dict(k_scale=ks, v_scale=vs, kv="int4")
    for a, kk in (((k, k[:2], kc, vc, s), kw), ((k, k, kc, vc, s[:2]), kw),
                  ((k, k, kc, vc, s.long()), kw), ((k.float(), k.float(), kc, vc, s), kw),
                  ((k, k, kc, vc, s), dict(kv="int4")), ((k, k, kc, vc[:2], s), kw),
                  ((k[:, :1].contiguous(), k[:, :1].contiguous(), kc, vc, s), kw),
                  ((k, k, kc, vc, s), dict(kw, kv="nibble")), ((k, k, kc, vc, s), dict(kv="same")),
                  ((k.transpose(0, 1), k.transpose(0, 1), kc, vc, s), kw)):
        with pytest.raises((ValueError, TypeError)):
            gq.kv_append_slots(*a, **kk)


# ---- the planner -----------------------------------------------------------------------
def plan_inputs(B, seed, *, top=300, finished=0.1, short=0, width=None):
    """Random lengths, new tokens, tables and ring; `short`: ids missing."""
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, top, size=B)
    new = np.where(rng.random(B) < finished, -1, rng.integers(0, top, size=B))
    held = -(-ctx // 16) + (rng.random(B) < 0.3) * rng.integers(1, 4, size=B)
    need = np.where(new < 0, 0, -(-(ctx + np.maximum(new, 0)) // 16))
    grow = np.maximum(0, need - held).sum()
    mb = width or int(max(held.max(), need.max()) + 2)
    used = int(held.sum())
    count = max(0, int(grow) + 3 - short)
    NB = used + count
    ids = rng.permutation(NB)
    tables = np.full((B, mb), -7)
    off = 0
    for b in range(B):
        tables[b, : held[b]] = ids[off: off + held[b]]
        off += held[b]
    head = int(rng.integers(NB))
    ring = np.full(NB, -9)
    ring[(head + np.arange(count)) % NB] = ids[used:]
    tokens = int(np.maximum(new, 0).sum())
    i = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return [i(ctx), i(new), i(tables), i(held), i(ring), i([head, count])], tokens


def run_plan(a, max_tokens, dev, **kw):
    d = [t(x, dev) for x in a]
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = gq.plan_blocks(*d, max_tokens=max_tokens, status=st, **kw)
    torch.cuda.synchronize()
    out = got._asdict() | dict(block_tables=d[2], free_ring=d[4])
    return {k: v.cpu().numpy() for k, v in out.items() if v is not None}, int(st.item()), d


def check_plan(a, max_tokens, dev, **kw):
    want, errors = f4.plan_blocks(*a, -1 if max_tokens is None else max_tokens)
    got, st, d = run_plan(a, max_tokens, dev, **kw)
    for k, v in got.items():
        np.testing.assert_array_equal(v, want[k], err_msg=k)
    assert (st in errors) if errors else st == 0
    return got, d


@pytest.mark.parametrize("B,top", [(1, 1), (1, 40), (3, 17), (256, 300), (1000, 50), (1025, 33),
                                   (16384, 3), (64, 2000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_its_restatement(gpu, B, top, in_place):
    """Growing, finished and shortened sequences together, both sides of the one- and
    many-block launches, the ring's wrap included."""
    a, tokens = plan_inputs(B, B + top, top=top)
    got, d = check_plan(a, tokens + 5, gpu, in_place=in_place)
    if in_place:
        for x, k in ((d[0], "context_lens"), (d[3], "held"), (d[5], "ring_state")):
            np.testing.assert_array_equal(x.cpu().numpy(), got[k])


@pytest.mark.parametrize("B", [5, 300])
@pytest.mark.parametrize("short,tight", [(4, 0), (40, 0), (10 ** 6, 0), (0, 1), (0, 150), (20, 30)])
def test_plan_refuses_what_does_not_fit(gpu, B, short, tight):
    a, tokens = plan_inputs(B, B + short + tight, short=short)
    check_plan(a, max(0, tokens - tight), gpu)
    check_plan(a, None, gpu)  # no slot map, no token limit


def test_plan_rejects_bad_lengths_and_states(gpu):
    a, tokens = plan_inputs(40, 3, finished=0.3)
    a[0][3], a[1][5], a[3][7], a[3][9] = -4, -2, -1, a[2].shape[1] + 1
    a[0][11] = 16 * a[2].shape[1]
    a[3][13], a[0][13] = 0, 1
    a[1][15] = 2 ** 31 - 1
    check_plan(a, tokens + 64, gpu)
    for state in ((-1, 3), (len(a[4]), 0), (0, -1), (0, len(a[4]) + 1)):
        a[5][:] = state
        check_plan(a, tokens + 64, gpu)


def test_plan_keeps_ids_the_ring_has_no_room_for(gpu):
    a, tokens = plan_inputs(30, 4, finished=0.6)
    a[5][1] = len(a[4])  # claims that every block is free already
    a[1][:] = np.where(a[1] < 0, -1, 0)
    check_plan(a, tokens, gpu)


def test_plan_with_more_returns_than_an_int_holds_beside_the_count(gpu):
    """2^31 - 16384 ids claimed back by 16384 tables and a ring that is full."""
    B, mb, NB = 16384, 131071, 1000003
    i32 = lambda n, v: torch.full((n,), v, dtype=torch.int32, device=gpu)  # noqa: E731
    ring = torch.arange(NB, dtype=torch.int32, device=gpu)
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    tables = torch.empty(B, mb, dtype=torch.int32, device=gpu)  # not read: nothing is returned
    state = torch.tensor([7, NB], dtype=torch.int32, device=gpu)
    plan = gq.plan_blocks(i32(B, 5), i32(B, -1), tables, i32(B, mb), ring, state, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == int(gq.Status.ERR_BLOCKS)
    assert (plan.held == mb).all() and (plan.context_lens == 0).all()
    assert plan.ring_state.tolist() == [7, NB]
    assert torch.equal(ring, torch.arange(NB, dtype=torch.int32, device=gpu))


def test_plan_reports_ids_that_are_no_blocks(gpu):
    a, tokens = plan_inputs(20, 6, finished=0.0)
    a[4][(a[5][0] + 1) % len(a[4])] = 10 ** 7
    check_plan(a, tokens, gpu)


def test_plan_without_sequences(gpu):
    z = np.zeros(0, np.int32)
    a = [z, z, np.zeros((0, 4), np.int32), z, np.arange(5, dtype=np.int32),
         np.array([2, 5], np.int32)]
    got, st, _ = run_plan(a, 9, gpu)
    assert st == 0 and list(got["ring_state"]) == [2, 5] and list(got["cu_new"]) == [0]
    assert (got["slots"] == -1).all() and (got["positions"] == -1).all()


def test_plan_binding_refuses(gpu):
    a, tokens = plan_inputs(4, 1)
    d = [t(x, gpu) for x in a]
    for i, bad in ((0, d[0][:2]), (1, d[1].long()), (3, d[3].float()), (5, d[5][:1]),
                   (2, d[2].T), (4, d[4].cpu())):
        e = list(d)
        e[i] = bad
        with pytest.raises((ValueError, TypeError)):
            gq.plan_blocks(*e)
    for kw in (dict(positions=d[0]), dict(in_place=True, held_out=d[3]),
               dict(cu_new=d[0]), dict(max_tokens=3, slots=d[0])):
        with pytest.raises(ValueError):
            gq.plan_blocks(*d, **kw)


# ---- the calls of a serving loop together ----------------------------------------------
@pytest.mark.parametrize("kv,H,dtype", [("int4", 128, "bf16"), ("int4", 64, "f16"),
                                        ("same", 128, "bf16")])
def test_prompts_then_speculative_steps(gpu, kv, H, dtype):
    """Prompts admitted in one step (plan, append by slot), then verify steps (plan
    in place, append by block table + attention, greedy acceptance shortens the
    lengths on the device, the next plan gives blocks back), one request
    finishing on the way.  The last step's outputs against the oracle over the
    tokens each request really holds."""
    B, K, N, T, V, steps = 4, 2, 8, 3, 50, 6
    tdt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    rng = np.random.default_rng(3)
    NB, mb = 40, 12
    (kc, vc), (ks, vs) = caches(kv, NB, K, H, tdt, gpu)
    sc = {} if kv == "same" else dict(k_scale=ks, v_scale=vs)
    i32 = lambda x: t(np.asarray(x, np.int32), gpu)  # noqa: E731
    ctx, held, state = i32([0] * B), i32([0] * B), i32([5, NB])
    tables, ring = i32(np.full((B, mb), -1)), i32(rng.permutation(NB))
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    prompt = [37, 1, 90, 16]
    plan = gq.plan_blocks(ctx, i32(prompt), tables, held, ring, state, max_tokens=160,
                          in_place=True, status=st)
    gen = torch.Generator().manual_seed(1)
    rows = [torch.randn(160, K, H, generator=gen).to(tdt) for _ in range(2)]
    gq.kv_append_slots(rows[0].to(gpu), rows[1].to(gpu), kc, vc, plan.slots, kv=kv, status=st, **sc)
    cu = plan.cu_new.cpu().numpy()
    kept = [[(rows[0][i], rows[1][i]) for i in range(cu[b], cu[b + 1])] for b in range(B)]
    for step in range(steps):
        new = [T] * B
        if step >= 3:
            new[1] = -1 if step == 3 else 0  # finished, its row of the batch idle
        gq.plan_blocks(ctx, i32(new), tables, held, ring, state, in_place=True, status=st)
        live = [b for b in range(B) if new[b] > 0]
        sel = torch.tensor(live, device=gpu)
        cl, bt = ctx[sel].contiguous(), tables[sel].contiguous()
        q = torch.randn(len(live), T, N, H, generator=gen).to(tdt)
        kn, vn = (torch.randn(len(live), T, K, H, generator=gen).to(tdt) for _ in range(2))
        if kv == "same":
            out = gq.append_verify_attention(q.to(gpu), kn.to(gpu), vn.to(gpu), kc, vc, bt, cl,
                                             status=st)
        else:
            out = gq.append_verify_attention_quant(q.to(gpu), kn.to(gpu), vn.to(gpu), kc, vc, ks,
                                                   vs, bt, cl, kv=kv, status=st)
        logits = torch.randn(len(live), T, V, generator=gen)
        draft = logits[:, :-1].argmax(-1).to(torch.int32)
        draft[:, 1] += torch.tensor([(b + step) % 2 for b in live], dtype=torch.int32)
        before = cl.clone()
        acc, _ = gq.accept_prefix(logits.to(gpu), draft.to(gpu), cl, status=st)
        ctx[sel] = cl
        torch.cuda.synchronize()
        for j, b in enumerate(live):
            kept[b] += [(kn[j, i], vn[j, i]) for i in range(T)]
            assert int(before[j]) == len(kept[b])
        last = [[*kept[b]] for b in live]
        for j, b in enumerate(live):
            del kept[b][len(kept[b]) - (T - 1 - int(acc[j])):]
    assert int(st.item()) == 0
    w = small(B=len(live), T=T, N=N, K=K, H=H, dtype=dtype, ctx=[len(x) for x in last])
    w.q = [q]
    for j, seq in enumerate(last):
        for pos, (a, b) in enumerate(seq):
            blk, r = int(w.block_tables[j, pos // 16]), pos % 16
            w.k_cache[0][blk, r], w.v_cache[0][blk, r] = a, b
    if kv == "same":
        from helpers import assert_close
        ref, _ = oracle.attention(q, w.k_cache[0], w.v_cache[0], w.block_tables, w.context_lens,
                                  dtype)
        assert_close(out.double().cpu().numpy(), ref, dtype)
    else:
        kq, vq = f4.quantize_cache(w.k_cache[0]), f4.quantize_cache(w.v_cache[0])
        ref, lim = exact(w, (kq[0], vq[0], kq[1], vq[1]))
        check(out, ref, lim)
    # every block is in a table or in the ring
    h, n = held.cpu().numpy(), state.cpu().numpy()
    tb, rg = tables.cpu().numpy(), ring.cpu().numpy()
    ids = [tb[b, j] for b in range(B) for j in range(h[b])] + [
        rg[(n[0] + i) % NB] for i in range(n[1])]
    assert sorted(ids) == list(range(NB)) and h[1] == 0


def test_a_captured_step_replays_as_the_calls_do(gpu):
    """Plan in place, append + attention and greedy acceptance in one CUDA graph: every
    replay is the next step, with the same lengths, tables and outputs as the
    calls made one by one."""
    B, K, N, H, T, V, NB, mb = 5, 2, 8, 64, 4, 40, 60, 10
    rng = np.random.default_rng(7)
    gen = torch.Generator().manual_seed(7)

    def fresh():
        (kc, vc), (ks, vs) = caches("int4", NB, K, H, None, gpu, fill=0)
        i32 = lambda x: t(np.asarray(x, np.int32), gpu)  # noqa: E731
        return dict(c=[kc, vc, ks, vs], ctx=i32([0] * B), held=i32([0] * B), st=i32([0]),
                    tables=i32(np.full((B, mb), -1)), ring=i32(order), state=i32([9, NB]),
                    new=i32([T] * B), out=torch.empty(B, T, N, H, dtype=torch.float16, device=gpu),
                    acc=i32([0] * B), nxt=i32([0] * B))

    order = rng.permutation(NB)
    q = torch.randn(B, T, N, H, generator=gen).half().to(gpu)
    k, v = (torch.randn(B, T, K, H, generator=gen).half().to(gpu) for _ in range(2))
    logits = torch.randn(B, T, V, generator=gen)
    draft = logits[:, :-1].argmax(-1).to(torch.int32)
    draft[::2, 1] += 1  # every other sequence loses its last two drafts each step
    logits, draft = logits.to(gpu), draft.to(gpu)
    aws = torch.zeros(1 << 16, dtype=torch.uint8, device=gpu)

    def step(s):
        gq.plan_blocks(s["ctx"], s["new"], s["tables"], s["held"], s["ring"], s["state"],
                       in_place=True, status=s["st"])
        gq.append_verify_attention_quant(q, k, v, *s["c"], s["tables"], s["ctx"], kv="int4",
                                         out=s["out"], status=s["st"], pdl=True)
        gq.accept_prefix(logits, draft, s["ctx"], accepted=s["acc"], next_token=s["nxt"],
                         workspace=aws, status=s["st"])

    a, b = fresh(), fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for i in range(12):
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("ctx", "held", "state", "tables", "ring", "out", "acc"):
            assert torch.equal(a[n], b[n]), (i, n)
        assert int(a["st"].item()) == int(b["st"].item()) == 0
    assert a["ctx"].tolist() == [24, 48, 24, 48, 24]
