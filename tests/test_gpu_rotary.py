"""GPU rotation by position on the way into a cache: bit for bit what the formula gives with
every operation rounded in fp32, stored as kv_append_slots stores it."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_02_gb300 as gq
from chunk_ref import turn
from test_gpu_slots import caches

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def angles(P, R):
    a = np.arange(P)[:, None] * np.exp(-np.arange(R // 2) * (2 / R) * np.log(1e4))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


def batch(M, N, K, H, R, dtype, P=500, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(M, x, H, generator=g).to(dtype) for x in (N, K, K))
    rng = np.random.default_rng(seed)
    NB = M // 16 + 2
    slots = rng.permutation(NB * 16)[:M].astype(np.int32)
    pos = rng.integers(0, P, M).astype(np.int32)
    return q, k, v, slots, pos, angles(P, R), NB


def i32(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev)


@pytest.mark.parametrize("kv", ["same", "int8", "e4m3", "int4"])
@pytest.mark.parametrize("H,R,dtype", [(128, 128, BF16), (64, 64, F16), (128, 32, F16),
                                       (64, 48, BF16), (128, 16, BF16), (64, 16, F16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (37, 14, 2), (300, 9, 3)])
def test_rows(gpu, kv, H, R, dtype, interleaved, M, N, K):
    q, k, v, slots, pos, table, NB = batch(M, N, K, H, R, dtype, seed=M + R)
    slots[::7] = -1  # turned, not stored
    pos[3::11] = -1  # no token
    (kc, vc), (ks, vs) = caches(kv, NB, K, H, dtype, gpu)
    (wk, wv), (wks, wvs) = caches(kv, NB, K, H, dtype, gpu)
    out = torch.full((M, N, H), 7.0, dtype=dtype, device=gpu)
    st = torch.zeros(1, dtype=torch.int32, device=gpu)
    got = gq.kv_append_rotary(q.to(gpu), k.to(gpu), v.to(gpu), kc, vc, i32(slots, gpu),
                              i32(pos, gpu), table.to(gpu), q_out=out, k_scale=ks, v_scale=vs,
                              kv=kv, interleaved=interleaved, status=st)
    assert got is out and int(st.item()) == 0
    none = pos < 0
    want = turn(q, table, pos, interleaved).to(dtype)
    want[none] = 7.0
    assert torch.equal(out.cpu(), want)
    turned = turn(k, table, pos, interleaved).to(dtype)
    stored = np.where(none, -1, slots).astype(np.int32)
    gq.kv_append_slots(turned.to(gpu), v.to(gpu), wk, wv, i32(stored, gpu), k_scale=wks,
                       v_scale=wvs, kv=kv)
    for a, b in ((kc, wk), (vc, wv), (ks, wks), (vs, wvs)):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
def test_parts_of_a_projection_and_in_place(gpu, interleaved):
    M, N, K, H = 70, 6, 2, 128
    q, k, v, slots, pos, table, NB = batch(M, N, K, H, 96, BF16)
    x = torch.cat([q, k, v], 1).to(gpu)
    d = (i32(slots, gpu), i32(pos, gpu), table.to(gpu))
    (kc, vc), _ = caches("same", NB, K, H, BF16, gpu)
    (wk, wv), _ = caches("same", NB, K, H, BF16, gpu)
    a = gq.kv_append_rotary(x[:, :N], x[:, N:N + K], x[:, N + K:], kc, vc, *d,
                            interleaved=interleaved)
    qd = q.to(gpu)
    b = gq.kv_append_rotary(qd, k.to(gpu), v.to(gpu), wk, wv, *d, q_out=qd,
                            interleaved=interleaved)
    assert b is qd and torch.equal(a, b)
    assert torch.equal(a.cpu(), turn(q, table, pos, interleaved).to(BF16))
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_special_values_turn_as_the_formula_says(gpu):
    q, k, v, slots, pos, table, NB = batch(20, 2, 1, 64, 64, F16)
    q[0, 0, 5], q[1, 0, 40], q[2, 1, 3] = float("inf"), float("nan"), -65504.0
    q[3] = 0.0
    q[4] = 6e-8
    (kc, vc), _ = caches("same", NB, 1, 64, F16, gpu)
    got = gq.kv_append_rotary(q.to(gpu), k.to(gpu), v.to(gpu), kc, vc, i32(slots, gpu),
                              i32(pos, gpu), table.to(gpu)).cpu()
    want = turn(q, table, pos, False).to(F16)
    assert torch.equal(torch.nan_to_num(got, nan=9.0), torch.nan_to_num(want, nan=9.0))


def test_bad_positions_and_slots(gpu):
    q, k, v, slots, pos, table, NB = batch(40, 4, 2, 64, 64, F16, P=50)
    for where, bad, code in (("pos", 50, 7), ("pos", -2, 7), ("pos", 2 ** 31 - 1, 7),
                             ("slot", NB * 16, 8), ("slot", -2, 8)):
        s, p = slots.copy(), pos.copy()
        (s if where == "slot" else p)[9] = bad
        (kc, vc), _ = caches("same", NB, 2, 64, F16, gpu)
        (wk, wv), _ = caches("same", NB, 2, 64, F16, gpu)
        out = torch.full((40, 4, 64), 7.0, dtype=F16, device=gpu)
        st = torch.zeros(1, dtype=torch.int32, device=gpu)
        gq.kv_append_rotary(q.to(gpu), k.to(gpu), v.to(gpu), kc, vc, i32(s, gpu), i32(p, gpu),
                            table.to(gpu), q_out=out, status=st)
        assert int(st.item()) == code
        want = turn(q, table, pos, False).to(F16)
        if where == "pos":
            want[9] = 7.0
        assert torch.equal(out.cpu(), want)
        s[9] = -1
        gq.kv_append_slots(turn(k, table, pos, False).to(F16).to(gpu), v.to(gpu), wk, wv,
                           i32(s, gpu))
        assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_no_rows_and_refusals(gpu):
    q, k, v, slots, pos, table, NB = batch(5, 4, 2, 64, 64, F16)
    (kc, vc), (ks, vs) = caches("same", NB, 2, 64, F16, gpu)
    d = [x.to(gpu) for x in (q, k, v)] + [kc, vc, i32(slots, gpu), i32(pos, gpu), table.to(gpu)]
    e = [x[:0] if i in (0, 1, 2, 5, 6) else x for i, x in enumerate(d)]
    assert gq.kv_append_rotary(*e).shape == (0, 4, 64)

    def but(i, x):
        return [x if j == i else y for j, y in enumerate(d)]

    for a, kw in ((but(0, d[0].float()), {}), (but(0, q), {}), (but(0, d[0][:, ::2]), {}),
                  (but(1, d[1][:4]), {}), (but(2, d[2].bfloat16()), {}), (but(1, d[1][:, :1]), {}),
                  (but(5, d[5].long()), {}), (but(6, d[6][:4]), {}), (but(7, d[7].double()), {}),
                  (d, dict(q_out=d[0][:4].clone())), (d, dict(kv="int8")), (d, dict(kv="x")),
                  (d, dict(q_out=torch.zeros(5, 8, 64, dtype=F16, device=gpu)[:, ::2]))):
        with pytest.raises((ValueError, TypeError)):
            gq.kv_append_rotary(*a, **kw)
    for R in (8, 40, 80):  # sixteenths of at most H
        with pytest.raises(gq.GqaError):
            gq.kv_append_rotary(*but(7, angles(9, R).to(gpu)))
    with pytest.raises(gq.GqaError):
        gq.kv_append_rotary(*but(7, torch.zeros(0, 64, device=gpu)))


def test_streams_and_graphs(gpu):
    q, k, v, slots, pos, table, NB = batch(33, 4, 2, 128, 128, BF16)
    d = [x.to(gpu) for x in (q, k, v)]
    (kc, vc), _ = caches("same", NB, 2, 128, BF16, gpu)
    s, p, t = i32(slots, gpu), i32(pos, gpu), table.to(gpu)
    want = gq.kv_append_rotary(*d, kc, vc, s, p, t)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq.kv_append_rotary(*d, kc, vc, s, p, t, q_out=out, pdl=True)
    k2 = kc.clone()
    kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    live = torch.zeros(NB * 16, dtype=torch.bool)
    live[torch.from_numpy(slots).long()] = True
    assert torch.equal(kc.view(-1, 2, 128)[live.to(gpu)], k2.view(-1, 2, 128)[live.to(gpu)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gq.kv_append_rotary(*d, kc, vc, s, p, t, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
