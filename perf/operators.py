"""What is measured of the 4-bit cache, the slot maps and the block planner.

Three operators, as a serving program uses them next to the paged attention calls:

  attend  decode / verify attention over a paged cache held in 4 bits
  slots   packed rows of several requests written into a paged cache by a slot
          map, then read back by it (what a chunked prompt does)
  plan    block tables, slot maps and lengths of a step, from request lengths

The 4-bit cache: every group of 32 consecutive elements of a cached row (one token
of one KV head) has a scale s = a / 7 (a the group's largest magnitude) rounded
to four significant bits (the byte b stands for the f16 number with bits b << 7;
at most 9216), and codes c = x / s rounded to nearest even, kept within [-7, 7].
A byte holds the codes of elements 2i (low half) and 2i + 1, each stored as c + 8.
Codes [blocks][KV heads][16][H / 2], scales [blocks][KV heads][16][H / 32].

`own` is False: plain torch operations.  True: the framework's calls.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

BS = 16  # tokens per cache block
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases ----------------------------------------------------------------------
def listed():
    return [
        # one short request alone: what a single user waits for at every token
        dict(name="decode-one", op="attend", B=1, T=1, N=14, K=2, H=64, dtype="f16",
             lens="fixed", lo=295, hi=295, lens_seed=1, window=0, tree=False),
        # one layer of a small model's decode batch, short ragged contexts
        dict(name="decode-short-64", op="attend", B=64, T=1, N=14, K=2, H=64, dtype="f16",
             lens="uniform", lo=16, hi=1024, lens_seed=102, window=0, tree=False),
        # one very long document, nothing else in the batch
        dict(name="decode-long-one", op="attend", B=1, T=1, N=32, K=8, H=128, dtype="bf16",
             lens="fixed", lo=100003, hi=100003, lens_seed=3, window=0, tree=False),
        # a full decode batch of very different lengths: the serving steady state
        dict(name="decode-ragged-256", op="attend", B=256, T=1, N=32, K=8, H=128, dtype="bf16",
             lens="lognormal", lo=1, hi=32768, lens_seed=104, window=0, tree=False),
        # a local layer of a hybrid model on long contexts
        dict(name="decode-local-32", op="attend", B=32, T=1, N=32, K=8, H=128, dtype="bf16",
             lens="fixed", lo=8192, hi=8192, lens_seed=106, window=1024, tree=False),
        # four drafts and the last token verified in one pass (40 rows per KV head)
        dict(name="verify-16", op="attend", B=16, T=5, N=64, K=8, H=128, dtype="bf16",
             lens="uniform", lo=512, hi=4096, lens_seed=105, window=0, tree=False),
        # the rows of one decode step of 256 requests, into a 4-bit cache
        dict(name="slots-step-256", op="slots", requests=256, lo=1, hi=1, lens_seed=7, K=8,
             H=128, dtype="bf16", kv="int4", spare=0),
        # a batch of prompts into a 4-bit cache; the map is longer than the rows in use
        dict(name="slots-prompts", op="slots", requests=24, lo=200, hi=3001, lens_seed=8, K=8,
             H=128, dtype="bf16", kv="int4", spare=77),
        # the same for a small model whose cache keeps the type of its rows
        dict(name="slots-prompts-same", op="slots", requests=17, lo=16, hi=1024, lens_seed=9,
             K=2, H=64, dtype="f16", kv="same", spare=5),
        # one decode step: a token each, some requests finished, some cut back by rejection
        dict(name="plan-step-256", op="plan", B=256, kind="step", lo=1, hi=4096, lens_seed=10,
             spare=0),
        # prompts admitted: every block table made new, a slot and a position per token
        dict(name="plan-prompts-64", op="plan", B=64, kind="prompts", lo=512, hi=8192,
             lens_seed=11, spare=100),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "slots", "plan"])
    if op == "slots":
        n = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 40000 // n))
        return dict(op=op, requests=n, lo=rng.randint(1, hi), hi=hi,
                    lens_seed=rng.randrange(1 << 30), K=rng.choice([1, 2, 3, 4, 8]),
                    H=rng.choice([64, 128]), dtype=rng.choice(["f16", "bf16"]),
                    kv=rng.choice(["int4", "int4", "same", "int8", "e4m3"]),
                    spare=rng.choice([0, 1, 13, 250]))
    if op == "plan":
        kind = rng.choice(["step", "prompts"])
        B = _log(rng, 1, 1000 if kind == "step" else 128)
        hi = _log(rng, 20, 8192 if kind == "step" else 4096)
        return dict(op=op, B=B, kind=kind, lo=rng.randint(1, hi), hi=hi,
                    lens_seed=rng.randrange(1 << 30), spare=rng.choice([0, 3, 1000]))
    cap = work(listed()[3])["bytes"]
    while True:
        K = rng.choice([1, 2, 4, 8])
        T = rng.choice([1, 1, 1, rng.randint(2, 8)])
        tree = T > 1 and rng.random() < 0.4
        hi = _log(rng, 8, 32768)
        case = dict(op=op, B=_log(rng, 1, 256), T=T, N=K * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]),
                    K=K, H=rng.choice([64, 128]), dtype=rng.choice(["f16", "bf16"]),
                    lens="uniform", lo=max(T, rng.randint(1, hi)), hi=max(T, hi),
                    lens_seed=rng.randrange(1 << 30),
                    window=0 if tree or rng.random() < 0.6 else _log(rng, 1, 4096), tree=tree)
        whole = work(dict(case, window=0))["bytes"]  # a window reads little of a big cache
        if (work(case)["bytes"] <= cap and whole <= 2 * cap
                and work(case)["flops"] <= work(listed()[3])["flops"]):
            return case


def _lens(case):
    """The lengths of a case: they belong to the case, not to the seed."""
    rng = random.Random(case["lens_seed"])
    n = case.get("B", case.get("requests"))
    if case.get("lens") == "lognormal":
        out = [int(round(math.exp(rng.gauss(math.log(2048), 1.0)))) for _ in range(n)]
        return [min(case["hi"], max(case["lo"], x)) for x in out]
    return [rng.randint(case["lo"], case["hi"]) for _ in range(n)]


def _row_bytes(kv, H):
    return {"same": 2 * H, "int8": H + 4, "e4m3": H + 4, "int4": H // 2 + H // 32}[kv]


def work(case):
    if case["op"] == "attend":
        lens, T, W = _lens(case), case["T"], case["window"]
        seen = [min(c, W + T - 1) if W else c for c in lens]  # positions read per sequence
        dots = sum(min(c - T + t + 1, W) if W else c - T + t + 1
                   for c in lens for t in range(T))
        blocks = sum((c + BS - 1) // BS - (max(0, c - T - W + 1) // BS if W else 0) for c in lens)
        io = 2 * case["B"] * T * case["N"] * case["H"] * 2
        tree = 8 * case["B"] * T if case["tree"] else 0
        return {"bytes": sum(seen) * case["K"] * 2 * _row_bytes("int4", case["H"]) + io
                + 4 * blocks + 4 * case["B"] + tree,
                "flops": 4 * dots * case["N"] * case["H"]}
    if case["op"] == "slots":
        M, side = sum(_lens(case)), case["K"] * 2
        # rows in, cache rows out; cache rows in, rows out (rows without a slot: zeros)
        return {"bytes": side * (M * (2 * case["H"] * 2 + 2 * _row_bytes(case["kv"], case["H"]))
                                 + case["spare"] * 2 * case["H"]) + 8 * (M + case["spare"]),
                "flops": side * M * case["H"] * 4}
    p = _plan_lists(case)
    total = sum(max(n, 0) for n in p["new"])
    moved = sum(abs(-(-(c + n if n >= 0 else 0) // BS) - h)
                for c, n, h in zip(p["ctx"], p["new"], p["held"]))
    return {"bytes": 12 * case["B"] + 12 * case["B"] + 8 * moved
            + 4 * sum(-(-n // BS) for n in p["new"] if n > 0) + 8 * (total + case["spare"]),
            "flops": 20 * case["B"] + 4 * total}


# ---- the 4-bit form ------------------------------------------------------------------
def _quantize4(x):
    """float32 [..., H] -> bytes [..., H/2], scale bytes [..., H/32]."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    y = g.abs().amax(-1)
    y = y / torch.full_like(y, 7.0)  # a tensor: by a number, torch multiplies by its reciprocal
    bits = y.contiguous().view(torch.int32)
    normal = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (112 << 3)
    small = torch.round(y * 131072.0).to(torch.int32)
    sb = torch.where(y >= 2.0 ** -14, normal, small)
    sb = torch.where(y >= 9216.0, torch.full_like(sb, 225), sb)
    s = _scale4(sb)[..., None]
    c = torch.where(s > 0, torch.round(g / s).clamp(-7, 7), torch.zeros_like(g))
    c = (c.to(torch.int32) + 8).reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8), sb.to(torch.uint8)


def _scale4(sb):
    return (sb.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()


def _values4(codes, sb):
    """float32 values [..., H] of bytes [..., H/2] and scale bytes [..., H/32]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0
    return (c.unflatten(-1, (-1, 32)) * _scale4(sb)[..., None]).flatten(-2)


# ---- inputs ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _chunks(n, per):
    return [(i, min(n, i + per)) for i in range(0, n, per)]


def _cache4(NB, K, H, g):
    """A filled 4-bit cache: normal rows whose channels differ in size, as keys' do."""
    codes = torch.empty(NB, K, BS, H // 2, dtype=torch.uint8, device="cuda")
    sb = torch.empty(NB, K, BS, H // 32, dtype=torch.uint8, device="cuda")
    size = torch.exp(0.5 * torch.randn(K, 1, H, device="cuda", generator=g))
    for i, j in _chunks(NB, max(1, (1 << 25) // (K * BS * H))):
        x = torch.randn(j - i, K, BS, H, device="cuda", generator=g) * size
        codes[i:j], sb[i:j] = _quantize4(x)
    return codes, sb


def _prepare_attend(case, seed):
    g, lens = _gen(seed), _lens(case)
    B, T, N, K, H, dt = (case["B"], case["T"], case["N"], case["K"], case["H"],
                         DT[case["dtype"]])
    nblk = [(c + BS - 1) // BS for c in lens]
    NB = sum(nblk) + 3
    ids = torch.randperm(NB, device="cuda", generator=g).to(torch.int32)
    tables = torch.full((B, max(nblk)), 2 ** 31 - 1, dtype=torch.int32)
    host, off = ids.cpu(), 0
    for b, n in enumerate(nblk):
        tables[b, :n] = host[off:off + n]
        off += n
    kc, ks = _cache4(NB, K, H, g)
    vc, vs = _cache4(NB, K, H, g)
    st = dict(case=case, lens=lens, kc=kc, ks=ks, vc=vc, vs=vs, tables=tables.cuda(),
              ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              q=torch.randn(B, T, N, H, device="cuda", generator=g).to(dt), mask=None)
    if case["tree"]:  # each node under a random earlier one: bit j set for an ancestor j
        rng = random.Random(seed)
        rows = []
        for _ in range(B):
            m = [0]
            for t in range(1, T):
                a = rng.randrange(t)
                m.append(m[a] | (1 << a))
            rows.append(m)
        st["mask"] = torch.tensor(rows, dtype=torch.int64, device="cuda")
    return st


def _prepare_slots(case, seed):
    g, lens = _gen(seed), _lens(case)
    K, H, dt, kv = case["K"], case["H"], DT[case["dtype"]], case["kv"]
    nblk = [(c + BS - 1) // BS for c in lens]
    NB, M = sum(nblk) + 2, sum(lens)
    ids = torch.randperm(NB, device="cuda", generator=g)
    slots, off = [], 0
    for c, n in zip(lens, nblk):
        p = torch.arange(c, device="cuda")
        slots.append(ids[off + p // BS] * BS + p % BS)
        off += n
    slots.append(torch.full((case["spare"],), -1, device="cuda"))
    rows = M + case["spare"]
    size = torch.exp(0.5 * torch.randn(K, H, device="cuda", generator=g))
    st = dict(case=case, slots=torch.cat(slots).to(torch.int32), unused=ids[off],
              k=(torch.randn(rows, K, H, device="cuda", generator=g) * size).to(dt),
              v=torch.randn(rows, K, H, device="cuda", generator=g).to(dt))
    if kv == "same":
        shape, sshape, cdt, sdt = (NB, BS, K, H), None, dt, None
    elif kv == "int4":
        shape, sshape, cdt, sdt = (NB, K, BS, H // 2), (NB, K, BS, H // 32), torch.uint8, torch.uint8
    else:
        shape, sshape, cdt, sdt = (NB, BS, K, H), (NB, K, BS), torch.uint8, torch.float32
    for n in "kv":
        st[n + "c"] = torch.zeros(shape, dtype=cdt, device="cuda")
        st[n + "s"] = None if sshape is None else torch.zeros(sshape, dtype=sdt, device="cuda")
    return st


def _plan_lists(case):
    """Lengths, new tokens and blocks held, as they stand before the step."""
    rng, lens = random.Random(case["lens_seed"] + 1), _lens(case)
    if case["kind"] == "prompts":
        return dict(ctx=[0] * case["B"], new=lens, held=[0] * case["B"])
    new = [-1 if rng.random() < 0.03 else rng.choice([1, 1, 1, 5]) for _ in lens]
    # rejected drafts leave a block or two more than the length needs
    held = [-(-c // BS) + (rng.random() < 0.1) + (rng.random() < 0.02) for c in lens]
    return dict(ctx=lens, new=new, held=[int(h) for h in held])


def _prepare_plan(case, seed):
    p, rng = _plan_lists(case), np.random.default_rng(seed)
    B = case["B"]
    total = sum(max(n, 0) for n in p["new"])
    grow = sum(max(0, -(-(c + n) // BS) - h) for c, n, h in zip(p["ctx"], p["new"], p["held"])
               if n >= 0)
    width = max(max(-(-(c + max(n, 0)) // BS), h) for c, n, h in
                zip(p["ctx"], p["new"], p["held"])) + 1
    used = sum(p["held"])
    NB = used + grow + 40
    ids = rng.permutation(NB).astype(np.int32)
    tables = np.full((B, width), -1, np.int32)
    off = 0
    for b, h in enumerate(p["held"]):
        tables[b, :h] = ids[off:off + h]
        off += h
    count, head = NB - used, int(rng.integers(NB))
    ring = np.full(NB, -1, np.int32)
    ring[(head + np.arange(count)) % NB] = ids[used:]
    dev = lambda a: torch.as_tensor(np.asarray(a, np.int32)).cuda()  # noqa: E731
    st = dict(case=case, ctx=dev(p["ctx"]), new=dev(p["new"]), held=dev(p["held"]),
              tables=dev(tables), ring=dev(ring), state=dev([head, count]),
              tokens=total + case["spare"])
    # the step's outputs, kept from step to step as a serving loop keeps them
    st["out"] = dict(context_lens_out=torch.empty_like(st["ctx"]),
                     held_out=torch.empty_like(st["held"]),
                     ring_state_out=torch.empty_like(st["state"]),
                     cu_new=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                     slots=torch.empty(st["tokens"], dtype=torch.int32, device="cuda"),
                     positions=torch.empty(st["tokens"], dtype=torch.int32, device="cuda"))
    return st


def prepare(case, seed):
    return {"attend": _prepare_attend, "slots": _prepare_slots,
            "plan": _prepare_plan}[case["op"]](case, seed)


# ---- one pass, plain ------------------------------------------------------------------
def _plain_attend(st):
    case, q = st["case"], st["q"].float()
    B, T, N, K, H, W = (case[x] for x in ("B", "T", "N", "K", "H", "window"))
    out = torch.empty_like(st["q"])
    for b, c in enumerate(st["lens"]):
        first = max(0, c - T - W + 1) // BS if W else 0
        blk = st["tables"][b, first:(c + BS - 1) // BS].long()
        n = c - first * BS
        k = _values4(st["kc"][blk], st["ks"][blk]).transpose(0, 1).reshape(K, -1, H)[:, :n]
        v = _values4(st["vc"][blk], st["vs"][blk]).transpose(0, 1).reshape(K, -1, H)[:, :n]
        qb = q[b].reshape(T, K, N // K, H).permute(1, 0, 2, 3).reshape(K, -1, H)
        s = torch.matmul(qb, k.transpose(1, 2)) * (H ** -0.5)
        if T > 1 or W:
            pos = torch.arange(first * BS, c, device=q.device)
            at = (c - T + torch.arange(T, device=q.device))[:, None]
            off = pos > at
            if W:
                off = off | (pos <= at - W)
            if st["mask"] is not None:
                j = (pos - (c - T)).clamp(0, 63)
                bit = (st["mask"][b][:, None] >> j) & 1
                off = off | ((pos >= c - T) & (pos < at) & (bit == 0))
            s = s.reshape(K, T, N // K, n).masked_fill(off[None, :, None], -math.inf)
            s = s.reshape(K, -1, n)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out[b] = o.reshape(K, T, N // K, H).permute(1, 0, 2, 3).reshape(T, N, H).to(out.dtype)
    return out


def _plain_slots(st):
    case, out = st["case"], []
    at = st["slots"].long()
    ok = at >= 0
    to = torch.where(ok, at, st["unused"] * BS)  # rows without a slot: a block nobody holds
    blk, row = to // BS, to % BS
    for n in "kv":
        x, codes, scale = st[n].float(), st[n + "c"], st[n + "s"]
        if case["kv"] == "int4":
            c, s = _quantize4(x)
            codes[blk, :, row], scale[blk, :, row] = c, s
            y = _values4(codes[blk, :, row], scale[blk, :, row])
        elif case["kv"] == "same":
            codes[blk, row] = st[n]
            y = codes[blk, row].float()
        else:
            qmax = 127.0 if case["kv"] == "int8" else 448.0
            s = x.abs().amax(-1)
            s = s / torch.full_like(s, qmax)
            y = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x))
            if case["kv"] == "int8":
                c = torch.round(y).clamp(-128, 127).to(torch.int8).view(torch.uint8)
            else:
                c = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[blk, row], scale[blk, :, row] = c, s
            kind = torch.int8 if case["kv"] == "int8" else torch.float8_e4m3fn
            y = codes[blk, row].view(kind).float() * scale[blk, :, row][..., None]
        out.append(torch.where(ok[:, None, None], y, torch.zeros_like(y)).to(st[n].dtype))
    return tuple(out)


def _plain_plan(st):
    ctx, new, held = st["ctx"].long(), st["new"].long(), st["held"].long()
    C, B, tokens = st["ring"].numel(), ctx.numel(), st["tokens"]
    head, count = st["state"][0].long(), st["state"][1].long()
    target = torch.where(new < 0, torch.zeros_like(ctx), ctx + new)
    need = (target + BS - 1) // BS
    grow, give = (need - held).clamp(min=0), (held - need).clamp(min=0)
    add = new.clamp(min=0)
    fits = ((grow == 0) | (grow.cumsum(0) <= count)) & ((add == 0) | (add.cumsum(0) <= tokens))
    zero = torch.zeros_like(ctx)
    grow, give, add = (torch.where(fits, x, zero) for x in (grow, give, add))
    lens = torch.where(fits, target, ctx)
    need = torch.where(fits, need, held)
    # table entries taken from the ring's head, entries given back at its tail
    col = torch.arange(st["tables"].shape[1], device=ctx.device)[None]
    src = (head + (grow.cumsum(0) - grow)[:, None] + col - held[:, None]) % C
    tables = torch.where((col >= held[:, None]) & (col < need[:, None]), st["ring"][src],
                         st["tables"])
    back = (col >= need[:, None]) & (col < held[:, None])
    dst = (head + count + (give.cumsum(0) - give)[:, None] + col - need[:, None]) % C
    ring = torch.cat([st["ring"], st["ring"][:1]])
    ring[torch.where(back, dst, torch.full_like(dst, C))] = st["tables"]
    state = torch.stack([(head + grow.sum()) % C, count - grow.sum() + give.sum()])
    end = add.cumsum(0)
    i = torch.arange(tokens, device=ctx.device)
    b = torch.searchsorted(end, i, right=True).clamp(max=B - 1)
    pos = lens[b] - end[b] + i
    on = i < end[-1]
    slot = tables[b, torch.where(on, pos // BS, torch.zeros_like(pos))].long() * BS + pos % BS
    none = torch.full_like(i, -1)
    cu = torch.cat([zero[:1], end])
    return tuple(x.to(torch.int32) for x in (lens, need, state, cu, torch.where(on, slot, none),
                                             torch.where(on, pos, none), tables, ring[:C]))


# ---- one pass ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "slots": _plain_slots, "plan": _plain_plan}[op](st)
    import gqa_decode_attention_02_gb300 as gq

    if op == "attend":
        if st["case"]["T"] == 1:
            return gq.decode_attention_quant(st["q"], st["kc"], st["vc"], st["ks"], st["vs"],
                                             st["tables"], st["ctx"], kv="int4",
                                             window=st["case"]["window"])
        return gq.verify_attention_quant(st["q"], st["kc"], st["vc"], st["ks"], st["vs"],
                                         st["tables"], st["ctx"], kv="int4",
                                         window=st["case"]["window"], tree_mask=st["mask"])
    if op == "slots":
        kv = st["case"]["kv"]
        gq.kv_append_slots(st["k"], st["v"], st["kc"], st["vc"], st["slots"], k_scale=st["ks"],
                           v_scale=st["vs"], kv=kv)
        return gq.kv_gather_slots(st["kc"], st["vc"], st["slots"], k_scale=st["ks"],
                                  v_scale=st["vs"], kv=kv, dtype=st["k"].dtype)
    got = gq.plan_blocks(st["ctx"], st["new"], st["tables"], st["held"], st["ring"],
                         st["state"], **st["out"])
    return tuple(got) + (st["tables"], st["ring"])


# ---- the operators' definitions in 64 bits ------------------------------------------------
def _exact_rows4(codes, sb):
    """float64 rows of one head: codes [n, H/2], scale bytes [n, H/32] (uint8)."""
    e, m = (sb >> 3).double(), (sb & 7).double()
    s = torch.where(e > 0, torch.exp2(e - 15) * (1 + m / 8), m * 2.0 ** -17)
    x = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    x[:, 0::2] = codes.remainder(16).double() - 8
    x[:, 1::2] = codes.div(16, rounding_mode="floor").double() - 8
    return x * s.repeat_interleave(32, dim=1)


def _exact_attend(case, seed):
    st = _prepare_attend(case, seed)
    B, T, N, K, H, W = (case[x] for x in ("B", "T", "N", "K", "H", "window"))
    G = N // K
    out = torch.zeros(B, T, N, H, dtype=torch.float64, device="cuda")
    mask = None if st["mask"] is None else st["mask"].tolist()
    q = st["q"].double() / math.sqrt(H)
    for b, c in enumerate(st["lens"]):
        lo = max(0, c - T - W + 1) if W else 0
        pos = torch.arange(lo, c, device="cuda")
        blk, row = st["tables"][b][pos // BS].long(), pos % BS
        for h in range(K):
            k = _exact_rows4(st["kc"][blk, h, row], st["ks"][blk, h, row])
            v = _exact_rows4(st["vc"][blk, h, row], st["vs"][blk, h, row])
            for t in range(T):
                i = c - T + t  # the token's own position
                keep = torch.ones(c - lo, dtype=torch.bool)
                keep[i + 1 - lo:] = False
                if W and i - W + 1 > lo:
                    keep[:i - W + 1 - lo] = False
                if mask is not None:
                    for j in range(t):
                        keep[c - T + j - lo] = bool((mask[b][t] >> j) & 1)
                kk, vv = (k, v) if bool(keep.all()) else (k[keep.cuda()], v[keep.cuda()])
                p = torch.softmax(q[b, t, h * G:(h + 1) * G] @ kk.T, -1)
                out[b, t, h * G:(h + 1) * G] = p @ vv
    return out


def _exact_slots(case, seed):
    if case["kv"] in ("int8", "e4m3"):
        return None  # their codes are defined by 32-bit divisions
    st = _prepare_slots(case, seed)
    live = (st["slots"] >= 0)[:, None, None]
    out = []
    for n in "kv":
        x = st[n].double()
        if case["kv"] == "int4":
            g = x.unflatten(-1, (-1, 32))
            y = g.abs().amax(-1, keepdim=True) / 7
            # the grid of four significant bits above 2^-14, of 2^-17 below
            step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -14))) - 3)
            s = (torch.round(y / step) * step).clamp(max=9216.0)
            c = torch.round(g / torch.where(s > 0, s, torch.ones_like(s))).clamp(-7, 7)
            x = (c * s).flatten(-2)
        out.append(torch.where(live, x, torch.zeros_like(x)))
    return tuple(out)


def _exact_plan(case, seed):
    st = _prepare_plan(case, seed)
    ctx, new, held, (head, count) = (st[x].tolist() for x in ("ctx", "new", "held", "state"))
    tables, ring = st["tables"].cpu().numpy().copy(), st["ring"].cpu().numpy().copy()
    C, tokens = len(ring), st["tokens"]
    wanted, asked, taken, given, cu, slots, places = 0, 0, 0, 0, [0], [], []
    for b in range(case["B"]):
        goal = ctx[b] + new[b] if new[b] >= 0 else 0
        want = -(-goal // BS)
        more, n = max(0, want - held[b]), max(0, new[b])
        wanted, asked = wanted + more, asked + n
        if (more and wanted > count) or (n and asked > tokens):
            cu.append(cu[-1])
            continue
        for j in range(held[b], want):
            tables[b, j] = ring[(head + taken) % C]
            taken += 1
        for j in range(want, held[b]):
            ring[(head + count + given) % C] = tables[b, j]
            given += 1
        p = np.arange(ctx[b], ctx[b] + n)
        slots.append(tables[b, p // BS].astype(np.int64) * BS + p % BS)
        places.append(p)
        cu.append(cu[-1] + n)
        ctx[b], held[b] = goal, want
    rest = [np.full(tokens - cu[-1], -1)]
    return tuple(torch.as_tensor(np.asarray(x, np.int64)).cuda() for x in (
        ctx, held, [(head + taken) % C, count - taken + given], cu,
        np.concatenate(slots + rest), np.concatenate(places + rest), tables, ring))


def exact(case, seed):
    if case["op"] == "attend" and 2 * case["B"] * case["K"] * case["T"] > 20000:
        return None
    return {"attend": _exact_attend, "slots": _exact_slots,
            "plan": _exact_plan}[case["op"]](case, seed)
