"""What is measured of prompt chunks and of decoding over chosen blocks.

Five operators, as a serving program uses them next to the paged attention calls:

  rotary  queries rotated by position, keys rotated and stored with their values
          in a paged cache by a slot map
  chunk   attention of the new tokens of several requests (prompts, parts of
          prompts, single tokens) over a paged cache, causal, with a window or without
  bounds  largest and smallest key of every cache block that a step has touched,
          in 8 bits
  select  the blocks of a long cache that a query should read, by those bounds
  sparse  attention of one token per request over chosen blocks, each KV head with
          a table of its own

rotary: pairs of elements (i, i + R/2) of the first R of H, or (2i, 2i + 1)
(interleaved), turn by the angle whose cosine and sine the table holds for the token's
position: x1 c - x2 s and x2 c + x1 s, rounded to the 16-bit type, then stored as the
cache holds its rows.
bounds, of one block and KV head: scale = max |k| / 127 over the rows held, codes
ceil(max_d / scale) and floor(min_d / scale), at most 127 in size, per element d.
select: q's rows become 8-bit codes too (scale max |q| / 127, nearest even); a block's
score is the largest over a KV head's queries of
(q scale * block scale) * sum_d max(q_d max_d, q_d min_d).  The first and the newest
blocks are always kept, the others by score, ties to the lowest block.

`own` is False: plain torch operations.  True: the framework's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BS = 16  # tokens per cache block
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases ----------------------------------------------------------------------
def listed():
    return [
        # the rest of a short prompt of one user behind a cached prefix
        dict(name="chunk-one", op="chunk", N=14, K=2, H=64, dtype="f16", kind="chunk", B=1,
             lo=37, hi=37, ctx=295, lens_seed=1, window=0, spare=0),
        # a mixed step: a part of one prompt among requests that decode one token each
        dict(name="chunk-mixed-32", op="chunk", N=32, K=8, H=128, dtype="bf16", kind="mixed",
             B=32, lo=512, hi=512, ctx=4096, lens_seed=2, window=0, spare=13),
        # a batch of new prompts of very different lengths
        dict(name="chunk-prompts-24", op="chunk", N=32, K=8, H=128, dtype="bf16",
             kind="prompts", B=24, lo=200, hi=3001, ctx=0, lens_seed=8, window=0, spare=77),
        # a part of one very long prompt, behind what is cached already
        dict(name="chunk-behind-32k", op="chunk", N=32, K=8, H=128, dtype="bf16", kind="chunk",
             B=1, lo=2048, hi=2048, ctx=32768, lens_seed=4, window=0, spare=0),
        # one decode step of 256 requests
        dict(name="rotary-step-256", op="rotary", N=32, K=8, H=128, R=128, dtype="bf16",
             requests=256, lo=1, hi=1, far=32768, lens_seed=7, kv="same", interleaved=False,
             packed=True, spare=0),
        # a batch of prompts; the slot map is longer than the rows in use
        dict(name="rotary-prompts-24", op="rotary", N=32, K=8, H=128, R=128, dtype="bf16",
             requests=24, lo=200, hi=3001, far=0, lens_seed=8, kv="same", interleaved=False,
             packed=True, spare=77),
        # the newest block of every request after a decode step
        dict(name="bounds-step-256", op="bounds", K=8, H=128, dtype="bf16", B=256, lo=1, hi=1,
             ctx=8192, lens_seed=10),
        # every block of a batch of new prompts
        dict(name="bounds-prompts-24", op="bounds", K=8, H=128, dtype="bf16", B=24, lo=200,
             hi=3001, ctx=0, lens_seed=8),
        # one very long document, nothing else in the batch
        dict(name="select-long-one", op="select", N=32, K=8, H=128, dtype="bf16", B=1,
             lo=100003, hi=100003, lens_seed=3, keep=256, first=1, recent=2),
        # a batch of long documents
        dict(name="select-64x32k", op="select", N=32, K=8, H=128, dtype="bf16", B=64,
             lo=30000, hi=32768, lens_seed=12, keep=128, first=1, recent=2),
        # the same one document, one decode step over what was chosen
        dict(name="sparse-long-one", op="sparse", N=32, K=8, H=128, dtype="bf16", B=1, keep=256,
             full=1.0, lens_seed=3),
        # the batch, one decode step
        dict(name="sparse-64", op="sparse", N=32, K=8, H=128, dtype="bf16", B=64, keep=128,
             full=0.9, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rotary", "bounds", "select", "sparse"])
    K = rng.choice([1, 2, 3, 4, 8])
    case = dict(op=op, K=K, H=rng.choice([64, 128]), dtype=rng.choice(["f16", "bf16"]),
                lens_seed=rng.randrange(1 << 30))
    N = K * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "rotary":
        n = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 20000 // n))
        return dict(case, N=N, requests=n, lo=rng.randint(1, hi), hi=hi,
                    R=rng.choice([case["H"], case["H"], 32, 48]), far=_log(rng, 1, 32768),
                    kv=rng.choice(["same", "same", "int8", "e4m3", "int4"]),
                    interleaved=rng.random() < 0.4, packed=rng.random() < 0.5,
                    spare=rng.choice([0, 1, 13, 250]))
    if op == "bounds":
        B = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, 30000 // B))
        return dict(case, B=B, lo=rng.randint(1, hi), hi=hi, ctx=_log(rng, 1, 4096))
    if op == "select":
        B, keep = _log(rng, 1, 64), rng.randint(4, 300)
        hi = _log(rng, 1, 32768)
        return dict(case, N=N, B=B, lo=rng.randint(max(1, hi // 2), hi), hi=hi, keep=keep,
                    first=rng.choice([0, 1, 1, 2]), recent=rng.choice([1, 2]))
    if op == "sparse":
        return dict(case, N=N, B=_log(rng, 1, 64), keep=_log(rng, 1, 128),
                    full=rng.choice([1.0, 0.7]))
    top = work(listed()[3])
    while True:
        kind = rng.choice(["chunk", "prompts", "mixed"])
        B = 1 if kind == "chunk" else _log(rng, 2, 48)
        hi = _log(rng, 1, 4096)
        one = dict(case, N=N, kind=kind, B=B, lo=rng.randint(max(1, hi // 8), hi), hi=hi,
                   ctx=0 if kind == "prompts" else max(hi, _log(rng, 8, 32768)),
                   window=0 if rng.random() < 0.7 else _log(rng, 1, 4096),
                   spare=rng.choice([0, 0, 5, 200]))
        w = work(dict(one, window=0))
        if w["flops"] <= top["flops"] and w["bytes"] <= 4 * top["bytes"]:
            return one


def _lens(case):
    """New tokens and lengths with them, per request: of the case, not of the seed."""
    rng = random.Random(case["lens_seed"])
    n = case.get("B", case.get("requests"))
    new = [rng.randint(case["lo"], case["hi"]) for _ in range(n)]
    if case["op"] == "rotary":
        return new, [rng.randint(0, case["far"]) + x for x in new]
    if case["op"] == "select":
        return new, new
    if case.get("kind") == "chunk":
        return new, [max(case["ctx"], x) for x in new]
    if case.get("kind") == "mixed":
        at = rng.randrange(n)
        new = [x if i == at else 1 for i, x in enumerate(new)]
    return new, [x + (rng.randint(0, max(0, case["ctx"] - x)) if case["ctx"] else 0) for x in new]


def _sparse_lens(case):
    """Tokens read per request: whole blocks, the last one in part."""
    rng, S = random.Random(case["lens_seed"]), case["keep"]
    blocks = [S if rng.random() < case["full"] else rng.randint(1, S) for _ in range(case["B"])]
    return [(n - 1) * BS + rng.randint(1, BS) for n in blocks]


def _row_bytes(kv, H):
    return {"same": 2 * H, "int8": H + 4, "e4m3": H + 4, "int4": H // 2 + H // 32}[kv]


def work(case):
    op, K, H = case["op"], case["K"], case["H"]
    if op == "sparse":
        lens = _sparse_lens(case)
        tok = sum(lens)
        return {"bytes": tok * K * 4 * H + 4 * case["B"] * case["N"] * H
                + 4 * K * sum(-(-n // BS) for n in lens) + 4 * case["B"],
                "flops": 4 * tok * case["N"] * H}
    new, ctx = _lens(case)
    if op == "chunk":
        W = case["window"]
        dots = read = 0
        for n, c in zip(new, ctx):
            first = c - n  # position of the first new token; token t sees min(first + t + 1, W)
            full = n if not W else max(0, min(n, W - first))  # tokens whose window reaches 0
            dots += full * first + full * (full + 1) // 2 + (n - full) * W
            read += min(c, W + n - 1) if W else c
        rows = sum(new)
        return {"bytes": read * K * 4 * H + 4 * rows * case["N"] * H + 4 * (read // BS)
                + 8 * len(new), "flops": 4 * dots * case["N"] * H}
    if op == "rotary":
        M = sum(new)
        back = 0 if case["kv"] == "same" else 2 * K * (_row_bytes(case["kv"], H) + 2 * H)
        return {"bytes": M * (4 * case["N"] * H + 2 * K * (2 * H + _row_bytes(case["kv"], H))
                              + 4 * case["R"] + back) + 8 * (M + case["spare"]),
                "flops": 3 * M * (case["N"] + K) * case["R"]}
    if op == "bounds":
        rows = sum(c - (c - n) // BS * BS for n, c in zip(new, ctx))
        blocks = sum(-(-c // BS) - (c - n) // BS for n, c in zip(new, ctx))
        return {"bytes": rows * K * 2 * H + blocks * (K * (2 * H + 4) + 4) + 8 * case["B"],
                "flops": 3 * rows * K * H}
    nb = [-(-c // BS) for c in ctx]
    scored = sum(n for n in nb if n > case["keep"])
    return {"bytes": scored * (K * (2 * H + 4) + 4) + 2 * case["B"] * case["N"] * H
            + 8 * case["B"] * K * case["keep"] + 8 * case["B"],
            "flops": 4 * scored * case["N"] * H}


# ---- inputs ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _normal(shape, dt, g):
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        n = min(1 << 26, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, device="cuda", generator=g)
    return out


def _tables(nblk, g, width=None):
    """Shuffled block ids for requests of nblk blocks each; how many blocks there are."""
    NB = sum(nblk) + 3
    ids = torch.randperm(NB, device="cuda", generator=g).to(torch.int32).cpu()
    tables = torch.full((len(nblk), width or max(max(nblk), 1)), 2 ** 31 - 1, dtype=torch.int32)
    off = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = ids[off:off + n]
        off += n
    return tables.cuda(), NB, int(ids[off])


def _cu(new):
    return _i32([0] + [sum(new[:i + 1]) for i in range(len(new))])


def _prepare_chunk(case, seed):
    g, (new, ctx) = _gen(seed), _lens(case)
    N, K, H, dt = case["N"], case["K"], case["H"], DT[case["dtype"]]
    tables, NB, _ = _tables([-(-c // BS) for c in ctx], g)
    rows = sum(new) + case["spare"]
    size = torch.exp(0.5 * torch.randn(K, H, device="cuda", generator=g)).to(dt)
    return dict(case=case, new=new, lens=ctx, tables=tables, ctx=_i32(ctx), cu=_cu(new),
                q=_normal((rows, N, H), dt, g), kc=_normal((NB, BS, K, H), dt, g).mul_(size),
                vc=_normal((NB, BS, K, H), dt, g),
                out=torch.zeros(rows, N, H, dtype=dt, device="cuda"))


def _prepare_rotary(case, seed):
    g, (new, ctx) = _gen(seed), _lens(case)
    N, K, H, R, dt, kv = (case["N"], case["K"], case["H"], case["R"], DT[case["dtype"]],
                          case["kv"])
    # the cache holds the new rows; where in the sequence they are only the positions say
    nblk = [-(-n // BS) + 1 for n in new]
    NB, M = sum(nblk) + 1, sum(new)
    ids = torch.randperm(NB, device="cuda", generator=g)
    slots, places, off = [], [], 0
    for n, c, k in zip(new, ctx, nblk):
        p = torch.arange(n, device="cuda") + (c - n) % BS
        slots.append(ids[off + p // BS] * BS + p % BS)
        places.append(torch.arange(c - n, c, device="cuda"))
        off += k
    none = torch.full((case["spare"],), -1, device="cuda")
    rows = M + case["spare"]
    # a projection's output holds q, k and v side by side; or three tensors
    x = _normal((rows, N + 2 * K, H), dt, g)
    q, k, v = x[:, :N], x[:, N:N + K], x[:, N + K:]
    if not case["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    far = max(ctx) + 1
    freq = torch.exp(torch.arange(R // 2, device="cuda").double() * (-2.0 / R * math.log(5e5)))
    angle = torch.arange(far, device="cuda").double()[:, None] * freq
    st = dict(case=case, q=q, k=k, v=v, unused=ids[off], q_out=torch.zeros_like(q.contiguous()),
              table=torch.cat([angle.cos(), angle.sin()], 1).float(),
              slots=torch.cat(slots + [none]).to(torch.int32),
              places=torch.cat(places + [none]).to(torch.int32))
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


def _prepare_bounds(case, seed):
    g, (new, ctx) = _gen(seed), _lens(case)
    K, H, dt = case["K"], case["H"], DT[case["dtype"]]
    # the blocks before the new tokens' are not read: they may be any
    nblk = [-(-c // BS) for c in ctx]
    fresh = [n - (c - x) // BS for n, c, x in zip(nblk, ctx, new)]
    tail, NB, _ = _tables(fresh, g)
    tables = torch.full((case["B"], max(nblk)), 2 ** 31 - 1, dtype=torch.int32)
    host = tail.cpu()
    for b, (n, f) in enumerate(zip(nblk, fresh)):
        tables[b, n - f:n] = host[b, :f]
    size = torch.exp(0.5 * torch.randn(K, H, device="cuda", generator=g)).to(dt)
    return dict(case=case, tables=tables.cuda(), ctx=_i32(ctx), cu=_cu(new),
                kc=_normal((NB, BS, K, H), dt, g).mul_(size),
                codes=torch.zeros(NB, K, 2, H, dtype=torch.int8, device="cuda"),
                scale=torch.zeros(NB, K, dtype=torch.float32, device="cuda"),
                most=max(new))


def _prepare_select(case, seed):
    g, (_, ctx) = _gen(seed), _lens(case)
    B, N, K, H, dt = case["B"], case["N"], case["K"], case["H"], DT[case["dtype"]]
    tables, NB, _ = _tables([-(-c // BS) for c in ctx], g)
    codes = torch.empty(NB, K, 2, H, dtype=torch.int8, device="cuda")
    for i in range(0, NB, 4096):
        n = min(4096, NB - i)
        mid = 12.0 * torch.randn(n, K, H, device="cuda", generator=g)
        half = 40.0 + 12.0 * torch.randn(n, K, H, device="cuda", generator=g).abs()
        codes[i:i + n, :, 0] = (mid + half).round().clamp(-127, 127).to(torch.int8)
        codes[i:i + n, :, 1] = (mid - half).round().clamp(-127, 127).to(torch.int8)
    return dict(case=case, tables=tables, ctx=_i32(ctx), codes=codes,
                scale=0.03 * torch.exp(0.1 * torch.randn(NB, K, device="cuda", generator=g)),
                q=_normal((B, 1, N, H), dt, g))


def _prepare_sparse(case, seed):
    g, lens = _gen(seed), _sparse_lens(case)
    B, N, K, H, S, dt = (case["B"], case["N"], case["K"], case["H"], case["keep"],
                         DT[case["dtype"]])
    # every KV head has chosen blocks of its own; no row of the cache is read twice
    NB = B * S + 3
    ids = torch.stack([torch.randperm(NB, device="cuda", generator=g)[:B * S] for _ in range(K)])
    tables = ids.view(K, B, S).transpose(0, 1).contiguous().to(torch.int32)
    held = _i32([-(-n // BS) for n in lens])
    tables[torch.arange(S, device="cuda")[None, None].expand(B, K, S) >= held[:, None, None]] = -1
    return dict(case=case, tables=tables, lens=_i32(lens), q=_normal((B, 1, N, H), dt, g),
                kc=_normal((NB, BS, K, H), dt, g), vc=_normal((NB, BS, K, H), dt, g))


def prepare(case, seed):
    return {"chunk": _prepare_chunk, "rotary": _prepare_rotary, "bounds": _prepare_bounds,
            "select": _prepare_select, "sparse": _prepare_sparse}[case["op"]](case, seed)


# ---- one pass, plain ------------------------------------------------------------------
def _plain_chunk(st):
    case, out = st["case"], st["out"]
    N, K, H, W = (case[x] for x in ("N", "K", "H", "window"))
    at = 0
    for b, (n, c) in enumerate(zip(st["new"], st["lens"])):
        first = max(0, c - n - W + 1) // BS if W else 0
        blk = st["tables"][b, first:(c + BS - 1) // BS].long()
        k = st["kc"][blk].view(-1, K, H)[:c - first * BS].float().permute(1, 2, 0)
        v = st["vc"][blk].view(-1, K, H)[:c - first * BS].float().transpose(0, 1)
        pos = torch.arange(first * BS, c, device=out.device)
        step = max(1, (1 << 31) // (N * pos.numel()))  # a part of the scores at a time
        for t in range(0, n, step):
            m = min(step, n - t)
            q = st["q"][at + t:at + t + m].float().view(m, K, N // K, H).permute(1, 2, 0, 3)
            s = torch.matmul(q.reshape(K, -1, H), k).mul_(H ** -0.5).view(K, N // K, m, -1)
            own_pos = (c - n + t + torch.arange(m, device=out.device))[:, None]
            off = pos > own_pos
            if W:
                off = off | (pos <= own_pos - W)
            s = s.masked_fill_(off, -math.inf)
            p = s.sub_(s.amax(-1, keepdim=True)).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(K, -1, pos.numel()), v).view(K, N // K, m, H) / total
            out[at + t:at + t + m] = o.permute(2, 0, 1, 3).reshape(m, N, H).to(out.dtype)
        at += n
    return out


def _turn(x, cos, sin, interleaved):
    """float32 rows [M, heads, H]; cos, sin [M, 1, R/2]."""
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., R:]], -1)


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


def _plain_rotary(st):
    case, dt, kv = st["case"], st["q"].dtype, st["case"]["kv"]
    ok, half = st["places"] >= 0, case["R"] // 2
    angles = st["table"][st["places"].clamp(min=0).long()][:, None]
    cos, sin = angles[..., :half], angles[..., half:]
    q = _turn(st["q"].float(), cos, sin, case["interleaved"]).to(dt)
    st["q_out"].copy_(torch.where(ok[:, None, None], q, st["q_out"]))
    rows = {"k": _turn(st["k"].float(), cos, sin, case["interleaved"]).to(dt), "v": st["v"]}
    to = torch.where(ok, st["slots"].long(), st["unused"] * BS)  # no slot: a block nobody holds
    blk, row, out = to // BS, to % BS, [st["q_out"]]
    for n, x in rows.items():
        x = torch.where(ok[:, None, None], x, torch.zeros_like(x))
        codes, scale = st[n + "c"], st[n + "s"]
        if kv == "same":
            codes[blk, row] = x
            out.append(codes)
            continue
        x = x.float()
        if kv == "int4":
            codes[blk, :, row], scale[blk, :, row] = _quantize4(x)
            y = _values4(codes[blk, :, row], scale[blk, :, row])
        else:
            s = x.abs().amax(-1)
            s = s / torch.full_like(s, 127.0 if kv == "int8" else 448.0)
            y = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x))
            kind = torch.int8 if kv == "int8" else torch.float8_e4m3fn
            y = torch.round(y).clamp(-128, 127) if kv == "int8" else y.clamp(-448, 448)
            codes[blk, row], scale[blk, :, row] = y.to(kind).view(torch.uint8), s
            y = codes[blk, row].view(kind).float() * scale[blk, :, row][..., None]
        out.append(torch.where(ok[:, None, None], y, torch.zeros_like(y)).to(dt))
    return tuple(out)


def _touched(st):
    """Blocks that hold new tokens: ids, rows held in each; False where there is none."""
    ctx, cu = st["ctx"].long(), st["cu"].long()
    first = (ctx - (cu[1:] - cu[:-1])) // BS
    i = first[:, None] + torch.arange(st["most"] // BS + 2, device=ctx.device)
    on = i * BS < ctx[:, None]
    ids = st["tables"].gather(1, i.clamp(max=st["tables"].shape[1] - 1))
    return ids[on].long(), (ctx[:, None] - i * BS).clamp(max=BS)[on]


def _plain_bounds(st):
    ids, held = _touched(st)
    k = st["kc"][ids].float()
    out = (torch.arange(BS, device=k.device) >= held[:, None])[:, :, None, None]
    scale = k.masked_fill(out, 0.0).abs().amax((1, 3))
    scale = scale / torch.full_like(scale, 127.0)
    s = torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    top = torch.ceil(k.masked_fill(out, -math.inf).amax(1) / s).clamp(-127, 127)
    low = torch.floor(k.masked_fill(out, math.inf).amin(1) / s).clamp(-127, 127)
    st["codes"][ids] = torch.stack([top, low], 2).to(torch.int8)
    st["scale"][ids] = scale
    return st["codes"], st["scale"]


def _plain_select(st):
    case, q, ctx = st["case"], st["q"][:, 0].float(), st["ctx"].long()
    B, N, K, H, S = (case[x] for x in ("B", "N", "K", "H", "keep"))
    tables = st["tables"]
    nb = (ctx + BS - 1) // BS
    i = torch.arange(tables.shape[1], device=q.device)[None]
    ids = torch.where(i < nb[:, None], tables, torch.zeros_like(tables)).long()
    qs = q.abs().amax(-1)
    qs = qs / torch.full_like(qs, 127.0)
    qc = torch.where(qs[..., None] > 0, torch.round(q / qs[..., None]), torch.zeros_like(q))
    qc = torch.cat([qc.clamp(min=0), qc.clamp(max=0)], -1).view(B, K, N // K, 2 * H)
    qs = qs.view(B, K, N // K, 1)
    score = torch.empty(B, K, tables.shape[1], device=q.device)
    for b in range(B):  # (whole numbers below 2^24: the product is exact)
        c = st["codes"][ids[b]].float().view(-1, K, 2 * H).permute(1, 2, 0)
        dot = torch.matmul(qc[b], c)
        score[b] = (qs[b] * st["scale"][ids[b]].T[:, None] * dot).amax(1)
    held = nb.clamp(max=S)
    always = (i < case["first"]) | (i >= nb[:, None] - case["recent"])
    score = torch.where(always[:, None], torch.full_like(score, math.inf), score)
    score = score.masked_fill((i >= nb[:, None])[:, None], -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :S]
    col = torch.arange(order.shape[-1], device=q.device)
    order = torch.where(col < held[:, None, None], order, torch.full_like(order, 1 << 40))
    order = torch.sort(order, dim=-1).values
    on = order < 1 << 40
    chosen = torch.where(on, order, torch.zeros_like(order))
    phys = tables[:, None].expand(B, K, -1).gather(2, chosen)
    blocks = torch.full((B, K, S), -1, dtype=torch.int32, device=q.device)
    out = blocks.clone()
    blocks[..., :order.shape[-1]] = torch.where(on, chosen, torch.full_like(chosen, -1)).int()
    out[..., :order.shape[-1]] = torch.where(on, phys, torch.full_like(phys, -1))
    return out, ((held - 1) * BS + ctx - (nb - 1) * BS).to(torch.int32), blocks


def _plain_sparse(st):
    case, q = st["case"], st["q"][:, 0].float()
    B, N, K, H, S = (case[x] for x in ("B", "N", "K", "H", "keep"))
    ids = st["tables"].clamp(min=0).long()
    head = torch.arange(K, device=q.device)[None, :, None, None]
    row = torch.arange(BS, device=q.device)
    k = st["kc"][ids[..., None], row, head].float().view(B, K, S * BS, H)
    v = st["vc"][ids[..., None], row, head].float().view(B, K, S * BS, H)
    off = torch.arange(S * BS, device=q.device) >= st["lens"][:, None, None, None]
    s = torch.matmul(q.view(B, K, N // K, H), k.transpose(2, 3)) * (H ** -0.5)
    s = s.masked_fill(off, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.view(B, 1, N, H).to(st["q"].dtype)


# ---- one pass ---------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"chunk": _plain_chunk, "rotary": _plain_rotary, "bounds": _plain_bounds,
                "select": _plain_select, "sparse": _plain_sparse}[op](st)
    import gqa_decode_attention_02_gb300 as gq

    if op == "chunk":
        return gq.chunk_attention(st["q"], st["kc"], st["vc"], st["tables"], st["ctx"], st["cu"],
                                  out=st["out"], window=case["window"])
    if op == "rotary":
        kw = dict(k_scale=st["ks"], v_scale=st["vs"], kv=case["kv"])
        q = gq.kv_append_rotary(st["q"], st["k"], st["v"], st["kc"], st["vc"], st["slots"],
                                st["places"], st["table"], q_out=st["q_out"],
                                interleaved=case["interleaved"], **kw)
        if case["kv"] == "same":
            return q, st["kc"], st["vc"]
        return (q,) + tuple(gq.kv_gather_slots(st["kc"], st["vc"], st["slots"],
                                               dtype=st["q"].dtype, **kw))
    if op == "bounds":
        gq.kv_block_bounds(st["kc"], st["tables"], st["ctx"], st["cu"], st["codes"], st["scale"])
        return st["codes"], st["scale"]
    if op == "select":
        return tuple(gq.select_blocks(st["q"], st["codes"], st["scale"], st["tables"], st["ctx"],
                                      case["keep"], first=case["first"], recent=case["recent"]))
    return gq.sparse_decode_attention(st["q"], st["kc"], st["vc"], st["tables"], st["lens"])


# ---- the operators' definitions in 64 bits ------------------------------------------------
def _exact_chunk(case, seed):
    st = _prepare_chunk(case, seed)
    N, K, H, W = (case[x] for x in ("N", "K", "H", "window"))
    G, out, at = N // K, torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b in range(case["B"]):
        n, c = st["new"][b], st["lens"][b]
        lo = max(0, c - n - W + 1) if W else 0
        pos = torch.arange(lo, c, device="cuda")
        blk, row = st["tables"][b][pos // BS].long(), pos % BS
        for h in range(K):
            k, v = st["kc"][blk, row, h].double(), st["vc"][blk, row, h].double()
            for t in range(0, n, 1024):
                m = min(1024, n - t)
                mine = torch.arange(c - n + t, c - n + t + m, device="cuda")
                seen = pos[None] <= mine[:, None]
                if W:
                    seen &= mine[:, None] - pos[None] < W
                for g in range(h * G, h * G + G):
                    s = st["q"][at + t:at + t + m, g].double() @ k.T / math.sqrt(H)
                    p = torch.softmax(torch.where(seen, s, torch.full_like(s, -math.inf)), -1)
                    out[at + t:at + t + m, g] = p @ v
        at += n
    return out


def _exact_rotary(case, seed):
    st = _prepare_rotary(case, seed)
    R, live = case["R"], st["places"] >= 0
    place = st["places"][live].long()
    c, s = st["table"][place, None, :R // 2].double(), st["table"][place, None, R // 2:].double()
    i = torch.arange(R // 2, device="cuda")
    one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)

    def turned(x):
        y = x.double().clone()
        y[..., one] = x[..., one].double() * c - x[..., two].double() * s
        y[..., two] = x[..., two].double() * c + x[..., one].double() * s
        return y

    q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    q[live] = turned(st["q"][live])
    if case["kv"] != "same":
        return q, None, None  # codes of what was rounded to 16 bits first
    caches = [x.double() for x in (st["kc"], st["vc"])]
    slot = st["slots"][live].long()
    caches[0].view(-1, case["K"], case["H"])[slot] = turned(st["k"][live])
    caches[1].view(-1, case["K"], case["H"])[slot] = st["v"][live].double()
    return (q,) + tuple(caches)


def _exact_sparse(case, seed):
    st = _prepare_sparse(case, seed)
    K, G, H = case["K"], case["N"] // case["K"], case["H"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_sparse_lens(case)):
        j = torch.arange(n, device="cuda")
        for h in range(K):
            blk = st["tables"][b, h][j // BS].long()
            k, v = st["kc"][blk, j % BS, h].double(), st["vc"][blk, j % BS, h].double()
            s = st["q"][b, 0, h * G:(h + 1) * G].double() @ k.T / math.sqrt(H)
            out[b, 0, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
    return out


def _exact_bounds(case, seed):
    st = _prepare_bounds(case, seed)
    scale = st["scale"].double()
    ids, ctx, cu = st["tables"].tolist(), st["ctx"].tolist(), st["cu"].tolist()
    at, held = [], []
    for b, c in enumerate(ctx):
        for i in range((c - cu[b + 1] + cu[b]) // BS, -(-c // BS)):
            at.append(ids[b][i])
            held.append(min(BS, c - i * BS))
    big = st["kc"][torch.tensor(at, device="cuda")].abs().amax(-1).double()
    none = torch.arange(BS, device="cuda")[None] >= torch.tensor(held, device="cuda")[:, None]
    scale[torch.tensor(at, device="cuda")] = big.masked_fill(none[..., None], 0.0).amax(1) / 127
    return None, scale  # (the codes are whole numbers, of divisions in 32 bits)


def exact(case, seed):
    """select: whole numbers of exact sums, nothing to be off by."""
    if case["op"] == "select":
        return None
    return {"chunk": _exact_chunk, "rotary": _exact_rotary, "bounds": _exact_bounds,
            "sparse": _exact_sparse}[case["op"]](case, seed)
