"""The operators between a fused projection and attention over a 4-bit cache, as measured cases.

  rope    sv_norm_rope: norms of query and key heads and the position rotation, rows to rows
  append  sv_rope_write_kv: the same, keys rotated on the way into the paged cache, values beside them
  write4  sv_write_kv4 and sv_read_kv4: packed K/V rows into a 4-bit cache, and back out of it
  reps4   sv_build_reps_kv4: block representatives from 4-bit keys
  attend4 sv_attend_kv4: draft verification (one draft: a decoding step) over a 4-bit cache

A 4-bit cache holds, for every group of 16 dims of a head of a token, 16 E2M1 codes and one E4M3
scale: value = code * scale * 2^exponent of the head. Pools are [pages, Hkv, blk / 16, 9 d] bytes:
pieces of 16 tokens, their codes (8 d bytes), then their scales (d bytes).
  K codes [d / 16][16 tokens][8]: byte j holds dims 2j (low half) and 2j + 1; scales [16 tokens][d / 16]
  V codes [d / 16][8][16 tokens]: byte c holds dims c (low half) and c + 8;   scales [d / 16][16 tokens]

Lengths stand in a case as text ("1,77,300"), so that a case holds plain values only.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TREE16 = "-1,0,0,1,1,2,2,3,4,5,6,7,8,9,10,3"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _text(values):
    return ",".join(str(int(v)) for v in values)


def _blocks(n, blk):
    return -(-n // blk)


# ------------------------------------------------------------------ cases
def listed():
    gqa8 = {"dtype": "bf16", "Hq": 32, "Hkv": 8, "d": 128, "blk": 64}
    gqa4 = {"dtype": "bf16", "Hq": 32, "Hkv": 4, "d": 128, "blk": 64}
    tiny = {"dtype": "f32", "Hq": 8, "Hkv": 4, "d": 64, "blk": 16}
    return [
        # the drafts of one verification step: 4 sequences of 8, their keys not accepted yet
        {"name": "rope_drafts", "op": "rope", **gqa8, "n": 32, "pad": 0, "far": 131072, "rot": 128,
         "norm": False, "inter": False},
        # a long prompt's rows with normed heads
        {"name": "rope_prompt", "op": "rope", **gqa4, "n": 20011, "pad": 469, "far": 32768, "rot": 128,
         "norm": True, "inter": False},
        # one token of every sequence of a small batch, part of each head rotated, neighbours paired
        {"name": "append_step", "op": "append", **{**tiny, "d": 96}, "ctx": _text([17 + 61 * i for i in range(23)]),
         "new": _text([1] * 23), "pad": 9, "far": 4096, "rot": 64, "norm": True, "inter": True},
        # a batch of prompts, padded to a fixed number of rows as a captured step has it
        {"name": "append_prompts", "op": "append", **gqa8, "ctx": "4096,1,2500,8000,777,65",
         "new": "4096,1,2500,8000,777,65", "pad": 945, "far": 131072, "rot": 128, "norm": False,
         "inter": False},
        # the accepted token of every sequence of a decoding batch
        {"name": "write4_step", "op": "write4", **gqa8, "ctx": _text([1 + 211 * i for i in range(48)]),
         "new": _text([1] * 48), "pad": 16, "exps": True},
        # prompts into the 4-bit cache
        {"name": "write4_prompts", "op": "write4", **gqa8, "ctx": "6000,1,2500,4100,777,2000",
         "new": "6000,1,2500,4000,777,65", "pad": 57, "exps": False},
        # the blocks that one verification step filled
        {"name": "reps4_step", "op": "reps4", **gqa8, "ctx": _text([700 + 61 * i for i in range(32)]),
         "from": _text([693 + 61 * i for i in range(32)]), "exps": True},
        # every block of long prompts
        {"name": "reps4_prompts", "op": "reps4", **gqa8, "ctx": "131072,65536,100000,30001",
         "from": "0,0,0,0", "exps": False},
        # a decoding step of a ragged batch
        {"name": "attend4_decode", "op": "attend4", **gqa8, "T": 1, "parents": "", "sel": 0, "exps": True,
         "ctx": "8192,131,20000,1,32768,5000,12345,640,2047,16384,9999,64,30001,4097,700,15000"},
        # full verification of 8 drafts over long contexts
        {"name": "attend4_full_128k", "op": "attend4", **gqa8, "T": 8, "parents": "", "sel": 0,
         "exps": False, "ctx": "131072,131072,131072,131072"},
        # 16-node draft trees over selected blocks of long contexts
        {"name": "attend4_sparse_tree", "op": "attend4", **gqa4, "T": 16, "parents": TREE16, "sel": 64,
         "exps": False, "ctx": "65536,65500,64001,65536,50000,65599,60000,65536"},
        # fp32, small heads and pages, odd lengths
        {"name": "attend4_f32", "op": "attend4", **tiny, "T": 4, "parents": "", "sel": 0, "exps": True,
         "ctx": "1500,0,333,1,1000"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "write4", "reps4", "attend4", "attend4", "attend4"])
    Hq, Hkv, d = rng.choice([(32, 8, 128), (32, 4, 128), (32, 4, 64), (28, 4, 128), (8, 2, 96),
                             (16, 16, 128), (12, 12, 64), (6, 2, 256), (8, 8, 112)])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]), "Hq": Hq, "Hkv": Hkv, "d": d,
         "blk": rng.choice([16, 32, 64, 64])}
    if op in ("rope", "append"):
        c.update(far=rng.choice([4096, 32768, 131072]), rot=rng.choice([d, d, d // 2]),
                 norm=rng.choice([True, False]), inter=rng.choice([True, False, False]),
                 pad=rng.choice([0, rng.randint(1, 100)]))
    if op == "rope":
        return {**c, "n": _log(rng, 1, 16384)}
    if op == "append" or op == "write4":
        B = _log(rng, 1, 64)
        most = _log(rng, 1, 12000 // B)
        new = [rng.randint(1, most) for _ in range(B)]
        ctx = [n + rng.choice([0, rng.randint(0, 500)]) for n in new]
        c.update(ctx=_text(ctx), new=_text(new))
        if op == "append":
            return {**c, "far": max(c["far"], max(ctx))}
        return {**c, "pad": rng.choice([0, rng.randint(1, 64)]),
                "exps": rng.choice([True, False])}
    c["exps"] = rng.choice([True, False])
    if op == "reps4":
        B = _log(rng, 1, 32)
        most = _log(rng, 1, 260000 // B)
        ctx = [rng.randint(0, most) for _ in range(B)]
        ctx[0] = max(ctx[0], c["blk"])  # one block at least
        step = rng.choice([8, 100, most])
        return {**c, "ctx": _text(ctx), "from": _text([0] + [max(0, n - step) for n in ctx[1:]])}
    B, T = _log(rng, 1, 64), rng.choice([1, 1, 4, 8, 8, 16, 33])
    most = _log(rng, 1, (16384 if c["dtype"] == "f32" else 262144 if T <= 8 else 65536) // B)
    ctx = [min(most, _log(rng, 1, most + 1) - rng.choice([0, 1])) for _ in range(B)]
    parents = _text([-1] + [rng.randint(max(0, t - 3), t - 1) for t in range(1, T)])
    few = min(ctx) // c["blk"]
    return {**c, "T": T, "parents": rng.choice(["", parents]), "ctx": _text(ctx),
            "sel": rng.choice([0, _log(rng, 1, few)]) if few else 0}


def work(case):
    elt, d, Hq, Hkv = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hq"], case["Hkv"]
    token4 = Hkv * d * 9 // 16  # bytes of a token's keys (or values) in 4 bits
    if case["op"] == "rope":
        return {"bytes": case["n"] * (2 * (Hq + Hkv) * d * elt + 4 * case["rot"] + 4)}
    if case["op"] == "append":
        n = sum(_ints(case["new"]))
        return {"bytes": n * (2 * (Hq + 2 * Hkv) * d * elt + 4 * case["rot"] + 8)}
    if case["op"] == "write4":  # rows in, codes out; codes in, rows out
        return {"bytes": sum(_ints(case["new"])) * (4 * Hkv * d * elt + 4 * token4 + 8)}
    if case["op"] == "reps4":
        n = sum(c // case["blk"] - f // case["blk"] for c, f in zip(_ints(case["ctx"]), _ints(case["from"])))
        return {"bytes": n * (case["blk"] * token4 + 4 * Hkv * d)}
    T, ctx = case["T"], _ints(case["ctx"])
    keys = [case["sel"] * case["blk"] + c % case["blk"] if case["sel"] else c for c in ctx]
    seen = sum(_depths(_ints(case["parents"]) or [t - 1 for t in range(T)])) + T
    return {"bytes": 2 * sum(keys) * token4 + len(ctx) * T * (2 * Hkv + 2 * Hq) * d * elt,
            "flops": 4 * d * Hq * (T * sum(keys) + len(ctx) * seen)}


def _depths(parents):
    out = []
    for p in parents:
        out.append(0 if p < 0 else out[p] + 1)
    return out


# ------------------------------------------------------------------ inputs
def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _dev(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(g, lens, blk, spare):
    """A table whose rows hold randomly placed pages, and the number of pages."""
    need = [_blocks(n, blk) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need) + 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages


def _slots(table, ctx, new, blk, pad):
    """Slots of the last new[b] of ctx[b] tokens of every sequence, -1 behind them."""
    parts = []
    for b, (c, n) in enumerate(zip(ctx, new)):
        p = torch.arange(c - n, c, device="cuda")
        parts.append(table[b, p // blk] * blk + (p % blk).to(torch.int32))
    parts.append(torch.full((pad,), -1, dtype=torch.int32, device="cuda"))
    return torch.cat(parts).contiguous()


def _angles(far, rot):
    """Cosines and sines [far, rot] of every position, as a model keeps them."""
    freq = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pool4(g, pages, Hkv, blk, d, is_v):
    """A pool of quantised normal values, made some pages at a time."""
    out = torch.empty(pages, Hkv, blk // 16, 9 * d, dtype=torch.uint8, device="cuda")
    # keys have a few dims that are far larger than the others
    size = 1 + 7 * (torch.rand(Hkv, d, generator=g, device="cuda") > 0.96) * (not is_v)
    for at in range(0, pages, 512):
        x = _randn(g, min(512, pages - at), Hkv, blk // 16, 16, d, dtype=torch.float32)
        codes, scales = _quantise(x * size[:, None, None])
        out[at:at + 512] = _pack(codes, scales, is_v)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    op, dt, Hq, Hkv, d, blk = (case["op"], DTYPES[case["dtype"]], case["Hq"], case["Hkv"], case["d"],
                               case["blk"])
    s = {"case": case, "op": op, "blk": blk, "dtype": dt}
    if op in ("rope", "append", "write4"):
        if op == "rope":
            n, pos = case["n"], torch.randint(0, case["far"], (case["n"],), generator=g, device="cuda")
            pos = pos.to(torch.int32)
        else:
            ctx, new = _ints(case["ctx"]), _ints(case["new"])
            n, (table, pages) = sum(new), _pages(g, ctx, blk, 3)
            # a sequence may be far into its context: its positions count from there
            far = max(0, case.get("far", 0) - max(ctx))
            pos = torch.cat([torch.arange(c - m, c, device="cuda") + far * b // len(ctx)
                             for b, (c, m) in enumerate(zip(ctx, new))]).to(torch.int32)
            s["slots"] = _slots(table, ctx, new, blk, case["pad"])
        # a fused projection's rows: queries, keys and values side by side
        qkv = _randn(g, n + case["pad"], (Hq + 2 * Hkv) * d, dtype=dt)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        s.update(n=n, q=q, k=k, v=v)
        if op != "write4":
            s.update(pos=torch.cat([pos, pos.new_full((case["pad"],), -1)]),
                     table=_angles(case["far"], case["rot"]), q_out=torch.zeros(q.shape, dtype=dt, device="cuda"),
                     qw=1 + _randn(g, d, dtype=dt) / 8 if case["norm"] else None,
                     kw=1 + _randn(g, d, dtype=dt) / 8 if case["norm"] else None)
        if op != "append":
            s.update(k_out=torch.zeros(k.shape, dtype=dt, device="cuda"),
                     v_out=torch.zeros(k.shape, dtype=dt, device="cuda"))
        else:
            s.update(k_pool=_randn(g, pages, Hkv, blk, d, dtype=dt), v_pool=_randn(g, pages, Hkv, blk, d, dtype=dt))
    if op in ("write4", "reps4", "attend4"):
        e = torch.randint(-3, 4, (2, Hkv), generator=g, device="cuda").to(torch.int32)
        s.update(k_exp=e[0].contiguous() if case["exps"] else None,
                 v_exp=e[1].contiguous() if case["exps"] else None)
    if op == "write4":
        for name in ("k_pool", "v_pool"):
            s[name] = torch.zeros(pages, Hkv, blk // 16, 9 * d, dtype=torch.uint8, device="cuda")
        return s
    if op in ("reps4", "attend4"):
        ctx = _ints(case["ctx"])
        table, pages = _pages(g, ctx, blk, 3)
        s.update(ctx=ctx, seq_ctx=_dev(ctx), table=table, k_pool=_pool4(g, pages, Hkv, blk, d, False))
    if op == "reps4":
        start = _ints(case["from"])
        s.update(start=start, from_len=_dev(start), v_pool=s["k_pool"],
                 most=max(c // blk - f // blk for c, f in zip(ctx, start)),
                 reps=torch.zeros(len(ctx), Hkv, table.shape[1], d, device="cuda"))
    if op == "attend4":
        B, T = len(ctx), case["T"]
        s.update(T=T, parents=_ints(case["parents"]) or None, v_pool=_pool4(g, pages, Hkv, blk, d, True),
                 q=_randn(g, B, T, Hq, d, dtype=dt), draft_k=_randn(g, B, T, Hkv, d, dtype=dt),
                 draft_v=_randn(g, B, T, Hkv, d, dtype=dt), sel=None)
        s["out"] = torch.zeros_like(s["q"])
        if case["sel"]:  # what a selection keeps: distinct blocks, ascending, the first among them
            keep = []
            for c in ctx:
                score = torch.rand(Hkv, c // blk, generator=g, device="cuda")
                score[:, 0] = 2
                keep.append(score.topk(case["sel"]).indices.sort().values)
            s["sel"] = torch.stack(keep).to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------ plain forms
def _softmax_rows(s):
    """Softmax over the last axis."""
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _draft_mask(parents, T, device):
    see = torch.zeros(T, T, dtype=torch.bool)
    for t in range(T):
        u = t
        while u >= 0:
            see[t, u] = True
            u = parents[u] if parents else u - 1
    return see.to(device)


def _rotated(x, weight, s):
    """Rows x [n, heads, d], normed with `weight` and turned to their positions, in 32 bits."""
    rot, pos = s["case"]["rot"], s["pos"][:s["n"]].long()
    y = x[:s["n"]].float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
    cos, sin = s["table"][pos][:, None].split(rot // 2, -1)
    if s["case"]["inter"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    s["q_out"][:s["n"]] = _rotated(s["q"], s["qw"], s)
    s["k_out"][:s["n"]] = _rotated(s["k"], s["kw"], s)
    return [s["q_out"], s["k_out"]]


def _plain_append(s):
    s["q_out"][:s["n"]] = _rotated(s["q"], s["qw"], s)
    slots = s["slots"][:s["n"]].long()
    page, off = slots // s["blk"], slots % s["blk"]
    s["k_pool"][page, :, off] = _rotated(s["k"], s["kw"], s)
    s["v_pool"][page, :, off] = s["v"][:s["n"]]
    return [s["q_out"], s["k_pool"], s["v_pool"]]


def _quantise(x):
    """Codes [..., d] (uint8, 0 to 15) and scales [..., d / 16] (e4m3) of x [..., d]."""
    x = x.unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1) / 6).clamp_max(448).to(torch.float8_e4m3fn)
    step = scale.float()[..., None]
    m = torch.where(step > 0, x.abs() / step, torch.zeros_like(x))
    # halfway values go to the even code
    code = torch.zeros_like(m, dtype=torch.uint8)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                       (5.0, False)):
        code += m >= border if up else m > border
    return (code + 8 * (x < 0).to(torch.uint8)).flatten(-2), scale


def _pack(codes, scales, is_v):
    """Pieces [..., 16 tokens, d] of codes and [..., 16, d / 16] of scales as bytes [..., 9 d]."""
    c = codes.unflatten(-1, (-1, 16)).transpose(-3, -2)  # [..., group, token, 16]
    s = scales.view(torch.uint8)
    if is_v:
        c = (c[..., :8] | c[..., 8:] << 4).transpose(-2, -1)
        s = s.transpose(-2, -1)
    else:
        c = c[..., 0::2] | c[..., 1::2] << 4
    return torch.cat([c.flatten(-3), s.flatten(-2)], -1)


def _unpack(pieces, exp, is_v):
    """Values [..., 16 tokens, Hkv, d] in 32 bits of pieces [..., Hkv, 9 d]."""
    d = pieces.shape[-1] // 9
    value = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=pieces.device)
    c, s = pieces[..., :8 * d], pieces[..., 8 * d:].contiguous().view(torch.float8_e4m3fn).float()
    low, high = value[(c & 15).int()], value[(c >> 4).int()]
    if is_v:
        x = torch.cat([low.unflatten(-1, (-1, 8, 16)), high.unflatten(-1, (-1, 8, 16))], -2).transpose(-2, -1)
        s = s.unflatten(-1, (-1, 16))
    else:
        x = torch.stack([low, high], -1).flatten(-2).unflatten(-1, (-1, 16, 16))
        s = s.unflatten(-1, (16, -1)).transpose(-2, -1)
    x = (x * s[..., None]).transpose(-3, -2).flatten(-2)  # [..., Hkv, token, d]
    if exp is not None:
        x = x * torch.exp2(exp.float())[:, None, None]
    return x.transpose(-3, -2)


def _plain_write4(s):
    slots, d = s["slots"][:s["n"]].long(), s["case"]["d"]
    page, piece, tok = slots // s["blk"], slots % s["blk"] // 16, slots % 16
    for x, exp, pool, out, is_v in ((s["k"], s["k_exp"], s["k_pool"], s["k_out"], False),
                                    (s["v"], s["v_exp"], s["v_pool"], s["v_out"], True)):
        u = x[:s["n"]].float()
        if exp is not None:
            u = u * torch.exp2(-exp.float())[:, None]
        codes, scales = _quantise(u)
        # the pieces that the rows belong to, the rows' bytes put into them
        code = pool[..., :8 * d].unflatten(-1, (d // 16, 8, 16) if is_v else (d // 16, 16, 8))
        scale = pool[..., 8 * d:].unflatten(-1, (d // 16, 16) if is_v else (16, d // 16))
        c = codes.unflatten(-1, (-1, 16))
        if is_v:
            code[page, :, piece, :, :, tok] = c[..., :8] | c[..., 8:] << 4
            scale[page, :, piece, :, tok] = scales.view(torch.uint8)
        else:
            code[page, :, piece, :, tok] = c[..., 0::2] | c[..., 1::2] << 4
            scale[page, :, piece, tok] = scales.view(torch.uint8)
        back = _unpack(pool[page, :, piece], exp, is_v)
        out[:s["n"]] = back[torch.arange(s["n"], device=tok.device), tok].to(out.dtype)
    return [s["k_out"], s["v_out"]]


def _rows4(pool, exp, is_v, pages):
    """The tokens of some pages in 32 bits: [len(pages) * blk, Hkv, d]."""
    return _unpack(pool[pages].transpose(1, 2), exp, is_v).flatten(0, 2)


def _plain_reps4(s):
    blk = s["blk"]
    for b, (c, f) in enumerate(zip(s["ctx"], s["start"])):
        lo, hi = f // blk, c // blk
        if hi > lo:
            x = _rows4(s["k_pool"], s["k_exp"], False, s["table"][b, lo:hi].long())
            s["reps"][b, :, lo:hi] = x.unflatten(0, (-1, blk)).mean(1).transpose(0, 1)
    return s["reps"]


def _plain_attend4(s):
    case, blk, T, d = s["case"], s["blk"], s["T"], s["case"]["d"]
    G, dev = case["Hq"] // case["Hkv"], s["q"].device
    see = _draft_mask(s["parents"], T, dev)
    for b, c in enumerate(s["ctx"]):
        pages = s["table"][b, :_blocks(c, blk)].long()
        k = _rows4(s["k_pool"], s["k_exp"], False, pages)[:c]
        v = _rows4(s["v_pool"], s["v_exp"], True, pages)[:c]
        for h in range(case["Hkv"]):
            kh, vh = k[:, h], v[:, h]
            if s["sel"] is not None:
                where = (s["sel"][b, h].long()[:, None] * blk + torch.arange(blk, device=dev)).flatten()
                where = torch.cat([where, torch.arange(c // blk * blk, c, device=dev)])
                kh, vh = kh[where], vh[where]
            kh = torch.cat([kh, s["draft_k"][b, :, h].float()])
            vh = torch.cat([vh, s["draft_v"][b, :, h].float()])
            q = s["q"][b, :, h * G:(h + 1) * G].float().transpose(0, 1)  # [G, T, d]
            z = q @ kh.T * (1 / math.sqrt(d))
            z[:, :, -T:] = z[:, :, -T:].masked_fill(~see, -math.inf)
            s["out"][b, :, h * G:(h + 1) * G] = (_softmax_rows(z) @ vh).transpose(0, 1).to(s["dtype"])
    return s["out"]


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from sparse_verification_attention_gb300 import api

    c, op = s["case"], s["op"]
    B = len(s["ctx"]) if "ctx" in s else 1
    shape = api.make_shape(B, c["Hq"], c["Hkv"], c["d"], c["blk"], s.get("T", 1), s["dtype"])
    if op in ("rope", "append"):
        rope = api.make_rope(s["table"], c["rot"], c["inter"], s["qw"], s["kw"], 1e-6)
        if op == "rope":
            api.sv_norm_rope(shape, rope, s["pos"], s["q"], s["k"], s["q_out"], s["k_out"])
            return [s["q_out"], s["k_out"]]
        api.sv_rope_write_kv(shape, rope, s["pos"], s["q"], s["k"], s["v"], s["q_out"], s["slots"],
                             s["k_pool"], s["v_pool"])
        return [s["q_out"], s["k_pool"], s["v_pool"]]
    kv = api.make_kv4(s["k_pool"], s["v_pool"], s.get("table"), s.get("seq_ctx"), s["k_exp"], s["v_exp"])
    if op == "write4":
        api.sv_write_kv4(shape, s["k"], s["v"], s["slots"], kv)
        api.sv_read_kv4(shape, kv, s["slots"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    if op == "reps4":
        api.sv_build_reps_kv4(shape, kv, s["most"], s["reps"], s["from_len"])
        return s["reps"]
    if "ws" not in s:
        s["ws"] = api.alloc_kv4_workspace(shape)
    api.sv_attend_kv4(shape, s["q"], kv, s["sel"], s["draft_k"], s["draft_v"], s["parents"], s["out"], s["ws"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "write4": _plain_write4, "reps4": _plain_reps4,
            "attend4": _plain_attend4}[state["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_rope(s, x, w):
    """One pair of dims at a time, as complex numbers."""
    rot, n = s["case"]["rot"], s["n"]
    y = x[:n].double()
    if w is not None:
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
    t = s["table"].double()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if s["case"]["inter"] else (i, i + rot // 2)
        p = s["pos"][:n].long()
        z = torch.complex(y[..., a], y[..., b]) * torch.complex(t[p, i], t[p, rot // 2 + i])[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_value(x, e):
    """What 4 bits hold of x [n, Hkv, d], from the definition of the two formats."""
    if e is not None:
        x = x * (2.0 ** -e.double())[:, None]
    x = x.unflatten(-1, (-1, 16))
    t = x.abs().amax(-1, keepdim=True) / 6
    # e4m3: three bits behind the first one, steps of 2^-9 at least, 448 at most
    step = torch.exp2(torch.floor(torch.log2(t.clamp_min(2.0 ** -6))) - 3)
    scale = (torch.round(t / step) * step).clamp_max(448.0)
    # e2m1: one bit behind the first one, steps of 1/2 at least, 6 at most
    m = x / torch.where(scale > 0, scale, torch.ones_like(scale)) * (scale > 0)
    step = torch.exp2(torch.floor(torch.log2(m.abs().clamp_min(1.0))) - 1)
    y = ((torch.round(m / step) * step).clamp(-6, 6) * scale).flatten(-2)
    return y if e is None else y * (2.0 ** e.double())[:, None]


def _exact_page(pool, exp, is_v, pages, h):
    """Tokens [len(pages) * blk, d] of head h in 64 bits, each code taken apart into its bits."""
    d = pool.shape[-1] // 9
    x = pool[pages, h].flatten(0, 1)  # pieces of 16 tokens
    codes, sc = x[:, :8 * d], x[:, 8 * d:].long()
    scale = torch.where(sc & 0x78 > 0, (8 + (sc & 7)) * 2.0 ** ((sc >> 3 & 15).double() - 10), (sc & 7) * 2.0 ** -9)
    out = torch.empty(len(x), 16, d // 16, 16, dtype=torch.float64, device=x.device)  # piece, token, group, dim
    if is_v:
        n, scale = codes.unflatten(1, (-1, 8, 16)).permute(0, 3, 1, 2), scale.unflatten(1, (-1, 16)).transpose(1, 2)
    else:
        n, scale = codes.unflatten(1, (-1, 16, 8)).transpose(1, 2), scale.unflatten(1, (16, -1))
    for high in (0, 1):
        where = slice(8 * high, 8 * high + 8) if is_v else slice(high, None, 2)
        c = (n >> 4 if high else n & 15).int()
        mag = torch.where(c & 6 > 0, (2 + (c & 1)) * 2.0 ** ((c >> 1 & 3).double() - 2), (c & 1) * 0.5)
        out[..., where] = torch.where(c & 8 > 0, -mag, mag) * scale[..., None]
    out = out.flatten(2)
    out = out.flatten(0, 1)
    return out if exp is None else out * 2.0 ** exp[h].item()


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    if work(case).get("flops", 0) > 1e12:
        return None
    s = prepare(case, seed)
    blk, op = s["blk"], s["op"]
    if op == "rope" or op == "append":
        q = s["q_out"].double()
        q[:s["n"]] = _exact_rope(s, s["q"], s["qw"])
        k = _exact_rope(s, s["k"], s["kw"])
        if op == "rope":
            k_out = s["k_out"].double()
            k_out[:s["n"]] = k
            return [q, k_out]
        out = [s["k_pool"].double(), s["v_pool"].double()]
        for pool, x in zip(out, (k, s["v"][:s["n"]].double())):
            # one row a token: [pages * blk, Hkv, d]
            flat = pool.transpose(1, 2).flatten(0, 1).contiguous()
            flat[s["slots"][:s["n"]].long()] = x
            pool.copy_(flat.unflatten(0, (-1, blk)).transpose(1, 2))
        return [q] + out
    if op == "write4":
        out = [s["k_out"].double(), s["v_out"].double()]
        out[0][:s["n"]] = _exact_value(s["k"][:s["n"]].double(), s["k_exp"])
        out[1][:s["n"]] = _exact_value(s["v"][:s["n"]].double(), s["v_exp"])
        return out
    if op == "reps4":
        out = s["reps"].double()
        for b, (c, f) in enumerate(zip(s["ctx"], s["start"])):
            lo, hi = f // blk, c // blk
            for h in range(case["Hkv"] if hi > lo else 0):
                x = _exact_page(s["k_pool"], s["k_exp"], False, s["table"][b, lo:hi].long(), h)
                out[b, h, lo:hi] = x.view(hi - lo, blk, -1).sum(1) / blk
        return out
    G, T, out = case["Hq"] // case["Hkv"], s["T"], s["out"].double()
    bad = ~_draft_mask(s["parents"], T, "cuda")
    for b, c in enumerate(s["ctx"]):
        for h in range(case["Hkv"]):
            full, rest = torch.arange(c // blk, device="cuda"), c % blk
            if s["sel"] is not None:
                full = s["sel"][b, h].long()
            pages = s["table"][b].long()[torch.cat([full, full.new_tensor([c // blk] if rest else [])])]
            n = len(full) * blk + rest
            k = torch.cat([_exact_page(s["k_pool"], s["k_exp"], False, pages, h)[:n],
                           s["draft_k"][b, :, h].double()])
            v = torch.cat([_exact_page(s["v_pool"], s["v_exp"], True, pages, h)[:n],
                           s["draft_v"][b, :, h].double()])
            for qh in range(h * G, h * G + G):
                z = s["q"][b, :, qh].double() @ k.T / math.sqrt(case["d"])
                z[:, n:] = z[:, n:].masked_fill(bad, -math.inf)
                out[b, :, qh] = torch.exp(z - torch.logsumexp(z, -1, keepdim=True)) @ v
    return out
