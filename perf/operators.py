"""The paged-cache operators around verification, as measured cases.

  tables  sv_build_tables: pages for requests whose lengths change, and the slots of their new tokens
  write   sv_write_kv: packed K/V rows (slices of a fused projection) into the cache's pages
  prompt  sv_prompt_attend: causal attention of packed query rows over the paged cache
  prefix  sv_prefix_attend: verification of a batch whose sequences share their first blocks

Lengths stand in a case as text ("1,77,300"), so that a case holds plain values only.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TREE16 = "-1,0,0,1,1,2,2,3,4,5,6,7,8,9,10,3"


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _text(values):
    return ",".join(str(int(v)) for v in values)


def _blocks(n, blk):
    return -(-n // blk)


# ------------------------------------------------------------------ cases
def listed():
    llama = {"dtype": "bf16", "Hq": 32, "Hkv": 8, "d": 128, "blk": 64}
    qwen = {"dtype": "bf16", "Hq": 32, "Hkv": 4, "d": 128, "blk": 64}
    tiny = {"dtype": "f32", "Hq": 4, "Hkv": 2, "d": 64, "blk": 16}
    return [
        # one decoding step of a small batch: a few requests cross a page, one ends, one arrives
        {"name": "tables_step", "op": "tables", "blk": 64, "nb_max": 512, "pages": 4096,
         "old": "1000,640,77,0,8191,320,64,63", "new": "1008,648,0,131,8192,328,65,64", "pad": 200},
        # admission of a batch of prompts while others finish
        {"name": "tables_admit", "op": "tables", "blk": 16, "nb_max": 2048, "pages": 65536,
         "old": _text([0 if i % 4 else 900 + 37 * i for i in range(192)]),
         "new": _text([(211 * i) % 1021 + 1 if i % 4 else (0 if i % 8 else 905 + 37 * i)
                       for i in range(192)]), "pad": 0},
        # the accepted token of every sequence of a decoding batch
        {"name": "write_step", "op": "write", "dtype": "f32", "Hq": 8, "Hkv": 4, "d": 96, "blk": 32,
         "ctx": _text([17 + 61 * i for i in range(23)]), "new": _text([1] * 23), "pad": 9},
        # a batch of prompts, padded to a fixed number of rows as a captured step has it
        {"name": "write_prompts", "op": "write", **llama,
         "ctx": "4096,1,2500,8000,777,65", "new": "4096,1,2500,8000,777,65", "pad": 945},
        # one short question: latency
        {"name": "prompt_short", "op": "prompt", **llama, "ctx": "77", "new": "77", "pad": 0},
        # one token each of a ragged decoding batch
        {"name": "prompt_decode", "op": "prompt", **llama,
         "ctx": "8192,131,20000,1,32768,5000,12345,640,2047,16384,9999,64,30001,4097,700,15000",
         "new": _text([1] * 16), "pad": 0},
        # packed prompts of one prefill step, one row a cached sequence that only decodes
        {"name": "prompt_packed", "op": "prompt", **llama,
         "ctx": "6000,1,2500,4000,777,65,1500,9000", "new": "6000,1,2500,4000,777,65,1500,1",
         "pad": 156},
        # a whole long prompt
        {"name": "prompt_32k", "op": "prompt", **llama, "ctx": "32768", "new": "32768", "pad": 0},
        # fp32, small heads and pages, odd lengths
        {"name": "prompt_f32", "op": "prompt", **{**tiny, "Hq": 8}, "ctx": "1500,333,1,1000",
         "new": "1500,333,1,37", "pad": 3},
        # 16-node draft trees of 8 answers to one long document
        {"name": "prefix_tree16", "op": "prefix", **qwen, "T": 16, "parents": TREE16, "shared": 1024,
         "own_ctx": "1000,64,2049,0,700,3001,128,1500"},
        # single-token steps of 48 samples from one prompt
        {"name": "prefix_decode", "op": "prefix", **llama, "T": 1, "parents": "", "shared": 256,
         "own_ctx": _text([(397 * i) % 1900 for i in range(48)])},
        # fp32, small heads and pages
        {"name": "prefix_f32", "op": "prefix", **tiny, "T": 4, "parents": "", "shared": 63,
         "own_ctx": "40,0,333,16,1"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng):
    return rng.choice([(32, 8), (32, 4), (8, 2), (16, 16), (12, 4), (28, 4)])


def draw(rng):
    op = rng.choice(["tables", "write", "prompt", "prompt", "prompt", "prefix", "prefix"])
    if op == "tables":
        B, blk = _log(rng, 1, 256), rng.choice([16, 32, 64, 128])
        most = _log(rng, 2, 4096)
        old = [rng.choice([0, 1]) * rng.randint(0, most) for _ in range(B)]
        new = [rng.choice([0, n, n + 1, n + rng.randint(1, 8), rng.randint(0, most)]) for n in old]
        nb_max = _blocks(most + 8, blk) + rng.randint(0, 9)
        pages = sum(_blocks(max(x, y), blk) for x, y in zip(old, new)) + rng.randint(1, 500)
        return {"op": op, "blk": blk, "nb_max": nb_max, "pages": pages, "old": _text(old),
                "new": _text(new), "pad": rng.randint(0, 300)}
    Hq, Hkv = _heads(rng)
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]), "Hq": Hq, "Hkv": Hkv,
         "d": rng.choice([64, 96, 128, 128]), "blk": rng.choice([16, 32, 64, 64])}
    if op == "write":
        B = _log(rng, 1, 48)
        most = _log(rng, 1, 16384 // B)
        new = [rng.randint(1, most) for _ in range(B)]
        return {**c, "ctx": _text([n + rng.choice([0, rng.randint(0, 500)]) for n in new]),
                "new": _text(new), "pad": rng.choice([0, rng.randint(1, 64)])}
    if op == "prompt":
        kind = rng.choice(["decode", "whole", "chunk"])
        if kind == "decode":
            B = _log(rng, 1, 64)
            new, cached = [1] * B, [_log(rng, 1, 32768) - 1 for _ in range(B)]
        elif kind == "whole":
            B = _log(rng, 1, 12)
            new = [_log(rng, 1, 8192) for _ in range(B)]
            cached = [0] * B
        else:
            B = _log(rng, 1, 4)
            new = [_log(rng, 2, 1024) for _ in range(B)]
            cached = [_log(rng, 1, 32768) for _ in range(B)]
        if c["dtype"] == "f32":  # what a 32-bit check of a model runs: shorter
            new, cached = [max(1, n // 4) for n in new], [n // 4 for n in cached]
        return {**c, "ctx": _text([x + y for x, y in zip(new, cached)]), "new": _text(new),
                "pad": rng.choice([0, rng.randint(1, 100)])}
    B, T = _log(rng, 2, 48), rng.choice([1, 4, 8, 8, 16])
    if T * B > 256:
        B = 256 // T
    most = _log(rng, 1, 2500)
    shared = _log(rng, 1, (4096 if c["dtype"] == "f32" else 32768) // c["blk"])
    parents = _text([-1] + [rng.randint(max(0, t - 3), t - 1) for t in range(1, T)])
    return {**c, "T": T, "parents": rng.choice(["", parents]), "shared": shared,
            "own_ctx": _text([rng.randint(0, most) for _ in range(B)])}


def work(case):
    if case["op"] == "tables":
        blk, old, new = case["blk"], _ints(case["old"]), _ints(case["new"])
        tokens = sum(max(0, y - x) for x, y in zip(old, new))
        moved = sum(abs(_blocks(y, blk) - _blocks(x, blk)) for x, y in zip(old, new))
        # lengths, pinned counts and offsets; every moved page read and written; slots and positions
        return {"bytes": 4 * (4 * len(old) + 2 * moved + 2 * (tokens + case["pad"]) + 3)}
    elt, d, Hq, Hkv = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hq"], case["Hkv"]
    if case["op"] == "write":
        n = sum(_ints(case["new"]))
        return {"bytes": 4 * n * Hkv * d * elt + 4 * (n + case["pad"])}
    if case["op"] == "prompt":
        ctx, new = _ints(case["ctx"]), _ints(case["new"])
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for c, n in zip(ctx, new))
        return {"bytes": 2 * sum(ctx) * Hkv * d * elt + 2 * sum(new) * Hq * d * elt,
                "flops": 4 * d * Hq * pairs}
    T, P, mine = case["T"], case["shared"] * case["blk"], _ints(case["own_ctx"])
    parents = _ints(case["parents"]) or [t - 1 for t in range(T)]
    seen = sum(_depths(parents)) + T
    return {"bytes": 2 * (P + sum(mine) + len(mine) * T) * Hkv * d * elt
            + 2 * len(mine) * T * Hq * d * elt,
            "flops": 4 * d * Hq * (sum(T * (P + n) for n in mine) + len(mine) * seen)}


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


def _paged(g, lens, blk, spare):
    """A table whose rows hold randomly placed pages, and the number of pages."""
    need = [_blocks(n, blk) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need) + 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages, perm[at:]


def _slots(table, ctx, new, blk, pad):
    """Slots of the last new[b] of ctx[b] tokens of every sequence, -1 behind them."""
    parts = []
    for b, (c, n) in enumerate(zip(ctx, new)):
        p = torch.arange(c - n, c, device="cuda")
        parts.append(table[b, p // blk] * blk + (p % blk).to(torch.int32))
    parts.append(torch.full((pad,), -1, dtype=torch.int32, device="cuda"))
    return torch.cat(parts).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    s = {"case": case, "op": case["op"], "blk": case["blk"]}
    if case["op"] == "tables":
        blk, old, new = case["blk"], _ints(case["old"]), _ints(case["new"])
        held = [_blocks(n, blk) for n in old]
        perm = torch.randperm(case["pages"], generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(old), case["nb_max"]), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = perm[at:at + n]
            at += n
        stack = torch.zeros(case["pages"], dtype=torch.int32, device="cuda")
        stack[:case["pages"] - at] = perm[at:]
        tokens = sum(max(0, y - x) for x, y in zip(old, new)) + case["pad"]
        s.update(table=table, stack=stack, count=_dev([case["pages"] - at]), count_out=_dev([0]),
                 old=_dev(old), new=_dev(new), cu=_dev([0] * (len(old) + 1)),
                 slots=_dev([0] * max(tokens, 1)), pos=_dev([0] * max(tokens, 1)),
                 # every third finished request keeps its first block, as one shared with others
                 pinned=_dev([1 if n == 0 and b % 3 == 0 else 0 for b, n in enumerate(new)]))
        return s
    dt, Hq, Hkv, d = DTYPES[case["dtype"]], case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "prefix":
        T, P, mine = case["T"], case["shared"] * case["blk"], _ints(case["own_ctx"])
        tails, pages, spare = _paged(g, mine, case["blk"], case["shared"] + 3)
        table = torch.cat([spare[:case["shared"]].expand(len(mine), -1), tails], 1).contiguous()
        s.update(ctx=[P + n for n in mine], T=T, parents=_ints(case["parents"]) or None, table=table,
                 q=_randn(g, len(mine), T, Hq, d, dtype=dt),
                 draft_k=_randn(g, len(mine), T, Hkv, d, dtype=dt),
                 draft_v=_randn(g, len(mine), T, Hkv, d, dtype=dt))
        s["out"] = torch.zeros_like(s["q"])
    else:
        ctx, new = _ints(case["ctx"]), _ints(case["new"])
        table, pages, _ = _paged(g, ctx, case["blk"], 3)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        # a fused projection's rows: queries, keys and values side by side
        qkv = _randn(g, starts[-1] + case["pad"], (Hq + 2 * Hkv) * d, dtype=dt)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        s.update(ctx=ctx, new=new, n=starts[-1], table=table, q=q, k=k, v=v, seq_ctx=_dev(ctx),
                 cu=_dev(starts), starts=starts)
        if case["op"] == "write":
            s["slots"] = _slots(table, ctx, new, case["blk"], case["pad"])
        else:
            s["out"] = torch.zeros(q.shape, dtype=dt, device="cuda")
    s["k_pool"] = _randn(g, pages, Hkv, case["blk"], d, dtype=dt)
    s["v_pool"] = _randn(g, pages, Hkv, case["blk"], d, dtype=dt)
    return s


# ------------------------------------------------------------------ plain forms
def _softmax_rows(s):
    """Softmax over the last axis; a row without any key is zero."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _attend(q, k, v, see):
    """q [B, n, Hq, d]; k, v [B, L, Hkv, d]; see [B, n, L]: in 32 bits, one KV head at a time."""
    B, n, Hq, d = q.shape
    G = Hq // k.shape[2]
    out = torch.empty(B, n, Hq, d, dtype=torch.float32, device=q.device)
    for h in range(k.shape[2]):
        qh = q[:, :, h * G:(h + 1) * G].float().permute(0, 2, 1, 3)
        s = qh @ k[:, None, :, h].float().transpose(-1, -2) * (1 / math.sqrt(d))
        p = _softmax_rows(s.masked_fill(~see[:, None], -math.inf))
        out[:, :, h * G:(h + 1) * G] = (p @ v[:, None, :, h].float()).permute(0, 2, 1, 3)
    return out.to(q.dtype)


def _gather(pool, table, n, blk):
    """The first n tokens of every row of `table`, [B, n, Hkv, d]."""
    rows = pool[table[:, :_blocks(n, blk)].long()].transpose(2, 3)
    return rows.flatten(1, 2)[:, :n]


def _plain_prompt(s):
    ctx, new, blk, dev = s["ctx"], s["new"], s["blk"], s["q"].device
    if max(new) == 1 and sum(ctx) * 4 > len(ctx) * max(ctx):
        L = max(ctx)  # one token each: the batch at once, padded to the longest
        see = torch.arange(L, device=dev) < s["seq_ctx"][:, None]
        s["out"][:s["n"]] = _attend(s["q"][:s["n"], None], _gather(s["k_pool"], s["table"], L, blk),
                                    _gather(s["v_pool"], s["table"], L, blk), see[:, None])[:, 0]
        return s["out"]
    for b, (c, n) in enumerate(zip(ctx, new)):
        rows, t = slice(s["starts"][b], s["starts"][b] + n), s["table"][b:b + 1]
        see = torch.arange(c, device=dev) <= torch.arange(c - n, c, device=dev)[:, None]
        s["out"][rows] = _attend(s["q"][rows][None], _gather(s["k_pool"], t, c, blk),
                                 _gather(s["v_pool"], t, c, blk), see[None])[0]
    return s["out"]


def _draft_mask(parents, T, device):
    see = torch.zeros(T, T, dtype=torch.bool)
    for t in range(T):
        u = t
        while u >= 0:
            see[t, u] = True
            u = parents[u] if parents else u - 1
    return see.to(device)


def _plain_prefix(s):
    ctx, blk, T, dev = s["ctx"], s["blk"], s["T"], s["q"].device
    B, L = len(ctx), max(s["ctx"])
    # the batch at once, padded to the longest context, its drafts behind it
    k = torch.cat([_gather(s["k_pool"], s["table"], L, blk), s["draft_k"]], 1)
    v = torch.cat([_gather(s["v_pool"], s["table"], L, blk), s["draft_v"]], 1)
    see = torch.arange(L, device=dev) < torch.tensor(ctx, device=dev)[:, None]
    see = torch.cat([see[:, None].expand(B, T, L),
                     _draft_mask(s["parents"], T, dev)[None].expand(B, T, T)], 2)
    s["out"].copy_(_attend(s["q"], k, v, see))
    return s["out"]


def _plain_write(s):
    slots = s["slots"][:s["n"]].long()
    page, off = slots // s["blk"], slots % s["blk"]
    s["k_pool"][page, :, off] = s["k"][:s["n"]]
    s["v_pool"][page, :, off] = s["v"][:s["n"]]
    return [s["k_pool"], s["v_pool"]]


def _plain_tables(s):
    blk, table, stack, dev = s["blk"], s["table"], s["stack"], s["table"].device
    old, new = s["old"].long(), s["new"].long()
    held, need = (old + blk - 1) // blk, (new + blk - 1) // blk
    j = torch.arange(table.shape[1], device=dev)
    drop = ((j >= torch.maximum(need, s["pinned"].long())[:, None]) & (j < held[:, None])).flatten()
    take = ((j >= held[:, None]) & (j < need[:, None])).flatten()
    count, dropped = s["count"].long(), drop.sum()
    # what is let go is pushed from the last block of the last request to the first of the first
    at = count + dropped - drop.cumsum(0)
    grown = torch.cat([stack, stack.new_zeros(1)])
    grown[torch.where(drop, at, len(stack))] = table.flatten()
    stack.copy_(grown[:-1])
    # what is needed is taken from the top, from the first block of the first request on
    top = (count + dropped - take.cumsum(0)).clamp_min(0)
    table.copy_(torch.where(take, stack[top], table.flatten()).view_as(table))
    s["count_out"].copy_((count + dropped - take.sum()).to(torch.int32))
    s["cu"][1:] = (new - old).clamp_min(0).cumsum(0)
    i = torch.arange(len(s["slots"]), device=dev)
    b = torch.searchsorted(s["cu"][1:].long(), i, right=True).clamp_max(len(old) - 1)
    pos, real = old[b] + i - s["cu"][b], i < s["cu"][-1]
    slot = table[b, (pos // blk).clamp(0, table.shape[1] - 1)] * blk + pos % blk
    s["slots"].copy_(torch.where(real, slot, -1))
    s["pos"].copy_(torch.where(real, pos, -1))
    return _tables_out(s)


def _tables_out(s):
    return [s["table"], s["stack"], s["count_out"], s["cu"], s["slots"], s["pos"]]


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from sparse_verification_attention_gb300 import api

    c = s["case"]
    if s["op"] == "tables":
        api.sv_build_tables(s["blk"], s["old"], s["new"], s["table"], s["stack"], s["count"],
                            s["count_out"], s["cu"], s["slots"], s["pos"], pinned=s["pinned"])
        return _tables_out(s)
    T = s.get("T", 1)
    shape = api.make_shape(len(s["ctx"]), c["Hq"], c["Hkv"], c["d"], c["blk"], T, DTYPES[c["dtype"]])
    if s["op"] == "write":
        api.sv_write_kv(shape, s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"])
        return [s["k_pool"], s["v_pool"]]
    if s["op"] == "prompt":
        if "ws" not in s:
            s["ws"] = api.alloc_prompt_workspace(shape, s["q"].shape[0])
        api.sv_prompt_attend(shape, s["q"], s["k_pool"], s["v_pool"], s["table"], s["seq_ctx"],
                             s["cu"], s["out"], s["ws"])
        return s["out"]
    if "ws" not in s:
        s["ws"] = api.alloc_prefix_workspace(shape)
    kv = api.make_kv(s["k_pool"], s["v_pool"], s["table"], 0, s["ctx"])
    api.sv_prefix_attend(shape, s["q"], kv, c["shared"], s["draft_k"], s["draft_v"], s["parents"],
                         s["out"], s["ws"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "write": _plain_write, "prompt": _plain_prompt,
            "prefix": _plain_prefix}[state["op"]](state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, one request and one query head at a time."""
    w = work(case)
    if w.get("flops", 0) > 2.5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    if case["op"] == "write":
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        i, table = 0, s["table"].tolist()
        for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
            for at in range(c - n, c):  # at the first token of every page that it reaches
                if at == c - n or at % s["blk"] == 0:
                    end = min(c, (at // s["blk"] + 1) * s["blk"])
                    page, off = table[b][at // s["blk"]], at % s["blk"]
                    rows = slice(i, i + end - at)
                    kp[page, :, off:off + end - at] = s["k"][rows].double().transpose(0, 1)
                    vp[page, :, off:off + end - at] = s["v"][rows].double().transpose(0, 1)
                    i += end - at
        return [kp, vp]
    G, blk, root = case["Hq"] // case["Hkv"], s["blk"], 1 / math.sqrt(case["d"])
    out = s["out"].double()
    for b, c in enumerate(s["ctx"]):
        where = torch.arange(c, device="cuda")
        page, off = s["table"][b].long()[where // blk], where % blk
        for qh in range(case["Hq"]):
            k, v = s["k_pool"][page, qh // G, off].double(), s["v_pool"][page, qh // G, off].double()
            if case["op"] == "prompt":
                n, at = s["new"][b], s["starts"][b]
                q = s["q"][at:at + n, qh].double()
                bad = where[None] > torch.arange(c - n, c, device="cuda")[:, None]
            else:
                q = s["q"][b, :, qh].double()
                k = torch.cat([k, s["draft_k"][b, :, qh // G].double()])
                v = torch.cat([v, s["draft_v"][b, :, qh // G].double()])
                bad = torch.cat([torch.zeros(s["T"], c, dtype=torch.bool, device="cuda"),
                                 ~_draft_mask(s["parents"], s["T"], "cuda")], 1)
            z = (q @ k.T * root).masked_fill(bad, -math.inf)
            o = torch.exp(z - torch.logsumexp(z, -1, keepdim=True)) @ v
            if case["op"] == "prompt":
                out[at:at + n, qh] = o
            else:
                out[b, :, qh] = o
    return out


def _exact_tables(s):
    blk = s["blk"]
    table, stack = s["table"].tolist(), s["stack"].tolist()
    old, new, pinned = s["old"].tolist(), s["new"].tolist(), s["pinned"].tolist()
    top = s["count"].item()
    for b in reversed(range(len(old))):
        for j in reversed(range(max(_blocks(new[b], blk), pinned[b]), _blocks(old[b], blk))):
            stack[top] = table[b][j]
            top += 1
    cu, slots, pos = [0], [], []
    for b in range(len(old)):
        for j in range(_blocks(old[b], blk), _blocks(new[b], blk)):
            top -= 1
            table[b][j] = stack[top]
        for p in range(old[b], new[b]):
            slots.append(table[b][p // blk] * blk + p % blk)
            pos.append(p)
        cu.append(len(slots))
    rest = [-1] * (len(s["slots"]) - len(slots))
    return [_dev(v) for v in (table, stack, [top], cu, slots + rest, pos + rest)]
