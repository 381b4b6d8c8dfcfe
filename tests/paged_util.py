"""Plain 64-bit forms of the paged-cache operators, and how far the kernels may
be from them.

Tolerances (elementwise). With p the softmax weights, A = sum p |v| and o the
result: a weight's relative error is that of its score's absolute error plus
that of 2^x. A score is a sum of d products with 32-bit sums, off by at most
(d + 2) 2^-24 sum |q k| / sqrt(d), and its multiplication by log2(e) / sqrt(d)
and the subtraction of the maximum round once each (2^-23 |s| together); 2^x
itself is within 2^-21. Sums over n keys in 32 bits add n 2^-24, rescaling once
per tile of 64 keys another 2^-23 each, and the final division 2^-22. Every
such error counts twice (numerator and sum). With bf16 inputs the weights are
rounded to bf16 before the product with V (half a step, 2^-8) and so is the
result (2^-8 |o|).
"""
import math

import torch

BF16_STEP = torch.finfo(torch.bfloat16).eps / 2


def attend(q, k, v, see):
    """q [n, Hq, d], k and v [L, Hkv, d], see [n, L] (bool): o [n, Hq, d] in 64
    bits and the tolerance of every element for inputs of q's dtype."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    o = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for h in range(Hq):
        qh, kh, vh = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        s = qh @ kh.T / math.sqrt(d)
        s = torch.where(see, s, torch.full_like(s, -math.inf))
        m = s.amax(-1, keepdim=True) if L else s.new_full((n, 1), -math.inf)
        p = torch.where(see, torch.exp(s - torch.where(m.isinf(), torch.zeros_like(m), m)),
                        torch.zeros_like(s))
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l == 0, torch.ones_like(l), l)
        o[:, h] = p @ vh
        a = p @ vh.abs()
        size = (qh.abs() @ kh.abs().T / math.sqrt(d)).where(see, torch.zeros_like(s))
        big = size.amax(-1, keepdim=True) if L else torch.zeros_like(l)
        w = 2 * ((d + 2) * 2.0 ** -24 * big + 2.0 ** -23 * big + 2.0 ** -21 + L * 2.0 ** -24
                 + (L / 64 + 1) * 2.0 ** -23 + 2.0 ** -22)
        if q.dtype == torch.bfloat16:
            tol[:, h] = (BF16_STEP + w) * a + BF16_STEP * o[:, h].abs()
        else:
            tol[:, h] = w * a + 2.0 ** -24 * o[:, h].abs()
    return o, tol


def check(got, want, tol):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} elements off, the worst by "
                           f"{float((err / tol.clamp_min(1e-300)).nan_to_num(9e9).max()):.2f} tolerances")


def gather(pool, row, n, blk):
    """The first n tokens of a block-table row: [n, Hkv, d]."""
    i = torch.arange(n, device=pool.device)
    return pool[row[i // blk].long(), :, i % blk]


def causal(n, ctx, device):
    """Row i of the last n of ctx tokens sees keys 0 .. ctx - n + i."""
    return torch.arange(ctx, device=device) <= torch.arange(ctx - n, ctx, device=device)[:, None]


def draft_mask(parents, T, device):
    see = torch.zeros(T, T, dtype=torch.bool, device=device)
    for t in range(T):
        u = t
        while u >= 0:
            see[t, u] = True
            u = parents[u] if parents is not None else u - 1
    return see


def nb(n, blk):
    return -(-n // blk)


def tables(blk, old, new, pinned, table, stack, count):
    """sv_build_tables on lists: (table, stack, count, cu, slots, positions).
    A page that is not there is -1."""
    table, stack = [list(r) for r in table], list(stack)
    for b in reversed(range(len(old))):
        for j in reversed(range(max(nb(new[b], blk), pinned[b]), nb(old[b], blk))):
            stack[count] = table[b][j]
            count += 1
    cu, slots, pos = [0], [], []
    for b in range(len(old)):
        for j in range(nb(old[b], blk), nb(new[b], blk)):
            count -= 1
            table[b][j] = stack[count] if count >= 0 else -1
        for p in range(old[b], new[b]):
            page = table[b][p // blk]
            slots.append(page * blk + p % blk if page >= 0 else -1)
            pos.append(p)
        cu.append(len(slots))
    return table, stack, max(count, 0), cu, slots, pos


def paged_pools(g, lens, Hkv, blk, d, dtype, spare=2, device="cuda", hole=float("nan")):
    """Pools whose pages are placed at random and hold `hole` wherever no
    sequence has a token, and the table (-1 past each row's own blocks)."""
    need = [nb(n, blk) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    k = torch.full((pages, Hkv, blk, d), hole, dtype=dtype)
    v = torch.full((pages, Hkv, blk, d), hole, dtype=dtype)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]].to(torch.int32)
        at += need[b]
        i = torch.arange(n)
        page = table[b].long()[i // blk]
        k[page, :, i % blk] = torch.randn(n, Hkv, d, generator=g).to(dtype)
        v[page, :, i % blk] = torch.randn(n, Hkv, d, generator=g).to(dtype)
    return k.to(device), v.to(device), table.to(device)
