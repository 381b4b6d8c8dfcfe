"""Plain 64-bit forms of head norms with rotation and of the 4-bit cache, and how
far the kernels may be from them.

Tolerances (elementwise), u = 2^-24 half a step of fp32.
Rotation: an output a c - b s of normed elements a, b takes two products and a sum,
3 u of |a c| + |b s|; the norm multiplies twice (2 u), its sum of d squares is off
by d u, halved by the root, and the division, root and sums around it by less than
8 u. Together (d / 2 + 16) u of |a c| + |b s|, and half a step of the output's type.
4-bit values: the rounding is defined bit by bit and the values are exact.
Representatives: blk sums on the tensor cores, which may cut off instead of rounding (a
whole step, 2 u, each), and a factor: (2 blk + 2) u of the mean of |x|.
Attention: as in paged_util.attend for the scores, weights, sums and the division;
scores may be summed with whole steps (2 u) on the tensor cores. There a weight is
rounded to f16, 2^-11 of it, and below f16's normal range by half a step of 2^-24 at
most; weights are held 2^7 times their size against a reference that no score
before it exceeds, so the latter is 2^-32 of the largest weight for every key.
"""
import math

import torch

U = 2.0 ** -24
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ rotation
def rope(x, weight, eps, table, rot, inter, pos):
    """Rows x [n, heads, d] normed and rotated, in 64 bits, and the tolerance."""
    n, _, d = x.shape
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
    out, size = y.clone(), y.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = (table[pos.long(), j].double()[:, None] for j in (i, rot // 2 + i))
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        size[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
        size[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    tol = (d / 2 + 16) * U * size + half_step(x.dtype) * out.abs()
    return out, tol


# ------------------------------------------------------------------ formats
def e4m3_values():
    """The value of every scale byte below 128 (the last is NaN)."""
    v = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)]
    v[127] = math.nan
    return torch.tensor(v, dtype=torch.float64)


def nearest_even(x, values):
    """Index of the nearest of the ascending `values`, the even index of two as near."""
    hi = torch.searchsorted(values, x).clamp(1, len(values) - 1)
    lo = hi - 1
    up, down = values[hi] - x, x - values[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise(x, exp=None):
    """Codes [..., H, d] and scale bytes [..., H, d / 16] of rows x [..., H, d]."""
    u = x.double()
    if exp is not None:
        u = u * torch.exp2(-exp.double())[:, None]
    u = u.unflatten(-1, (-1, 16))
    nan = u.isnan().any(-1)
    values = e4m3_values()[:127].to(u.device)
    # 32-bit elements: amax / 6 in 64 bits lies on a border only if it is one
    sb = nearest_even((u.nan_to_num(0.0, math.inf, -math.inf).abs().amax(-1) / 6).clamp_max(448.0), values)
    scale = values[sb][..., None]
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=u.device)
    m = torch.where(scale > 0, (u.abs() / scale).nan_to_num(0.0, 9.0).clamp_max(6.0), torch.zeros_like(u))
    code = nearest_even(m, levels) + 8 * ((u < 0) & (scale > 0))
    return code.flatten(-2), torch.where(nan, torch.full_like(sb, 127), sb)


def values(code, sb, exp=None):
    """The values of codes [..., H, d] and scale bytes [..., H, d / 16], in 64 bits."""
    levels = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device=code.device)
    v = (levels[code.long()].unflatten(-1, (-1, 16)) * e4m3_values().to(code.device)[sb.long()][..., None]).flatten(-2)
    return v if exp is None else v * torch.exp2(exp.double())[:, None]


def byte_of(d, dim, tok, is_v):
    """Where code `dim` of token tok stands in a piece: byte, high half?"""
    g, i = divmod(dim, 16)
    return (g * 128 + i % 8 * 16 + tok, i >= 8) if is_v else (g * 128 + tok * 8 + i // 2, i % 2 == 1)


def scale_of(d, g, tok, is_v):
    return 8 * d + (g * 16 + tok if is_v else tok * (d // 16) + g)


def put(pool, page, tok_in_page, code, sb, is_v):
    """Write one token's codes [H, d] and scale bytes into a pool (CPU)."""
    d = pool.shape[-1] // 9
    piece, tok = divmod(tok_in_page, 16)
    p = pool[page, :, piece]
    for dim in range(d):
        at, high = byte_of(d, dim, tok, is_v)
        keep = 15 if high else 240
        p[:, at] = (p[:, at] & keep) | (code[:, dim].to(torch.uint8) << (4 if high else 0))
    for g in range(d // 16):
        p[:, scale_of(d, g, tok, is_v)] = sb[:, g].to(torch.uint8)


def put_rows(pool, slots, blk, code, sb, is_v):
    for i, s in enumerate(slots):
        if s >= 0:
            put(pool, s // blk, s % blk, code[i], sb[i], is_v)


def pools(g, lens, Hkv, blk, d, spare=2, hole=0xff, k_exp=None, v_exp=None, size=1.0):
    """A 4-bit cache of random rows: byte pools whose unused bytes are `hole` (0xff: a NaN
    scale), the table, and every sequence's rows as the cache holds them, in 64 bits
    (k [L, Hkv, d], v). CPU tensors. Pools are put together piecewise from the layout."""
    need = [-(-n // blk) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    out = []
    for exp, is_v in ((k_exp, False), (v_exp, True)):
        flat = torch.full((pages * (blk // 16), Hkv, 9 * d), hole, dtype=torch.uint8)  # by piece
        at, rows = 0, []
        for b, n in enumerate(lens):
            table[b, :need[b]] = perm[at:at + need[b]].to(torch.int32)
            at += need[b]
            x = (torch.randn(n, Hkv, d, generator=g) * size).float()
            code, sb = quantise(x, exp)
            rows.append(values(code, sb, exp))
            i = torch.arange(n)
            piece = table[b].long()[i // blk] * (blk // 16) + i % blk // 16
            tok = i % 16
            for dim in range(0, d, 1):
                where, high = byte_of(d, dim, 0, is_v)
                col = where + tok * (1 if is_v else 8)
                old = flat[piece, :, col]
                new = code[:, :, dim].to(torch.uint8)
                flat[piece, :, col] = (old & 15 | new << 4) if high else (old & 240 | new)
            for gr in range(d // 16):
                flat[piece, :, scale_of(d, gr, 0, is_v) + tok * (1 if is_v else d // 16)] = sb[:, :, gr].to(torch.uint8)
        out.append((flat.unflatten(0, (pages, blk // 16)).transpose(1, 2).contiguous(), rows))
    (kp, k), (vp, v) = out
    return kp, vp, table, k, v


# ------------------------------------------------------------------ attention
def attend(q, k, v, see, f16):
    """q [n, Hq, d], k and v [L, Hkv, d] (64 bits), see [n, Hkv, L]: o [n, Hq, d] in 64 bits
    and the tolerance; f16: the tensor cores' roundings."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    o = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        qh, kh, vh, on = q[:, h].double(), k[:, kv], v[:, kv], see[:, kv]
        s = (qh @ kh.T / math.sqrt(d)).masked_fill(~on, -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        l = p.sum(-1, keepdim=True)
        o[:, h] = p / l @ vh
        a = p / l @ vh.abs()
        big = (qh.abs() @ kh.abs().T / math.sqrt(d)).masked_fill(~on, 0).amax(-1, keepdim=True)
        w = 2 * ((d + 2) * (2 if f16 else 1) * U * big + 2 * U * big + 8 * U + L * U + (L / 64 + 1) * 2 * U + 4 * U)
        if f16:
            w = w + 2.0 ** -11
            tol[:, h] += 2.0 ** -32 * (on.double() @ vh.abs())
        tol[:, h] += w * a + half_step(q.dtype) * o[:, h].abs()
    return o, tol


def check(got, want, tol):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} elements off, the worst by "
                           f"{float((err / tol.clamp_min(1e-300)).nan_to_num(9e9).max()):.2f} tolerances")
