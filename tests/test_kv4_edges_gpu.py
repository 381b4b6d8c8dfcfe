"""The 4-bit cache's attention where rows, lengths or sizes go wrong first: rows that are
not finite beside others, references of the softmax that have to move, very large and very
small queries. Against the 64-bit forms of tests/kv4_util.py (where the tolerances stand)."""
import math

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib
from tests import kv4_util as U
from tests import paged_util as P

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    api.lib()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def cache(g, s, k, v, k_exp=None):
    """A 4-bit cache of the rows k, v [B, n, Hkv, d] on pages in any order, and the rows as
    the cache holds them, in 64 bits."""
    B, n, H, d = k.shape
    blk = s.blk
    nb = -(-n // blk)
    table = torch.randperm(B * nb, generator=g, device="cuda").to(torch.int32).view(B, nb)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    kv = api.make_kv4(*[api.alloc_kv4_pool(s, B * nb) for _ in range(2)], table, lens, k_exp)
    i = torch.arange(n, device="cuda")
    slots = (table.long()[:, i // blk] * blk + i % blk).flatten().to(torch.int32)
    rows = [x.flatten(0, 1) for x in (k, v)]
    api.sv_write_kv4(s, *rows, slots, kv)
    held = [U.values(*U.quantise(x, e), e).view(B, n, H, d) for x, e in zip(rows, (k_exp, None))]
    return kv, *held


def attend(s, q, kv, dk, dv):
    out, ws = torch.full_like(q, 7), api.alloc_kv4_workspace(s)
    api.sv_attend_kv4(s, q, kv, None, dk, dv, None, out, ws)
    assert api.sv_read_status(ws) == 0
    return out


def all_keys(T, Hkv, n):
    see = torch.ones(T, Hkv, n + T, dtype=torch.bool)
    see[:, :, n:] = P.draft_mask(None, T, "cpu")[:, None]
    return see.cuda()


# ------------------------------------------------------------------ rows that are not finite
# A head's stacked row is r = t * G + g. The tensor cores' softmax has rows 8 j + 2 i and
# 8 j + 2 i + 1 (i fixed) in one thread.
def mates(r):
    return [x for x in range(64) if x % 8 // 2 == r % 8 // 2]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,G,row", [(16, 4, 0), (16, 4, 27), (8, 4, 9), (4, 4, 14), (3, 5, 2)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_a_row_that_is_not_finite_reaches_no_other(dtype, T, G, row, what):
    """The rows that share their threads with it have scores that rise all the way, a dozen
    powers of two in a tile of 128 keys, so that each share of the keys moves their references
    many times; the other rows' scores stay small and move none."""
    B, Hkv, d, n, blk = 8, 8, 128, 3000, 64
    g = gen(row + T)
    s = api.make_shape(B, G * Hkv, Hkv, d, blk, T, dtype)
    k, v = randn(g, B, n, Hkv, d) / 2, randn(g, B, n, Hkv, d)
    # 16 dims of 3 in the rows: 48 k / sqrt(128) log2(e) = 6.1 k
    k[..., :16] = (torch.arange(n, device="cuda") * (2 / 128))[None, :, None, None]
    kv, hk, hv = cache(g, s, k.to(dtype), v.to(dtype))
    q = randn(g, B, T, Hkv, G, d) / 2
    q[..., :16] = 0
    for r in mates(row):
        if r < T * G:
            q[:, r // G, :, r % G, :16] = 3
    q = q.to(dtype)
    dk, dv = (randn(g, B, T, Hkv, d).to(dtype) for _ in range(2))
    dk[..., :16] = 0
    odd = q.clone()
    odd[:, row // G, :, row % G] = what
    q[:, row // G, :, row % G] = 0
    got, plain = (attend(s, x.flatten(2, 3), kv, dk, dv).view(B, T, Hkv, G, d) for x in (odd, q))
    assert got[:, row // G, :, row % G].isnan().all()
    rest = torch.ones(T, Hkv, G, dtype=torch.bool, device="cuda")
    rest[row // G, :, row % G] = False
    if math.isnan(what):  # such a row takes no part in when references move
        assert torch.equal(got[:, rest], plain[:, rest])
    see = all_keys(T, Hkv, n)
    for b in range(B):
        o, tol = U.attend(q[b].flatten(1, 2), torch.cat([hk[b], dk[b].double()]), torch.cat([hv[b], dv[b].double()]),
                          see, dtype == BF16)
        for x in (got, plain):
            U.check(x[b][rest], *(y.view(T, Hkv, G, d)[rest] for y in (o, tol)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("of", ["draft_k", "draft_v"])
def test_a_draft_that_is_not_finite_reaches_those_that_see_it(dtype, of):
    """A tree of drafts, one of them NaN in one head: its own rows of that head and its
    children's are NaN, the others the same bits as without."""
    B, T, Hkv, G, d, n = 2, 6, 2, 4, 64, 200
    parents = [-1, 0, 0, 1, 1, 2]
    g = gen(3)
    s = api.make_shape(B, G * Hkv, Hkv, d, 16, T, dtype)
    kv, _, _ = cache(g, s, randn(g, B, n, Hkv, d).to(dtype), randn(g, B, n, Hkv, d).to(dtype))
    q = randn(g, B, T, Hkv * G, d).to(dtype)
    x = dict(draft_k=randn(g, B, T, Hkv, d).to(dtype), draft_v=randn(g, B, T, Hkv, d).to(dtype))
    outs = []
    for what in (0.0, math.nan):
        x[of][1, 1, 1] = what
        out, ws = torch.full_like(q, 7), api.alloc_kv4_workspace(s)
        api.sv_attend_kv4(s, q, kv, None, x["draft_k"], x["draft_v"], parents, out, ws)
        assert api.sv_read_status(ws) == 0
        outs.append(out.view(B, T, Hkv, G, d))
    hit = torch.zeros(B, T, Hkv, dtype=torch.bool, device="cuda")
    hit[1, [1, 3, 4], 1] = True
    assert outs[1][hit].isnan().all() and torch.equal(outs[1][~hit], outs[0][~hit])


# ------------------------------------------------------------------ sizes of queries
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [32, -32])
def test_queries_of_any_size(dtype, d, power):
    """Queries 2^power times their size over keys 2^-power times theirs (by the heads'
    exponents), so that the scores are ordinary ones; and a row that is nothing but 1e30 in a dim
    that no key has, all of whose scores are zero."""
    B, T, Hkv, G, n = 2, 4, 2, 4, 700
    g = gen(d)
    s = api.make_shape(B, G * Hkv, Hkv, d, 64, T, dtype)
    k, v = randn(g, B, n, Hkv, d), randn(g, B, n, Hkv, d)
    k[..., 0] = 0
    e = torch.full((Hkv,), -power, dtype=torch.int32, device="cuda")
    kv, hk, hv = cache(g, s, (k * 2.0 ** -power).to(dtype), v.to(dtype), e)
    q, dk, dv = randn(g, B, T, Hkv * G, d), randn(g, B, T, Hkv, d), randn(g, B, T, Hkv, d)
    dk[..., 0] = 0
    q, dk, dv = (q * 2.0 ** power).to(dtype), (dk * 2.0 ** -power).to(dtype), dv.to(dtype)
    q[1, 2, 3] = 0
    q[1, 2, 3, 0] = 1e30
    out = attend(s, q, kv, dk, dv)
    see = all_keys(T, Hkv, n)
    for b in range(B):
        U.check(out[b], *U.attend(q[b], torch.cat([hk[b], dk[b].double()]), torch.cat([hv[b], dv[b].double()]), see,
                                  dtype == BF16))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e30, 3e38])
def test_largest_queries_under_the_largest_exponent(dtype, size):
    """A row of one huge element in a dim that neither keys nor drafts have: its scores are
    zero, whatever the keys' exponent, and its output is the mean of the values."""
    n, d = 300, 128
    g = gen(8)
    s = api.make_shape(1, 4, 1, d, 16, 2, dtype)
    k, v = randn(g, 1, n, 1, d).to(dtype), randn(g, 1, n, 1, d).to(dtype)
    k[..., 5] = 0
    kv, hk, hv = cache(g, s, k, v, torch.full((1,), 32, dtype=torch.int32, device="cuda"))
    q, dk, dv = torch.zeros(1, 2, 4, d), randn(g, 1, 2, 1, d), randn(g, 1, 2, 1, d).to(dtype)
    dk[..., 5] = 0
    q[0, :, ::2, 5], q[0, :, 3, 5] = size, -size
    q, dk = q.to(dtype).cuda(), dk.to(dtype)
    out = attend(s, q, kv, dk, dv)[0]
    U.check(out, *U.attend(q[0], torch.cat([hk[0], dk[0].double()]), torch.cat([hv[0], dv[0].double()]),
                           all_keys(2, 1, n), dtype == BF16))


# ------------------------------------------------------------------ long contexts
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_part_of_a_long_context_counts(dtype):
    """Dim j of the values is 1.5 in the j-th of 128 runs of keys and 0 elsewhere, so that output
    j is the weight of that run, to within a thousandth or so of itself: a piece of 16 keys
    left out or counted twice is 14 thousandths of its run.

    The tolerance is U.attend's with the additions that a sum goes through in place of one a
    key. On the tensor cores a stream takes every second of its CTA's key tiles in 8 products
    of 16 keys, each cut off like 17 additions at most (2 u). On the CUDA cores a thread adds
    a key at a time (u). Both then add a part for each CTA, at most 640. Factors of moved
    references, two roundings a tile, are counted with them."""
    n, T, Hq, d, blk = 150_001, 4, 4, 128, 64
    g = gen(5)
    s = api.make_shape(1, Hq, 1, d, blk, T, dtype)
    k = randn(g, 1, n, 1, d).to(dtype)
    run = torch.arange(n, device="cuda") * 128 // n
    v = (1.5 * torch.nn.functional.one_hot(run, 128)).to(dtype)[None, :, None]
    kv, hk, hv = cache(g, s, k, v)
    assert torch.equal(hv, v.double())
    q = randn(g, 1, T, Hq, d).to(dtype)
    dk, dv = randn(g, 1, T, 1, d).to(dtype), torch.zeros(1, T, 1, d, dtype=dtype, device="cuda")
    out = attend(s, q, kv, dk, dv)[0]
    f16 = dtype == BF16
    tiles = -(-n // (128 if f16 else 64))
    share = tiles // 152 + 2  # (of a CTA, at least so many CTAs have one)
    additions = (2 * (8 * 17 + 2) * (share // 2 + 1) if f16 else 66 * share) + 2 * 640
    kk = torch.cat([hk[0], dk[0].double()])[:, 0]
    see = all_keys(T, 1, n)[:, 0]
    runs = torch.cat([run, run.new_full((T,), 128)])
    for h in range(Hq):
        qh = q[0, :, h].double()
        x = (qh @ kk.T / math.sqrt(d)).masked_fill(~see, -math.inf)
        p = torch.softmax(x, -1)
        o = torch.zeros(T, 129, dtype=torch.float64, device="cuda").index_add_(1, runs, 1.5 * p)[:, :128]
        big = (qh.abs() @ kk.abs().T / math.sqrt(d)).masked_fill(~see, 0).amax(-1, keepdim=True)
        w = 2 * ((d + 4) * (2 if f16 else 1) * U.U * big + 12 * U.U + additions * U.U) + (2.0 ** -11 if f16 else 0)
        tol = (w + U.half_step(dtype)) * o + (2.0 ** -32 * 1.5 * n / 128 if f16 else 0)
        assert (tol < 0.007 * o).all()  # half of what a piece is
        U.check(out[:, h], o, tol)
