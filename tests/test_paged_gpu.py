"""The paged-cache operators against plain 64-bit forms (tests/paged_util.py)."""
import random

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status_ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ tables
def tables_case(seed, B, blk, most, spare, pin=False):
    r = random.Random(seed)
    old = [r.choice([0, r.randint(0, most)]) for _ in range(B)]
    new = [r.choice([0, n, n + 1, n + r.randint(1, 9), r.randint(0, most)]) for n in old]
    pinned = [r.choice([0, 1, P.nb(n, blk)]) if pin and n <= m else 0 for n, m in zip(new, old)]
    nb_max = max(P.nb(max(old + new), blk), 1) + r.randint(0, 3)
    held = [P.nb(n, blk) for n in old]
    # enough pages even when pinned ones are not given back
    pages = sum(held) + sum(P.nb(n, blk) for n in new) + spare
    perm = list(range(pages))
    r.shuffle(perm)
    table, at = [], 0
    for h in held:
        table.append(perm[at:at + h] + [-7] * (nb_max - h))
        at += h
    return old, new, pinned, table, perm[at:] + [-9] * at, pages - at


def run_tables(blk, old, new, table, stack, count, n_max, pinned=None, in_place=False, positions=True):
    t = dict(old_len=i32(old), new_len=i32(new), block_table=i32(table), free_pages=i32(stack),
             free_count=i32([count]), cu_new=i32([-5] * (len(old) + 1)), slot_map=i32([-5] * n_max))
    t["free_count_out"] = t["free_count"] if in_place else i32([-5])
    t["positions"] = i32([-5] * n_max) if positions else None
    t["pinned"] = None if pinned is None else i32(pinned)
    ws = status_ws()
    api.sv_build_tables(blk, ws=ws, **t)
    flags = api.sv_read_status(ws)
    got = [t[n].tolist() for n in ("block_table", "free_pages", "free_count_out", "cu_new", "slot_map")]
    return got + [t["positions"].tolist() if positions else None, flags]


@pytest.mark.parametrize("B,blk,most,pad,pin,in_place", [
    (1, 16, 40, 0, False, False), (1, 1, 5, 3, False, True), (3, 64, 500, 0, True, False),
    (33, 7, 90, 11, True, True), (257, 16, 300, 0, False, True), (1000, 32, 130, 5, True, False),
    (4096, 16, 20, 1, True, True), (8, 64, 9000, 100, False, False)])
def test_tables(B, blk, most, pad, pin, in_place):
    for seed in range(3):
        old, new, pinned, table, stack, count = tables_case(seed, B, blk, most, 5, pin)
        want = P.tables(blk, old, new, pinned, table, stack, count)
        n_max = want[3][-1] + pad
        got = run_tables(blk, old, new, table, stack, count, n_max, pinned if pin else None, in_place)
        rest = [-1] * pad
        assert got[6] == 0
        assert got[2] == [want[2]] and got[3] == want[3]
        assert got[4] == want[4] + rest and got[5] == want[5] + rest
        assert got[0] == want[0]
        assert got[1] == want[1]


def test_tables_release_undoes_allocation():
    old, new, _, table, stack, count = tables_case(5, 40, 16, 200, 10)
    new = [n + 100 for n in old]
    table = [r + [-7] * 20 for r in table]
    stack += [0] * 400  # and enough pages for it
    have = count
    pages = len(stack)
    for p in range(400):
        stack[have] = pages - 400 + p
        have += 1
    a = run_tables(16, old, new, table, stack, have, sum(new) - sum(old))
    b = run_tables(16, new, old, a[0], a[1], a[2][0], 0, positions=False)
    assert a[6] == b[6] == 0
    assert b[2] == [have] and b[1][:have] == stack[:have]


def test_tables_out_of_pages():
    """Blocks get pages in order until none is left; the rest, and their slots, are -1."""
    got = run_tables(4, [0, 3, 0], [6, 9, 5], [[-7] * 4, [5, -7, -7, -7], [-7] * 4], [0, 1, 2, 3, 4, 9],
                     3, 20)
    table, stack, count, cu, slots, pos, flags = got
    assert flags == api.SV_FLAG_NO_PAGE and count == [0]
    assert table == [[2, 1, -7, -7], [5, 0, -1, -7], [-1, -1, -7, -7]]
    assert cu == [0, 6, 12, 17]
    assert slots == [8, 9, 10, 11, 4, 5, 23, 0, 1, 2, 3, -1, -1, -1, -1, -1, -1, -1, -1, -1]
    assert pos[:17] == [0, 1, 2, 3, 4, 5, 3, 4, 5, 6, 7, 8, 0, 1, 2, 3, 4] and pos[17:] == [-1] * 3


def test_tables_bad_values_are_flagged_and_clamped():
    full = [[0, 1], [2, 3]]
    # a length past the table's width, a negative one
    got = run_tables(4, [0, -3], [99, 2], [[-7, -7], [-7, -7]], [0, 1, 2, 3], 4, 16)
    assert got[6] == api.SV_FLAG_BAD_LENGTH and got[3] == [0, 8, 10] and got[0] == [[3, 2], [1, -7]]
    # a count past the stack's size
    got = run_tables(4, [0, 0], [1, 0], [[-7, -7], [-7, -7]], [3, 2, 1, 0], 99, 1)
    assert got[6] == api.SV_FLAG_BAD_LENGTH and got[0][0][0] == 0 and got[2] == [3]
    # more new tokens than slots
    got = run_tables(4, [0, 0], [3, 3], [[-7, -7], [-7, -7]], [3, 2, 1, 0], 4, 4)
    assert got[6] == api.SV_FLAG_BAD_LENGTH and got[3] == [0, 3, 6] and got[4] == [0, 1, 2, 4]
    # released and partly filled blocks whose page is outside the pool
    got = run_tables(4, [6, 0], [0, 0], [[1, 44], [-7, -7]], [0, 0, 0, 0], 0, 0)
    assert got[6] == api.SV_FLAG_BAD_PAGE and got[2] == [2] and got[1][:2] == [-1, 1]
    got = run_tables(4, [2, 0], [3, 0], [[77, -7], [-7, -7]], [0, 0, 0, 0], 1, 1)
    assert got[6] == api.SV_FLAG_BAD_PAGE and got[4] == [-1]
    # a stack entry outside the pool
    got = run_tables(4, [0, 0], [3, 0], [[-7, -7], [-7, -7]], [50, 0, 0, 0], 1, 3)
    assert got[6] == api.SV_FLAG_BAD_PAGE and got[4] == [-1] * 3 and got[0][0][0] == -1
    # more pages given back than the stack holds
    got = run_tables(4, [8, 8], [0, 0], full, [0, 1, 2, 3], 2, 0)
    assert got[6] == api.SV_FLAG_BAD_LENGTH and got[2] == [4] and got[1][:2] == [0, 1]


# ------------------------------------------------------------------ K/V rows
@pytest.mark.parametrize("dtype,Hkv,d,blk,n,extra", [
    (BF16, 8, 128, 64, 1000, 4096), (BF16, 1, 8, 16, 1, 0), (F32, 2, 64, 16, 37, 0),
    (F32, 3, 24, 5, 130, 8), (BF16, 16, 256, 32, 77, 64), (BF16, 5, 40, 1, 9, 16)])
def test_write_kv(dtype, Hkv, d, blk, n, extra):
    g = gen(n)
    pages = P.nb(n, blk) + 3
    fused = torch.randn(n, 2 * Hkv * d + extra, generator=g).to(dtype).cuda()
    k = fused[:, extra:extra + Hkv * d].unflatten(1, (Hkv, d))
    v = fused[:, extra + Hkv * d:].unflatten(1, (Hkv, d))
    slots = torch.randperm(pages * blk, generator=g)[:n].to(torch.int32)
    slots[torch.rand(n, generator=g) < 0.1] = -1
    kp, vp = (torch.randn(pages, Hkv, blk, d, generator=g).to(dtype).cuda() for _ in range(2))
    want_k, want_v = kp.clone(), vp.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // blk, :, s % blk], want_v[s // blk, :, s % blk] = k[i], v[i]
    ws = status_ws()
    api.sv_write_kv(api.make_shape(1, Hkv, Hkv, d, blk, 1, dtype), k, v, slots.cuda(), kp, vp, ws)
    assert api.sv_read_status(ws) == 0
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


def test_write_kv_skips_bad_slots():
    kp, vp = torch.zeros(2, 2, 4, 8, device="cuda"), torch.zeros(2, 2, 4, 8, device="cuda")
    k = torch.ones(4, 2, 8, device="cuda")
    ws = status_ws()
    api.sv_write_kv(api.make_shape(1, 2, 2, 8, 4, 1, F32), k, k, i32([8, 7, -2, 1 << 30]), kp, vp, ws)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_PAGE
    assert float(kp.sum()) == float(vp.sum()) == 16.0 and float(kp[1, :, 3].sum()) == 16.0
    api.sv_write_kv(api.make_shape(1, 2, 2, 8, 4, 1, F32), k, k, i32([9, 9, 9, 9]), kp, vp)  # no workspace


# ------------------------------------------------------------------ prompt
def prompt_case(seed, dtype, Hq, Hkv, d, blk, ctx, new, pad=0, hole=float("nan"), extra=0):
    g = gen(seed)
    k, v, table = P.paged_pools(g, ctx, Hkv, blk, d, dtype, hole=hole)
    n = sum(new)
    q = torch.randn(n + pad, Hq * d + extra, generator=g).to(dtype).cuda()[:, :Hq * d]
    q = q.unflatten(1, (Hq, d))
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    return dict(shape=api.make_shape(len(ctx), Hq, Hkv, d, blk, 1, dtype), q=q, k_pool=k, v_pool=v,
                block_table=table, seq_ctx=i32(ctx), cu_q=i32(starts),
                out=torch.full((n + pad, Hq, d), 7.0, dtype=dtype, device="cuda"))


def prompt_want(c, ctx, new):
    blk = c["shape"].blk
    outs, tols = [], []
    for b, (x, n) in enumerate(zip(ctx, new)):
        at = int(c["cu_q"][b])
        q = c["q"][at:at + n]
        k, v = (P.gather(c[p], c["block_table"][b], x, blk) for p in ("k_pool", "v_pool"))
        o, t = P.attend(q, k, v, P.causal(n, x, "cuda"))
        outs.append(o)
        tols.append(t)
    return torch.cat(outs), torch.cat(tols)


def run_prompt(c, ws=None, **kw):
    ws = api.alloc_prompt_workspace(c["shape"], c["q"].shape[0]) if ws is None else ws
    api.sv_prompt_attend(ws=ws, **c, **kw)
    return api.sv_read_status(ws)


HEADS = [  # dtype, Hq, Hkv, d, blk
    (BF16, 8, 2, 128, 64), (BF16, 4, 4, 64, 16), (BF16, 7, 1, 128, 32), (BF16, 6, 2, 96, 64),
    (BF16, 8, 1, 128, 128), (BF16, 2, 1, 40, 8), (BF16, 4, 2, 256, 64), (BF16, 3, 1, 128, 48),
    (BF16, 40, 1, 64, 256), (BF16, 129, 1, 64, 16), (F32, 4, 2, 64, 16), (F32, 3, 3, 128, 64),
    (F32, 5, 1, 200, 5), (F32, 70, 1, 16, 16), (BF16, 2, 2, 8, 32), (BF16, 5, 1, 128, 512),
    (BF16, 128, 1, 64, 16), (F32, 2, 1, 256, 7)]
LENS = [  # ctx, new
    ([1], [1]), ([2, 1, 3], [2, 1, 3]), ([63, 64, 65, 127, 128, 129], [63, 64, 65, 127, 128, 129]),
    ([300, 1000, 5], [300, 7, 1]), ([700], [700]), ([1500, 1, 2049], [1, 1, 1]),
    ([900, 900, 900], [0, 33, 0]), ([2600], [130])]


@pytest.mark.parametrize("lens", range(len(LENS)))
@pytest.mark.parametrize("heads", range(len(HEADS)))
def test_prompt(heads, lens):
    ctx, new = LENS[lens]
    c = prompt_case(heads * 100 + lens, *HEADS[heads], ctx, new, pad=2, extra=16 * (lens % 2))
    assert run_prompt(c) == 0
    n = sum(new)
    P.check(c["out"][:n], *prompt_want(c, ctx, new))
    assert (c["out"][n:] == 7.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_prompt_split_runs(dtype, d):
    """Few rows over long contexts: runs of keys on many CTAs, merged."""
    for ctx, new in (([20000], [1]), ([9000, 30, 12000, 1], [3, 30, 1, 1]), ([16384], [100])):
        c = prompt_case(3, dtype, 8, 2, d, 64, ctx, new)
        ws = api.alloc_prompt_workspace(c["shape"], sum(new))
        assert run_prompt(c, ws) == 0
        first = c["out"].clone()
        P.check(first, *prompt_want(c, ctx, new))
        assert run_prompt(c, ws) == 0  # the counts are back at zero ...
        assert torch.equal(first, c["out"])  # ... and the result does not depend on the order


def test_prompt_very_long_context():
    ctx, new = [200001, 7], [2, 7]
    c = prompt_case(4, BF16, 4, 1, 64, 64, ctx, new)
    assert run_prompt(c) == 0
    P.check(c["out"], *prompt_want(c, ctx, new))


@pytest.mark.parametrize("dtype,pages", [(BF16, 36000), (F32, 18000)])
def test_pools_past_4_gib(dtype, pages):
    """Pages whose bytes lie past 2^32 of the pool (and elements past 2^31 in bf16):
    rows written, attended as a prompt and as a shared prefix."""
    Hq, Hkv, d, blk, n, T = 16, 8, 128, 64, 300, 2
    g = gen(6)
    kp, vp = (torch.empty(pages, Hkv, blk, d, dtype=dtype, device="cuda") for _ in range(2))
    table = i32([[pages - 1, pages - 3, 0, pages - 2, 7]])
    q, k, v = (torch.randn(n, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    p = torch.arange(n, device="cuda")
    slots = (table[0].long()[p // blk] * blk + p % blk).to(torch.int32)
    shape = api.make_shape(1, Hq, Hkv, d, blk, T, dtype)
    ws = api.alloc_prompt_workspace(shape, n)
    out = torch.empty_like(q)
    api.sv_write_kv(shape, k, v, slots, kp, vp, ws)
    api.sv_prompt_attend(shape, q, kp, vp, table, i32([n]), i32([0, n]), out, ws)
    assert api.sv_read_status(ws) == 0
    P.check(out, *P.attend(q, k, v, P.causal(n, n, "cuda")))
    kv = api.make_kv(kp, vp, table, n)
    dq, dk, dv, dout = q[None, :T].contiguous(), k[None, :T].contiguous(), v[None, :T].contiguous(), out[None, :T].clone()
    wp = api.alloc_prefix_workspace(shape)
    api.sv_prefix_attend(shape, dq, kv, 3, dk, dv, None, dout, wp)
    assert api.sv_read_status(wp) == 0
    see = torch.cat([torch.ones(T, n, dtype=torch.bool, device="cuda"), P.draft_mask(None, T, "cuda")], 1)
    P.check(dout[0], *P.attend(dq[0], torch.cat([k, dk[0]]), torch.cat([v, dv[0]]), see))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_rows_without_keys(dtype):
    """More rows than context: the first ones see nothing and are zero."""
    c = prompt_case(9, dtype, 4, 2, 64, 16, [20, 7, 40], [20, 7, 40])
    c["seq_ctx"] = i32([5, 0, 40])
    assert run_prompt(c) == api.SV_FLAG_BAD_LENGTH
    assert (c["out"][:15] == 0).all() and (c["out"][20:27] == 0).all()
    k, v = (P.gather(c[p], c["block_table"][0], 5, 16) for p in ("k_pool", "v_pool"))
    P.check(c["out"][15:20], *P.attend(c["q"][15:20], k, v, P.causal(5, 5, "cuda")))
    k, v = (P.gather(c[p], c["block_table"][2], 40, 16) for p in ("k_pool", "v_pool"))
    P.check(c["out"][27:], *P.attend(c["q"][27:], k, v, P.causal(40, 40, "cuda")))


@pytest.mark.parametrize("dtype,Hq,d", [(BF16, 4, 128), (BF16, 32, 64), (F32, 4, 64)])
def test_prompt_infinities_behind_the_mask(dtype, Hq, d):
    """Rows before a token with non-finite V (or K) do not feel it; rows after
    it give what the formula gives."""
    ctx = [200, 150]
    c = prompt_case(11, dtype, Hq, 2, d, 16, ctx, [200, 30])
    blk, t = 16, c["block_table"]
    want, tol = prompt_want(c, ctx, [200, 30])
    j = 130  # token 130 of sequence 0: V of one KV head
    for bad, h, col in ((float("inf"), 0, 3), (float("nan"), 0, 9), (-float("inf"), 0, 17)):
        c["v_pool"][t[0, j // blk].long(), h, j % blk, col] = bad
    c["k_pool"][t[1, 145 // blk].long(), 1, 145 % blk] = float("nan")  # sequence 1 sees it from row 25 on
    assert run_prompt(c) == 0
    out, G = c["out"], Hq // 2
    touched = torch.zeros_like(want, dtype=torch.bool)
    touched[j:200, :G, 3] = touched[j:200, :G, 9] = touched[j:200, :G, 17] = True
    touched[200 + 25:, G:] = True
    P.check(out[~touched], want[~touched], tol[~touched])
    assert (out[j:200, :G, 3] == float("inf")).all() and out[j:200, :G, 9].isnan().all()
    assert (out[j:200, :G, 17] == -float("inf")).all() and out[225:, G:].isnan().all()


def test_prompt_large_scores():
    """Scores of some hundreds: the running maximum moves far, in both directions."""
    for dtype in (BF16, F32):
        c = prompt_case(13, dtype, 8, 2, 64, 16, [700, 300], [700, 1])
        c["k_pool"].nan_to_num_()
        c["k_pool"].mul_(torch.linspace(0.1, 12, c["k_pool"].shape[0], device="cuda")[:, None, None, None])
        assert run_prompt(c) == 0
        P.check(c["out"], *prompt_want(c, [700, 300], [700, 1]))


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64), (16, 1, 128)])
def test_prompt_growing_scores(Hq, Hkv, d):
    """Keys that grow along the context: the running maximum of most rows moves
    by several powers of two in most key tiles, so that every tile rescales."""
    ctx, new = [4000, 2500], [1500, 2500]
    c = prompt_case(14, BF16, Hq, Hkv, d, 64, ctx, new, hole=0.0)
    for b, n in enumerate(ctx):
        i = torch.arange(n, device="cuda")
        page = c["block_table"][b].long()[i // 64]
        c["k_pool"][page, :, i % 64] *= (1 + i / 60)[:, None, None]
    want, tol = prompt_want(c, ctx, new)
    ws = api.alloc_prompt_workspace(c["shape"], sum(new))
    for _ in range(5):
        c["out"].fill_(7.0)
        assert run_prompt(c, ws) == 0
        P.check(c["out"], want, tol)


@pytest.mark.parametrize("jump", [30.0, 300.0])
def test_prompt_jumping_scores(jump):
    """Scores that jump by more than 2^64 inside a key tile, in the first or the
    second half of its keys, in both, for some rows only, up and down."""
    ctx = [1500]
    for Hq, Hkv, d in ((4, 1, 128), (2, 2, 64)):
        c = prompt_case(16, BF16, Hq, Hkv, d, 64, ctx, ctx, hole=0.0)
        t = c["block_table"][0].long()
        u = torch.zeros(d, device="cuda")
        u[3] = 1.0
        c["q"][:, :, 3] = 8.0 * (torch.arange(1500, device="cuda")[:, None] % 3 != 1)  # not every row
        for i, size in ((200, 1), (340, 2), (400, 2.5), (450, 2.5), (700, 4), (901, 3), (1280, 5), (1344, 5)):
            c["k_pool"][t[i // 64], :, i % 64] = (jump * size * u).to(BF16)
        c["k_pool"][t[300 // 64], :, 300 % 64] = (-jump * 9 * u).to(BF16)
        want, tol = prompt_want(c, ctx, ctx)
        for _ in range(3):
            c["out"].fill_(7.0)
            assert run_prompt(c) == 0
            P.check(c["out"], want, tol)


def test_prompt_bad_pages_and_offsets():
    c = prompt_case(15, BF16, 4, 2, 128, 64, [200, 100], [200, 100])
    c["block_table"][0, 1] = 99
    c["block_table"][1, 1] = -3
    assert run_prompt(c) == api.SV_FLAG_BAD_PAGE
    assert c["out"].isfinite().all()
    c = prompt_case(15, F32, 4, 2, 64, 16, [20, 10], [20, 10])
    c["cu_q"] = i32([0, 20, 99])  # past the rows: clamped to them
    assert run_prompt(c) == api.SV_FLAG_BAD_LENGTH
    P.check(c["out"], *prompt_want(c, [20, 10], [20, 10]))
    c["seq_ctx"] = i32([20, 1 << 30])  # past the table: clamped to its width, its last pages bad
    assert run_prompt(c) & api.SV_FLAG_BAD_LENGTH


def test_prompt_many_sequences():
    ctx = [(37 * i) % 90 + 1 for i in range(1024)]
    new = [min(x, (i % 5)) for i, x in enumerate(ctx)]
    c = prompt_case(17, BF16, 4, 2, 64, 16, ctx, new)
    assert run_prompt(c) == 0
    P.check(c["out"], *prompt_want(c, ctx, new))


@pytest.mark.parametrize("Hq,Hkv,d,blk", [(32, 8, 128, 64), (8, 8, 64, 16)])
def test_prompt_repeated_decoding_steps(Hq, Hkv, d, blk):
    """Some thousand steps of many short items: no wait of any role ever runs out,
    and every step gives the same bits."""
    ctx = [(i * 997) % 1500 + 1 for i in range(40)] + [9000, 4097]
    c = prompt_case(18, BF16, Hq, Hkv, d, blk, ctx, [1] * 42)
    ws = api.alloc_prompt_workspace(c["shape"], 42)
    assert run_prompt(c, ws) == 0
    P.check(c["out"], *prompt_want(c, ctx, [1] * 42))
    first = c["out"].clone()
    for _ in range(4):
        for _ in range(1000):
            api.sv_prompt_attend(ws=ws, **c)
        assert api.sv_read_status(ws) == 0
        assert torch.equal(c["out"], first)


def test_prompt_other_stream_and_graph():
    """On a side stream, and captured: a replay follows the lengths in device memory."""
    ctx, new = [400, 300], [100, 60]
    c = prompt_case(19, BF16, 8, 2, 128, 64, ctx, new)
    want = prompt_want(c, ctx, new)
    ws = api.alloc_prompt_workspace(c["shape"], 160)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.sv_prompt_attend(ws=ws, stream=s, **c)
    s.synchronize()
    P.check(c["out"], *want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        api.sv_prompt_attend(ws=ws, **c)
    for ctx, new in (([400, 300], [100, 60]), ([10, 290], [10, 1]), ([399, 3], [0, 3])):
        c["seq_ctx"].copy_(i32(ctx))
        c["cu_q"].copy_(i32([0, new[0], sum(new)]))
        c["out"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert api.sv_read_status(ws) == 0
        P.check(c["out"][:sum(new)], *prompt_want(c, ctx, new))
        assert (c["out"][sum(new):] == 7.0).all()


# ------------------------------------------------------------------ prefix
def prefix_case(seed, dtype, Hq, Hkv, d, blk, T, shared, own, parents=None, uniform=False):
    g = gen(seed)
    B = len(own)
    lens = [shared * blk] + list(own)
    k, v, rows = P.paged_pools(g, lens, Hkv, blk, d, dtype)
    width = shared + rows.shape[1]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[0, :shared] = rows[0, :shared]  # the other rows' shared entries are not read
    for b in range(B):
        n = P.nb(own[b], blk)
        table[b, shared:shared + n] = rows[b + 1, :n]
    ctx = [shared * blk + n for n in own]
    kv = api.make_kv(k, v, table, ctx[0], None if uniform else ctx)
    kv.keep = k, v, table  # the descriptor holds addresses only
    q, dk, dv = (torch.randn(B, T, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    c = dict(shape=api.make_shape(B, Hq, Hkv, d, blk, T, dtype), q=q, kv=kv, n_shared=shared, draft_k=dk,
             draft_v=dv, parents=parents, out=torch.full_like(q, 7.0))
    mask = P.draft_mask(parents, T, "cuda")
    outs, tols = [], []
    for b in range(B):
        full = torch.cat([rows[0, :shared], rows[b + 1]])
        kk, vv = (torch.cat([P.gather(p, full, ctx[b], blk), x[b]]) for p, x in ((k, dk), (v, dv)))
        see = torch.cat([torch.ones(T, ctx[b], dtype=torch.bool, device="cuda"), mask], 1)
        o, t = P.attend(q[b], kk, vv, see)
        outs.append(o)
        tols.append(t)
    return c, torch.stack(outs), torch.stack(tols)


TREE = [-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6, 7, 8, 9, 10, 3]
PREFIX = [  # dtype, Hq, Hkv, d, blk, T, shared, own, parents
    (BF16, 8, 2, 128, 64, 8, 20, [100, 0, 64, 700, 1], None),
    (BF16, 8, 1, 128, 64, 16, 33, [65, 130], TREE),
    (BF16, 4, 2, 64, 16, 1, 70, [0, 1, 15, 16, 17, 300, 40, 2, 5], None),
    (BF16, 32, 8, 128, 64, 1, 9, [3 * i for i in range(40)], None),
    (BF16, 6, 2, 96, 32, 5, 1, [10, 2000], [-1, 0, 0, 1, 0]),
    (BF16, 12, 2, 128, 64, 64, 3, [77, 0], None),
    (BF16, 4, 2, 256, 64, 4, 5, [9, 100], None),
    (BF16, 4, 1, 128, 64, 3, 0, [500, 0, 64], None),
    (BF16, 200, 1, 64, 16, 3, 4, [7, 40], None),
    (F32, 4, 2, 64, 16, 4, 63, [40, 0, 333, 16, 1], [-1, 0, 0, 2]),
    (F32, 3, 3, 128, 64, 7, 2, [1, 65, 640], None),
    (F32, 4, 2, 200, 5, 2, 9, [11], None)]


@pytest.mark.parametrize("case", range(len(PREFIX)))
def test_prefix(case):
    *args, parents = PREFIX[case]
    c, want, tol = prefix_case(case, *args, parents=parents)
    ws = api.alloc_prefix_workspace(c["shape"])
    for _ in range(2):
        c["out"].fill_(7.0)
        api.sv_prefix_attend(ws=ws, **c)
        assert api.sv_read_status(ws) == 0
        P.check(c["out"], want, tol)


def test_prefix_uniform_context_of_a_large_batch():
    c, want, tol = prefix_case(31, BF16, 4, 2, 64, 16, 2, 12, [21] * 100, uniform=True)
    ws = api.alloc_prefix_workspace(c["shape"])
    api.sv_prefix_attend(ws=ws, **c)
    assert api.sv_read_status(ws) == 0
    P.check(c["out"], want, tol)


def test_prefix_infinities_behind_the_mask():
    """A draft's non-finite V reaches the drafts that see it and no other."""
    parents = [-1, 0, 0, 1, 2]
    for dtype in (BF16, F32):
        c, want, tol = prefix_case(35, dtype, 4, 2, 64, 16, 5, 4, [20, 3], parents=parents)
        c["draft_v"][0, 1, 0, 5] = float("inf")
        ws = api.alloc_prefix_workspace(c["shape"])
        api.sv_prefix_attend(ws=ws, **c)
        assert api.sv_read_status(ws) == 0
        sees = P.draft_mask(parents, 5, "cuda")[:, 1]
        touched = torch.zeros_like(want, dtype=torch.bool)
        touched[0, :, :2, 5] = sees[:, None]
        P.check(c["out"][~touched], want[~touched], tol[~touched])
        assert (c["out"][touched] == float("inf")).all()


def test_prefix_captured():
    """A captured call replays on new drafts, on another stream, after other calls."""
    c, want, tol = prefix_case(37, BF16, 8, 2, 128, 64, 4, 9, [100, 30, 0])
    ws = api.alloc_prefix_workspace(c["shape"])
    api.sv_prefix_attend(ws=ws, **c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sv_prefix_attend(ws=ws, **c)
    c["q"].neg_()
    other = torch.empty_like(c["out"])
    api.sv_prefix_attend(ws=ws, **{**c, "out": other})
    c["q"].neg_()
    c["out"].fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert api.sv_read_status(ws) == 0
    P.check(c["out"], want, tol)
    assert not torch.equal(other, c["out"])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,d,blk", [(BF16, 128, 64), (F32, 64, 16)])
def test_serving_loop(dtype, d, blk):
    """A prompt shared by three requests, brought in by two chunks; each
    request continues with its own tokens; drafts are verified; one request
    ends and its pages serve the next. One workspace, one captured step."""
    g = gen(41)
    Hq, Hkv, T, pages, nb_max = 8, 2, 4, 60, 24
    shape1 = api.make_shape(3, Hq, Hkv, d, blk, T, dtype)
    kp, vp = (torch.full((pages, Hkv, blk, d), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.full((3, nb_max), -1, dtype=torch.int32, device="cuda")
    stack, count = i32(torch.randperm(pages, generator=g).tolist()), i32([pages])
    ws = api.alloc_prompt_workspace(shape1, 400)
    wp = api.alloc_prefix_workspace(shape1)
    n_max = 5 * blk + 3
    q, k, v = (torch.randn(n_max, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    old, new, pinned = i32([0] * 3), i32([0] * 3), i32([0] * 3)
    cu, slots, pos = i32([0] * 4), i32([0] * n_max), i32([0] * n_max)
    out = torch.zeros(n_max, Hq, d, dtype=dtype, device="cuda")
    history = [[], [], []]  # the (k, v) rows of every request so far

    def step():
        api.sv_build_tables(blk, old, new, table, stack, count, count, cu, slots, pos, pinned, ws)
        api.sv_write_kv(shape1, k, v, slots, kp, vp, ws)
        api.sv_prompt_attend(shape1, q, kp, vp, table, new, cu, out, ws)

    def advance(run, lens):
        """All requests to `lens`, with fresh rows; checks every row."""
        before = old.tolist()
        new.copy_(i32(lens))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(dtype))
        run()
        torch.cuda.synchronize()
        assert api.sv_read_status(ws) == 0
        at = 0
        for b, (x, y) in enumerate(zip(before, lens)):
            n = max(0, y - x)
            history[b] = history[b][:y] + [(k[i].clone(), v[i].clone()) for i in range(at, at + n)]
            if n:
                kk, vv = (torch.stack([r[e] for r in history[b]]) for e in (0, 1))
                P.check(out[at:at + n], *P.attend(q[at:at + n], kk, vv, P.causal(n, y, "cuda")))
                assert pos[at:at + n].tolist() == list(range(x, y))
            at += n
        assert slots[at:].tolist() == [-1] * (n_max - at)
        old.copy_(new)

    # the common prompt through request 0, in two chunks (4 full blocks)
    advance(step, [3 * blk - 5, 0, 0])
    advance(step, [4 * blk, 0, 0])
    # requests 1 and 2 start from its blocks, which they do not own
    table[1:, :4] = table[0, :4]
    old.copy_(i32([4 * blk] * 3))
    pinned.copy_(i32([0, 4, 4]))
    history[1], history[2] = list(history[0]), list(history[0])
    # from here on captured
    graph = torch.cuda.CUDAGraph()
    free_before = int(count)
    with torch.cuda.graph(graph):
        step()
    assert int(count) == free_before  # a capture runs nothing
    advance(graph.replay, [4 * blk + 7, 4 * blk + 1, 5 * blk])
    advance(graph.replay, [4 * blk + 8, 4 * blk + 2, 5 * blk + 1])
    # verification of T drafts of all three, the shared blocks read once
    ctx = old.tolist()
    kv = api.make_kv(kp, vp, table, 0, ctx)
    dq, dk, dv = (torch.randn(3, T, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    dout = torch.empty_like(dq)
    api.sv_prefix_attend(shape1, dq, kv, 4, dk, dv, None, dout, wp)
    assert api.sv_read_status(wp) == 0
    plain = torch.empty_like(dq)
    w0 = api.alloc_workspace(shape1, nb_max, nb_max)
    api.sv_sparse_attend(shape1, dq, kv, None, 0, 0, dk, dv, None, plain, w0)
    mask = P.draft_mask(None, T, "cuda")
    for b in range(3):
        kk, vv = (torch.cat([torch.stack([r[e] for r in history[b]]), x[b]]) for e, x in ((0, dk), (1, dv)))
        see = torch.cat([torch.ones(T, ctx[b], dtype=torch.bool, device="cuda"), mask], 1)
        want, tol = P.attend(dq[b], kk, vv, see)
        P.check(dout[b], want, tol)
        assert (plain[b].double() - want).abs().max() <= (1e-2 if dtype == BF16 else 1e-4)
    # request 1 ends: its own pages are free again, the shared ones are not
    free = int(count)
    advance(graph.replay, [4 * blk + 9, 0, 5 * blk + 2])
    assert int(count) == free + 1
    # and it starts anew with a prompt of its own, in the pages it gave back
    pinned.copy_(i32([0, 0, 4]))
    advance(graph.replay, [4 * blk + 9, blk + 3, 5 * blk + 2])
    assert int(count) == free - 1
