"""The paged-cache operators where calls of the documentation meet edges: plans
of very many sequences, rows that are not part of a tile, empty caches, pools
that ran out, large batches."""
import random

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib
from tests import paged_util as P
from tests import test_paged_gpu as G

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    build_lib.build()
    api.lib()
    torch.cuda.set_device(0)


def same(got, first, when):
    """Equal bit for bit (said without printing the tensors)."""
    n = int((got != first).sum())
    assert n == 0, f"{n} of {first.numel()} elements differ {when}"


# ------------------------------------------------------------------ plans
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_queries_behind_a_large_plan(Hq, Hkv, d):
    """1024 one-token sequences: the plan's scratch is at its largest, and the first
    query tile is copied to the same place right behind it."""
    ctx = [(29 * i) % 70 + 1 for i in range(1024)]
    c = G.prompt_case(51, BF16, Hq, Hkv, d, 16, ctx, [1] * 1024)
    ws = api.alloc_prompt_workspace(c["shape"], 1024)
    want = G.prompt_want(c, ctx, [1] * 1024)
    assert G.run_prompt(c, ws) == 0
    P.check(c["out"], *want)
    first = c["out"].clone()
    for _ in range(200):
        c["out"].fill_(7.0)
        api.sv_prompt_attend(ws=ws, **c)
        same(c["out"], first, "on repetition")
    assert api.sv_read_status(ws) == 0


# ------------------------------------------------------------------ rows outside an item
HEADS = [(3, 1, 128), (7, 1, 64), (12, 2, 128), (8, 2, 128), (4, 4, 64)]  # Hq, Hkv, d


def growing(c, ctx, blk):
    """Keys that grow along the context, so that the running maximum keeps moving."""
    for b, n in enumerate(ctx):
        i = torch.arange(n, device="cuda")
        c["k_pool"][c["block_table"][b].long()[i // blk], :, i % blk] *= (1 + i / 300)[:, None, None]


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_prompt_padding_rows_change_no_bit(Hq, Hkv, d):
    """A tile's rows that belong to no sequence, or to the next one, may hold anything."""
    ctx, new = [1500, 700], [1500, 37]
    c = G.prompt_case(61, BF16, Hq, Hkv, d, 64, ctx, new, pad=200)
    growing(c, ctx, 64)
    n = sum(new)
    ws = api.alloc_prompt_workspace(c["shape"], n + 200)
    assert G.run_prompt(c, ws) == 0
    first = c["out"].clone()
    P.check(first[:n], *G.prompt_want(c, ctx, new))
    for size in (0.0, 1e3, float("nan"), float("inf"), 1e30):
        c["q"][n:] = torch.randn_like(c["q"][n:]) * size
        assert G.run_prompt(c, ws) == 0
        same(c["out"][:n], first[:n], f"with padding rows of size {size}")
        assert (c["out"][n:] == 7.0).all()
    for size in (1e3, float("nan")):  # the second sequence's queries and the first one's rows
        c["q"][1500:n] = torch.randn_like(c["q"][1500:n]) * size
        assert G.run_prompt(c, ws) == 0
        same(c["out"][:1500], first[:1500], f"before a sequence with rows of size {size}")


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_attention_after_other_calls_changes_no_bit(Hq, Hkv, d):
    """What an earlier call left in shared memory does not matter: not to a prompt, not to
    drafts over a shared prefix."""
    ctx = [1100, 900]
    c = G.prompt_case(63, BF16, Hq, Hkv, d, 64, ctx, ctx)
    growing(c, ctx, 64)
    p, want, tol = G.prefix_case(65, BF16, Hq, Hkv, d, 64, 5, 17, [500, 0, 130])
    ws, wp = api.alloc_prompt_workspace(c["shape"], 2000), api.alloc_prefix_workspace(p["shape"])
    loud = G.prompt_case(67, BF16, 16, 4, 128, 64, [3000], [3000])
    wl = api.alloc_prompt_workspace(loud["shape"], 3000)
    first = None
    for size in (1.0, 0.0, 1e3, 1e30, float("nan")):
        loud["q"].copy_(torch.randn_like(loud["q"]) * size)
        api.sv_prompt_attend(ws=wl, **loud)
        assert G.run_prompt(c, ws) == 0
        api.sv_prompt_attend(ws=wl, **loud)
        api.sv_prefix_attend(ws=wp, **p)
        assert api.sv_read_status(wp) == 0
        got = [c["out"].clone(), p["out"].clone()]
        if first is None:
            first = got
            P.check(got[0], *G.prompt_want(c, ctx, ctx))
            P.check(got[1], want, tol)
        for x, y in zip(got, first):
            same(x, y, f"after a call with rows of size {size}")


# ------------------------------------------------------------------ pools that run out
def test_tables_release_undoes_an_allocation_that_ran_out():
    """8 blocks wanted, 6 pages there: giving the blocks back gives back these 6 pages."""
    got = G.run_tables(4, [0, 0], [12, 20], [[-7] * 5, [-7] * 5], [0, 1, 2, 3, 4, 5], 6, 32)
    assert got[6] == api.SV_FLAG_NO_PAGE and got[2] == [0]
    assert got[0] == [[5, 4, 3, -7, -7], [2, 1, 0, -1, -1]]
    back = G.run_tables(4, [12, 20], [0, 0], got[0], got[1], 0, 0)
    assert back[6] == 0 and back[2] == [6] and back[1] == [0, 1, 2, 3, 4, 5]


def model(blk, old, new, pinned, table, stack, count):
    """sv_build_tables on lists, blocks without a page (-1) and an empty stack included."""
    table, stack = [list(r) for r in table], list(stack)
    for b in reversed(range(len(old))):
        for j in reversed(range(max(P.nb(new[b], blk), pinned[b]), P.nb(old[b], blk))):
            if table[b][j] != -1:
                stack[count] = table[b][j]
                count += 1
    cu, slots, pos, short, held = [0], [], [], False, False
    for b in range(len(old)):
        for j in range(P.nb(old[b], blk), P.nb(new[b], blk)):
            count, table[b][j] = (count - 1, stack[count - 1]) if count else (0, -1)
            short |= table[b][j] < 0
        for p in range(old[b], new[b]):
            page = table[b][p // blk]
            held |= page < 0 and p // blk < P.nb(old[b], blk)
            slots.append(page * blk + p % blk if page >= 0 else -1)
            pos.append(p)
        cu.append(len(slots))
    flags = (api.SV_FLAG_NO_PAGE if short else 0) | (api.SV_FLAG_BAD_PAGE if held else 0)
    return table, stack, count, cu, slots, pos, flags


@pytest.mark.parametrize("B,blk,most,n_max", [
    (5, 4, 30, 200), (300, 8, 60, 4096), (300, 8, 60, 20000), (90, 16, 900, 70000), (4000, 3, 20, 90000)])
@pytest.mark.parametrize("share", [0.3, 0.8])
def test_tables_steps_around_an_empty_pool(B, blk, most, n_max, share):
    """Requests come, grow and end while the pool keeps running out: no page is lost or
    held twice, on one CTA, eight and sixteen."""
    r = random.Random(B + int(10 * share))
    nb_max = P.nb(most, blk) + 1
    pages = max(3, int(share * B * nb_max / 2))
    table, stack, count = [[-1] * nb_max for _ in range(B)], list(range(pages)), pages
    r.shuffle(stack)
    old = [0] * B
    for _ in range(6):
        new = [r.choice([0, n, min(n + 1, most), r.randint(0, most), r.randint(0, most)]) for n in old]
        want = model(blk, old, new, [0] * B, table, stack, count)
        got = G.run_tables(blk, old, new, table, stack, count, n_max, in_place=True)
        rest = [-1] * (n_max - len(want[4]))
        assert len(want[4]) <= n_max and got[6] == want[6]
        assert got[2] == [want[2]] and got[3] == want[3]
        assert got[0] == want[0]
        assert got[1][:want[2]] == want[1][:want[2]]
        assert got[4] == want[4] + rest and got[5] == want[5] + rest
        table, stack, count, old = got[0], got[1], got[2][0], new
        held = [p for row, n in zip(table, old) for p in row[:P.nb(n, blk)] if p >= 0]
        assert sorted(held + stack[:count]) == list(range(pages))


# ------------------------------------------------------------------ empty caches
@pytest.mark.parametrize("dtype,d,T", [(BF16, 128, 4), (BF16, 64, 1), (BF16, 256, 3), (F32, 64, 4), (F32, 200, 1)])
@pytest.mark.parametrize("pool", ["none", "no pages", "pages"])
def test_prefix_of_an_empty_cache(dtype, d, T, pool):
    """No sequence has a token: the drafts see the drafts, with or without a pool, as in
    sv_sparse_attend over every block."""
    B, Hq, Hkv, blk = 3, 4, 2, 16
    g = G.gen(71)
    q, dk, dv = (torch.randn(B, T, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    shape = api.make_shape(B, Hq, Hkv, d, blk, T, dtype)
    pages = torch.full((2 if pool == "pages" else 0, Hkv, blk, d), float("nan"), dtype=dtype, device="cuda")
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    kv = api.KV(None, None, None, 0, 0, 0) if pool == "none" else api.make_kv(pages, pages, table, 0)
    out, plain = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    ws, w0 = api.alloc_prefix_workspace(shape), api.alloc_workspace(shape, 1, 1)
    api.sv_prefix_attend(shape, q, kv, 0, dk, dv, None, out, ws)
    api.sv_sparse_attend(shape, q, kv, None, 0, 0, dk, dv, None, plain, w0)
    assert api.sv_read_status(ws) == api.sv_read_status(w0) == 0
    for b in range(B):
        want, tol = P.attend(q[b], dk[b], dv[b], P.draft_mask(None, T, "cuda"))
        P.check(out[b], want, tol)
        P.check(plain[b], want, tol)


def test_prefix_refuses_a_cache_on_another_device():
    """A descriptor of host tensors does not reach the library beside queries on the GPU."""
    c, _, _ = G.prefix_case(73, F32, 4, 2, 64, 16, 2, 1, [5, 9])
    k, v, table = c["kv"].keep
    ws = api.alloc_prefix_workspace(c["shape"])
    for tensors in ((k.cpu(), v, table), (k, v.cpu(), table), (k, v, table.cpu())):
        kv = api.make_kv(*tensors, 16, [21, 25])
        with pytest.raises(ValueError, match="one CUDA device"):
            api.sv_prefix_attend(ws=ws, **{**c, "kv": kv})


# ------------------------------------------------------------------ large batches
@pytest.mark.parametrize("dtype,B,T", [(BF16, 65, 1), (BF16, 300, 3), (F32, 129, 1), (BF16, 1024, 1)])
def test_prefix_of_a_large_ragged_batch(dtype, B, T):
    """More samples of one prompt than the verification calls take, each with its own tail."""
    own = [(37 * b) % 90 for b in range(B)]
    c, want, tol = G.prefix_case(75, dtype, 8, 2, 64, 16, T, 20, own)
    ws = api.alloc_prefix_workspace(c["shape"])
    api.sv_prefix_attend(ws=ws, **c)
    assert api.sv_read_status(ws) == 0
    P.check(c["out"], want, tol)


@pytest.mark.parametrize("dtype,Hq,Hkv,d,T,shared,own", [
    (BF16, 8, 2, 128, 1, 900, [3000, 5]), (BF16, 4, 1, 64, 5, 40, [9000]),
    (BF16, 32, 4, 128, 16, 400, [700] * 6), (BF16, 200, 1, 64, 3, 300, [4000, 40]),
    (BF16, 4, 4, 64, 1, 700, [(61 * b) % 800 for b in range(200)]),
    (BF16, 4, 2, 256, 2, 500, [2000, 9]), (F32, 4, 2, 64, 1, 900, [6000, 5]),
    (F32, 6, 2, 64, 20, 200, [3000, 100, 0]), (F32, 4, 4, 64, 1, 300, [(61 * b) % 400 for b in range(150)])])
def test_prefix_stays_in_its_workspace(dtype, Hq, Hkv, d, T, shared, own):
    """Plans with many cut runs: not a byte behind the workspace's size is written (what
    follows it here is as large as the partial rows of the widest plan)."""
    c, want, tol = G.prefix_case(77, dtype, Hq, Hkv, d, 16, T, shared, own)
    n = api.alloc_prefix_workspace(c["shape"]).numel()
    room = torch.zeros(n + 4 * 640 * 64 * (4 * d + 8), dtype=torch.uint8, device="cuda")
    room[n:] = 0xA5
    api.sv_prefix_attend(ws=room[:n], **c)
    assert api.sv_read_status(room[:n]) == 0
    assert bool((room[n:] == 0xA5).all())
    P.check(c["out"], want, tol)


# ------------------------------------------------------------------ plans of large calls
@pytest.mark.parametrize("B,blk,nb_max", [(300, 16, 30), (4096, 8, 6)])
def test_tables_of_a_large_admission(B, blk, nb_max):
    """More than 32768 new tokens, and padding behind them: a cluster of sixteen CTAs."""
    r = random.Random(B)
    old = [r.choice([0, 0, r.randint(0, nb_max * blk // 3)]) for _ in range(B)]
    new = [r.choice([0, r.randint(nb_max * blk // 2, nb_max * blk)]) if r.random() < 0.9 else n for n in old]
    pages = B * nb_max
    perm = list(range(pages))
    r.shuffle(perm)
    table, at = [], 0
    for n in old:
        h = P.nb(n, blk)
        table.append(perm[at:at + h] + [-7] * (nb_max - h))
        at += h
    want = P.tables(blk, old, new, [0] * B, table, perm[at:] + [0] * at, pages - at)
    n = want[3][-1]
    assert n > 32768
    got = G.run_tables(blk, old, new, table, perm[at:] + [0] * at, pages - at, n + 1000)
    assert got[6] == 0 and got[2] == [want[2]] and got[3] == want[3]
    assert got[0] == want[0] and got[1] == want[1]
    assert got[4] == want[4] + [-1] * 1000 and got[5] == want[5] + [-1] * 1000


@pytest.mark.parametrize("dtype,Hq,Hkv,n,every", [
    (BF16, 8, 8, 30000, 97), (F32, 8, 8, 15000, 61), (BF16, 32, 8, 32768, 251), (BF16, 14, 7, 30000, 97)])
def test_prompt_of_many_rows_over_large_heads(dtype, Hq, Hkv, n, every):
    """One long prompt: heads go out in groups whose keys fit a quarter of L2, and the
    last group is smaller where they do not divide (8 heads by three, 7 by three). Rows
    all along the prompt against 64 bits."""
    d, blk = 128, 64
    c = G.prompt_case(81, dtype, Hq, Hkv, d, blk, [n], [n])
    assert G.run_prompt(c) == 0
    rows = torch.arange(0, n, every, device="cuda")
    k, v = (P.gather(c[p], c["block_table"][0], n, blk) for p in ("k_pool", "v_pool"))
    see = torch.arange(n, device="cuda") <= rows[:, None]
    P.check(c["out"][rows], *P.attend(c["q"][rows], k, v, see))
    assert bool(c["out"].isfinite().all())


@pytest.mark.parametrize("dtype,Hkv,shared", [(BF16, 8, 30000), (F32, 7, 15008)])
def test_prefix_over_large_heads(dtype, Hkv, shared):
    """The same for a shared prefix whose heads do not fit a quarter of L2 together."""
    own = [(211 * b) % 500 for b in range(12)]
    c, want, tol = G.prefix_case(83, dtype, Hkv, Hkv, 128, 16, 4, shared // 16, own)
    ws = api.alloc_prefix_workspace(c["shape"])
    api.sv_prefix_attend(ws=ws, **c)
    assert api.sv_read_status(ws) == 0
    P.check(c["out"], want, tol)


# ------------------------------------------------------------------ roundings
def test_prompt_weights_are_rounded_once():
    """A row whose scores rise by 2^100 in the first half of a key tile moves the softmax
    reference of its warp's rows after the other half's weights were rounded to bf16. Only that
    half's values are not zero and its weights are alike, so a second rounding shows."""
    ctx, blk, d, H = [900] * 48, 64, 64, 4
    c = G.prompt_case(93, BF16, H, H, d, blk, ctx, ctx, hole=0.0)
    q, k, v, t = c["q"], c["k_pool"], c["v_pool"], c["block_table"].long()
    log2 = d ** 0.5 / 1.442695  # a product of two entries that makes a score of 2^1
    r = torch.Generator(device="cuda").manual_seed(1)
    for x in (q, k, v):
        x.zero_()
    q[:, :, 0] = (torch.arange(len(q), device="cuda") % 16 == 7)[:, None]
    k[t[:, 700 // blk], :, 700 % blk, 0] = 100 * log2
    q[:, :, 1] = torch.rand(len(q), H, generator=r, device="cuda") * log2  # the second half's scores
    q[:, :, 2] = torch.rand(len(q), H, generator=r, device="cuda") * log2  # one of the first half's
    k[t[:, 641 // blk], :, 641 % blk, 2] = 1
    for i in range(704, 768):
        k[t[:, i // blk], :, i % blk, 1] = 1
        v[t[:, i // blk], :, i % blk] = 1
    assert G.run_prompt(c) == 0
    P.check(c["out"], *G.prompt_want(c, ctx, ctx))


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [(BF16, 8, 2, 128), (BF16, 3, 3, 64), (BF16, 2, 1, 256), (F32, 4, 2, 64)])
def test_a_row_of_one_key_is_its_value(dtype, Hq, Hkv, d):
    ctx = [1, 300, 1, 70]
    c = G.prompt_case(95, dtype, Hq, Hkv, d, 16, ctx, ctx)
    assert G.run_prompt(c) == 0
    for b in range(4):
        value = P.gather(c["v_pool"], c["block_table"][b], 1, 16)[0]
        same(c["out"][int(c["cu_q"][b])], value.repeat_interleave(Hq // Hkv, 0), "from the value")
# ------------------------------------------------------------------ large values
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("octaves", [20, 31, 33, 50, 63, 66])
def test_prompt_large_values_behind_a_jump(Hq, Hkv, d, octaves):
    """Values of 1e24 (sums of 128 of them are far inside fp32) and a score that rises by up to
    2^66 inside a key tile: the result is a mean of values, and finite."""
    ctx, blk = [900] * 48, 64  # (so many that no sequence's keys are cut into runs)
    c = G.prompt_case(91, BF16, Hq, Hkv, d, blk, ctx, ctx, hole=0.0)
    t = c["block_table"].long()
    c["q"][:, :, 3] = 4.0
    c["k_pool"][:, :, :, 3] = 0.0
    for i, part in ((333, 1.0), (450, 2.0), (700, 3.0)):  # scores of 2^0, then these
        c["k_pool"][t[:, i // blk], :, i % blk] = 0.0
        c["k_pool"][t[:, i // blk], :, i % blk, 3] = part * octaves * 0.6931 * d ** 0.5 / 4.0
    c["v_pool"].mul_(1e24)
    want, tol = G.prompt_want(c, ctx, ctx)
    assert bool(want.abs().max() < 1e26)
    assert G.run_prompt(c) == 0
    P.check(c["out"], want, tol)


# ------------------------------------------------------------------ calls at the same time
def test_calls_on_two_streams_with_a_workspace_each():
    """Calls that overlap, each with a workspace of its own, give the bits that they give alone."""
    a = G.prompt_case(97, BF16, 8, 2, 128, 64, [3000, 1, 700], [3000, 1, 64])
    b = G.prompt_case(98, F32, 8, 2, 64, 16, [900, 300], [900, 300])
    p, _, _ = G.prefix_case(99, BF16, 8, 1, 128, 64, 4, 30, [300, 0, 77])
    wa, wb = (api.alloc_prompt_workspace(c["shape"], c["q"].shape[0]) for c in (a, b))
    wp = api.alloc_prefix_workspace(p["shape"])
    len0, len1 = G.i32([0, 40, 7]), G.i32([90, 0, 300])
    grow = dict(old_len=len0, new_len=len1, free_pages=G.i32(list(range(64))), free_count=G.i32([60]),
                free_count_out=G.i32([0]), cu_new=G.i32([0] * 4), slot_map=G.i32([0] * 400))
    tables = [torch.full((3, 32), 63, dtype=torch.int32, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()

    def first(table):
        api.sv_build_tables(16, block_table=table, ws=wa, **grow)
        api.sv_prompt_attend(ws=wa, **a)

    def second():
        api.sv_prefix_attend(ws=wp, **p)
        api.sv_prompt_attend(ws=wb, **b)

    first(tables[0])
    second()
    torch.cuda.synchronize()
    outs = [a["out"], b["out"], p["out"]]
    alone = [x.clone() for x in outs] + [grow["slot_map"].clone()]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(30):
        for x in outs:
            x.fill_(7.0)
        grow["free_pages"].copy_(G.i32(list(range(64))))
        tables[1].fill_(63)
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(t):
                second()
        with torch.cuda.stream(s):
            first(tables[1])
        torch.cuda.synchronize()
        for x, y in zip(outs + [grow["slot_map"]], alone):
            same(x, y, "beside calls on another stream")
        assert torch.equal(tables[0], tables[1])
    assert all(api.sv_read_status(w) == 0 for w in (wa, wb, wp))
