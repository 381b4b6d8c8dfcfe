"""The 4-bit cache: rows in and out, representatives and verification attention,
against the 64-bit forms of tests/kv4_util.py (where the tolerances stand)."""
import math
import random

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib
from sparse_verification_attention_gb300 import workloads as W
from tests import kv4_util as U
from tests import paged_util as P

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TREE16 = list(W.TREE16_PARENTS)


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


# ------------------------------------------------------------------ rows in and out
@pytest.mark.parametrize("n,Hkv,d,blk,dtype,exps", [
    (1, 8, 128, 64, BF16, True), (50, 4, 128, 16, BF16, False), (33, 2, 64, 32, F32, True),
    (17, 1, 16, 16, F32, False), (130, 3, 48, 48, BF16, True), (29, 2, 256, 64, BF16, False), (64, 5, 112, 16, F32, True)])
def test_write_and_read(n, Hkv, d, blk, dtype, exps):
    g = gen(n + d)
    rows = (torch.randn(n, 3, Hkv, d, generator=g) * torch.exp(torch.randn(n, 1, Hkv, 1, generator=g) * 2)).to(dtype)
    k, v = rows[:, 0], rows[:, 2]
    e = [torch.randint(-6, 7, (Hkv,), generator=g).to(torch.int32) if exps else None for _ in range(2)]
    pages = n // blk + 2
    # runs of following slots, some of them skipped
    slots = (torch.arange(n) * 1 + 7) % (pages * blk)
    slots[n // 2:] = torch.randperm(pages * blk, generator=g)[:n - n // 2]
    first = {int(x): i for i, x in reversed(list(enumerate(slots)))}
    slots = torch.tensor([int(x) if first[int(x)] == i and i % 11 != 10 else -1 for i, x in enumerate(slots)])
    s = api.make_shape(1, Hkv, Hkv, d, blk, 1, dtype)
    fill = torch.randint(0, 256, (2, pages, Hkv, blk // 16, 9 * d), generator=g).to(torch.uint8)
    pools = [x.cuda() for x in fill]
    kv = api.make_kv4(*pools, k_exp=None if e[0] is None else e[0].cuda(), v_exp=None if e[1] is None else e[1].cuda())
    ws, dev = status_ws(), rows.cuda()
    api.sv_write_kv4(s, dev[:, 0], dev[:, 2], slots.to(torch.int32).cuda(), kv, ws)
    out = [torch.full((n, Hkv, d), 7, dtype=dtype, device="cuda") for _ in range(2)]
    api.sv_read_kv4(s, kv, slots.to(torch.int32).cuda(), *out, ws)
    assert api.sv_read_status(ws) == 0
    for x, ex, pool, got, is_v, back in ((k, e[0], fill[0], pools[0], False, out[0]), (v, e[1], fill[1], pools[1], True, out[1])):
        code, sb = U.quantise(x, ex)
        mine = pool.clone()
        U.put_rows(mine, slots.tolist(), blk, code, sb, is_v)
        # the sign of a zero is free
        zero = lambda p: torch.where((p & 0x0f) == 8, p & 0xf0, p)  # noqa: E731
        both = lambda p: torch.where((zero(p) & 0xf0) == 0x80, zero(p) & 0x0f, zero(p))  # noqa: E731
        a, b = mine, got.cpu()
        assert torch.equal(a[..., 8 * d:], b[..., 8 * d:])
        assert torch.equal(both(a[..., :8 * d]), both(b[..., :8 * d]))
        w = torch.where((slots >= 0)[:, None, None], U.values(code, sb, ex), torch.full((), 7.0, dtype=torch.float64))
        assert torch.equal(back.cpu().double(), w)


def test_rounding_borders():
    """Elements on, just below and just above every border between two codes, at every
    scale, and group maxima around every border between two scales, in fp32."""
    val = U.e4m3_values()[:127]
    rows = []
    for s in val[1:].tolist():
        for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            x = torch.tensor(b * s, dtype=F32)
            up, down = torch.nextafter(x, x * 2), torch.nextafter(x, x * 0)
            rows.append(torch.stack([torch.tensor(6 * s, dtype=F32), x, up, down, -x, -up, -down, x * 0.5] + [x * 0] * 8))
    for a, b in zip(val[:-1].tolist(), val[1:].tolist()):
        m = torch.tensor(3 * (a + b), dtype=F32)  # 6 times the middle
        for t in (m, torch.nextafter(m, m * 2), torch.nextafter(m, m * 0)):
            rows.append(torch.stack([t, t / 2, t / 3, -t / 5] + [t * 0] * 12))
    x = torch.stack(rows).unsqueeze(1)
    n = len(x)
    pages = n // 16 + 1
    s = api.make_shape(1, 1, 1, 16, 16, 1, F32)
    kv = api.make_kv4(*[api.alloc_kv4_pool(s, pages) for _ in range(2)])
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    api.sv_write_kv4(s, x.cuda(), x.cuda(), slots, kv)
    out = [torch.empty_like(x, device="cuda") for _ in range(2)]
    api.sv_read_kv4(s, kv, slots, *out)
    w = U.values(*U.quantise(x))
    assert torch.equal(out[0].cpu().double(), w) and torch.equal(out[1].cpu().double(), w)


def test_values_that_are_not_finite_or_out_of_range():
    x = torch.randn(5, 1, 32, generator=gen(1)).to(BF16)
    x[0, 0, 3], x[1, 0, 20], x[2, 0, 1], x[3] = math.inf, math.nan, 3e38, 1e-30
    x[4, 0, :16] = 0
    for e in (None, i32([-32]), i32([32]), i32([-1000])):
        s = api.make_shape(1, 1, 1, 32, 16, 1, BF16)
        kv = api.make_kv4(*[api.alloc_kv4_pool(s, 1) for _ in range(2)], k_exp=e, v_exp=e)
        slots = i32([4, 1, 0, 9, 15])
        api.sv_write_kv4(s, x.cuda(), x.cuda(), slots, kv)
        out = [torch.empty_like(x, device="cuda") for _ in range(2)]
        api.sv_read_kv4(s, kv, slots, *out)
        ec = None if e is None else e.cpu().clamp(-32, 32)
        w = U.values(*U.quantise(x, ec), ec)
        assert w[1, 0, 16:].isnan().all() and not w[1, 0, :16].isnan().any()
        for o in out:
            assert torch.equal(o.cpu().double().nan_to_num(-123.0), w.nan_to_num(-123.0))


def test_bad_slots():
    s = api.make_shape(1, 2, 2, 32, 16, 1, BF16)
    x = torch.randn(4, 2, 32, generator=gen(2)).to(BF16).cuda()
    pools = [api.alloc_kv4_pool(s, 2) for _ in range(2)]
    kv, ws, slots = api.make_kv4(*pools), status_ws(), i32([32, 3, -2, 2 ** 31 - 1])
    api.sv_write_kv4(s, x, x, slots, kv, ws)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_PAGE
    out = [torch.full_like(x, 7) for _ in range(2)]
    ws = status_ws()
    api.sv_read_kv4(s, kv, slots, *out, ws)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_PAGE
    w = U.values(*U.quantise(x.cpu()))
    for o in out:
        assert torch.equal(o[1].cpu().double(), w[1]) and (o[[0, 2, 3]] == 7).all()
    # nothing but token 3 was written
    api.sv_write_kv4(s, torch.zeros_like(x), torch.zeros_like(x), slots, kv)
    assert not any(p.any() for p in pools)


def test_reading_slots_that_repeat():
    """From a second stream, into rows that are parts of wider ones."""
    s = api.make_shape(1, 3, 3, 48, 32, 1, BF16)
    x = torch.randn(64, 3, 48, generator=gen(4)).to(BF16)
    kv = api.make_kv4(*[api.alloc_kv4_pool(s, 2) for _ in range(2)])
    api.sv_write_kv4(s, x.cuda(), -x.cuda(), torch.arange(64, dtype=torch.int32, device="cuda"), kv)
    slots = torch.randint(0, 64, (200,), generator=gen(5)).to(torch.int32)
    wide = torch.full((200, 2, 3, 48), 7, dtype=BF16, device="cuda")
    on_gpu = slots.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.sv_read_kv4(s, kv, on_gpu, wide[:, 0], wide[:, 1])
    torch.cuda.current_stream().wait_stream(side)
    w = U.values(*U.quantise(x))[slots.long()]
    assert torch.equal(wide[:, 0].cpu().double(), w) and torch.equal(wide[:, 1].cpu().double(), -w)


def test_pool_past_4_gib():
    s = api.make_shape(1, 1, 1, 128, 16, 1, BF16)
    pages = 3_800_000  # 1152 bytes each
    kv = api.make_kv4(*[torch.empty(pages, 1, 1, 1152, dtype=torch.uint8, device="cuda") for _ in range(2)])
    x = torch.randn(40, 1, 128, generator=gen(3)).to(BF16)
    slots = torch.arange(pages * 16 - 40, pages * 16, dtype=torch.int32, device="cuda")
    api.sv_write_kv4(s, x.cuda(), -x.cuda(), slots, kv)
    out = [torch.empty_like(x, device="cuda") for _ in range(2)]
    api.sv_read_kv4(s, kv, slots, *out)
    w = U.values(*U.quantise(x))
    assert torch.equal(out[0].cpu().double(), w) and torch.equal(out[1].cpu().double(), -w)


# ------------------------------------------------------------------ representatives
@pytest.mark.parametrize("lens,old,Hkv,d,blk", [
    ([130, 16, 0, 15, 47], None, 2, 64, 16), ([700, 64], [100, 63], 8, 128, 64), ([96], [48], 1, 16, 48),
    ([513, 40, 300], [256, 0, 300], 2, 256, 32), ([90], [0], 3, 112, 16)])
def test_reps(lens, old, Hkv, d, blk):
    g = gen(d)
    e = torch.randint(-4, 5, (Hkv,), generator=g).to(torch.int32)
    kp, vp, table, k, _ = U.pools(g, lens, Hkv, blk, d, k_exp=e)
    s = api.make_shape(len(lens), Hkv, Hkv, d, blk, 1, F32)
    table = table.cuda()
    kv = api.make_kv4(kp.cuda(), vp.cuda(), table, i32(lens), e.cuda())
    most = max(n // blk - (old or [0] * 9)[b] // blk for b, n in enumerate(lens))
    for cut in (most, 1, 0):
        reps = torch.full((len(lens), Hkv, table.shape[1], d), 7.0, device="cuda")
        ws = status_ws()
        api.sv_build_reps_kv4(s, kv, cut, reps, None if old is None else i32(old), ws)
        assert api.sv_read_status(ws) == 0
        want, tol = torch.full(reps.shape, 7.0, dtype=torch.float64), torch.zeros(reps.shape, dtype=torch.float64)
        for b, n in enumerate(lens):
            j0 = old[b] // blk if old else 0
            for j in range(j0, min(n // blk, j0 + cut)):
                x = k[b][j * blk:(j + 1) * blk]
                want[b, :, j] = x.mean(0)
                tol[b, :, j] = (2 * blk + 2) * U.U * x.abs().mean(0)
        U.check(reps.cpu(), want, tol)


def test_reps_flags():
    kp, vp, table, k, _ = U.pools(gen(5), [40, 33], 2, 16, 32)
    s = api.make_shape(2, 2, 2, 32, 16, 1, BF16)
    table[1, 0] = 1000
    kv = api.make_kv4(kp.cuda(), vp.cuda(), table.cuda(), i32([40, 33]))
    reps, ws = torch.full((2, 2, table.shape[1], 32), 7.0, device="cuda"), status_ws()
    api.sv_build_reps_kv4(s, kv, 2, reps, None, ws)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_PAGE and (reps[1, :, 0] == 7).all() and (reps[1, :, 1] != 7).all()
    ws = status_ws()
    kv = api.make_kv4(kp.cuda(), vp.cuda(), table.cuda(), i32([40, 0]))
    api.sv_build_reps_kv4(s, kv, 2, reps, i32([-3, 5]), ws)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_LENGTH


# ------------------------------------------------------------------ attention
def on_tensor_cores(Hq, Hkv, d, dtype):
    return dtype == BF16 and d <= 128


def selection(g, lens, Hkv, blk, n_sel, short):
    """Ascending distinct blocks; with `short` some rows end early in -1."""
    sel = torch.full((len(lens), Hkv, n_sel + 1), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            keep = min(n // blk, n_sel - (h + b) % 3 if short else n_sel)
            keep = max(keep, 0)
            sel[b, h, :keep] = torch.randperm(n // blk, generator=g)[:keep].sort().values.to(torch.int32)
    return sel


def visible(lens, b, Hkv, blk, sel, parents, T):
    """Which of a sequence's tokens and drafts each draft sees: [T, Hkv, n + T]."""
    n = lens[b]
    see = torch.ones(T, Hkv, n + T, dtype=torch.bool)
    if sel is not None:
        see[:, :, :n // blk * blk] = False
        for h in range(Hkv):
            for j in sel[b, h].tolist():
                if j >= 0:
                    see[:, h, j * blk:(j + 1) * blk] = True
    see[:, :, n:] = P.draft_mask(parents, T, "cpu")[:, None]
    return see


def problem(seed, lens, Hq, Hkv, d, blk, T, dtype, exps=False, q_size=1.0, size=1.0):
    g = gen(seed)
    e = [torch.randint(-4, 5, (Hkv,), generator=g).to(torch.int32) if exps else None for _ in range(2)]
    kp, vp, table, k, v = U.pools(g, lens, Hkv, blk, d, k_exp=e[0], v_exp=e[1], size=size)
    B = len(lens)
    x = dict(q=(torch.randn(B, T, Hq, d, generator=g) * q_size).to(dtype),
             draft_k=torch.randn(B, T, Hkv, d, generator=g).to(dtype),
             draft_v=torch.randn(B, T, Hkv, d, generator=g).to(dtype))
    dev = {n: t.cuda() for n, t in x.items()}
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    kv = api.make_kv4(kp.cuda(), vp.cuda(), table.cuda(), i32(lens), cu(e[0]), cu(e[1]))
    return api.make_shape(B, Hq, Hkv, d, blk, T, dtype), kv, x, dev, k, v


def run(s, kv, dev, sel, parents, ws=None, n_sel=None, out=None):
    ws = api.alloc_kv4_workspace(s) if ws is None else ws
    out = torch.full_like(dev["q"], 7) if out is None else out
    api.sv_attend_kv4(s, dev["q"], kv, None if sel is None else sel.cuda(), dev["draft_k"], dev["draft_v"], parents, out,
                      ws, n_sel)
    return out, ws


def compare(out, x, k, v, lens, Hkv, blk, sel, parents, f16, only=None):
    T = x["q"].shape[1]
    for b in range(len(lens)) if only is None else only:
        kk = torch.cat([k[b], x["draft_k"][b].double()]).cuda()
        vv = torch.cat([v[b], x["draft_v"][b].double()]).cuda()
        see = visible(lens, b, Hkv, blk, sel, parents, T).cuda()
        U.check(out[b], *U.attend(x["q"][b].cuda(), kk, vv, see, f16))


SHAPES = [  # lens, Hq, Hkv, d, blk, T, parents, dtype
    ([1000, 0, 1, 77], 8, 2, 128, 64, 1, None, BF16),
    ([130, 64, 2049], 32, 8, 128, 64, 8, None, BF16),
    ([333, 16, 500], 8, 1, 128, 16, 16, TREE16, BF16),
    ([700, 129], 16, 2, 64, 32, 5, [-1, 0, 0, 2, 1], BF16),
    ([300, 15], 4, 4, 96, 48, 3, None, BF16),
    ([257], 6, 2, 112, 16, 2, None, BF16),
    ([600, 31], 4, 2, 16, 16, 4, None, BF16),
    ([500, 90], 16, 2, 128, 64, 64, None, BF16),       # 512 rows a KV head
    ([400, 128], 24, 2, 128, 128, 33, None, BF16),     # 396 rows
    ([600, 3], 4, 2, 256, 32, 8, None, BF16),
    ([1500, 0, 333, 1], 8, 4, 64, 16, 4, None, F32),
    ([300, 1000], 6, 1, 144, 16, 16, TREE16, F32),
    ([4000], 2, 2, 48, 16, 1, None, F32)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("exps", [False, True])
def test_attend_every_block(shape, exps):
    lens, Hq, Hkv, d, blk, T, parents, dtype = shape
    s, kv, x, dev, k, v = problem(3, lens, Hq, Hkv, d, blk, T, dtype, exps)
    out, ws = run(s, kv, dev, None, parents)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, lens, Hkv, blk, None, parents, on_tensor_cores(Hq, Hkv, d, dtype))
    again, _ = run(s, kv, dev, None, parents, ws)  # the same workspace, the same bits
    assert torch.equal(out, again)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("n_sel,short", [(1, False), (5, True)])
def test_attend_selection(shape, n_sel, short):
    lens, Hq, Hkv, d, blk, T, parents, dtype = shape
    s, kv, x, dev, k, v = problem(4, lens, Hq, Hkv, d, blk, T, dtype, True)
    n_sel = min(n_sel, kv.nb_max)
    sel = selection(gen(5), lens, Hkv, blk, n_sel, short)
    out, ws = run(s, kv, dev, sel, parents, n_sel=n_sel)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, lens, Hkv, blk, sel[:, :, :n_sel], parents, on_tensor_cores(Hq, Hkv, d, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("blk", [16, 48])
def test_attend_selection_in_any_order(dtype, blk):
    """Long rows with gaps, blocks out of order and some of them twice: a block counts as
    often as its row names it."""
    lens, Hkv, n_sel, T = [3000, 2500, 900], 2, 3000 // blk, 4
    s, kv, x, dev, k, v = problem(15, lens, 8, Hkv, 64, blk, T, dtype, True)
    r = random.Random(blk)
    sel = torch.full((3, Hkv, n_sel), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            for i in range(n_sel):
                if r.random() < (0.9, 0.5, 0.02)[b]:
                    sel[b, h, i] = r.randrange(n // blk)
    out, ws = run(s, kv, dev, sel, None)
    assert api.sv_read_status(ws) == 0
    G = 4
    for b, n in enumerate(lens):
        for h in range(Hkv):
            named = [t for j in sel[b, h].tolist() if j >= 0 for t in range(j * blk, (j + 1) * blk)]
            at = torch.tensor(named + list(range(n // blk * blk, n)), dtype=torch.long)
            kk, vv = (torch.cat([c[b][at, h], x[d][b, :, h].double()])[:, None].cuda()
                      for c, d in ((k, "draft_k"), (v, "draft_v")))
            see = torch.ones(T, 1, len(at) + T, dtype=torch.bool)
            see[:, :, len(at):] = P.draft_mask(None, T, "cpu")[:, None]
            q = x["q"][b, :, h * G:(h + 1) * G]
            U.check(out[b, :, h * G:(h + 1) * G], *U.attend(q.cuda(), kk, vv, see.cuda(), dtype == BF16))


@pytest.mark.parametrize("blk", [80, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_page_sizes(blk, dtype):
    """Pages that end inside a key tile, and pages of several tiles."""
    lens = [1234, blk, blk - 1, 3 * blk + 17]
    s, kv, x, dev, k, v = problem(16, lens, 8, 2, 64, blk, 3, dtype)
    out, ws = run(s, kv, dev, None, None)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, lens, 2, blk, None, None, dtype == BF16)
    sel = selection(gen(17), lens, 2, blk, 3, True)[:, :, :3].contiguous()
    out, ws = run(s, kv, dev, sel, None)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, lens, 2, blk, sel, None, dtype == BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_without_selected_blocks(dtype):
    """n_sel = 0: the partial last blocks and the drafts alone."""
    lens = [100, 64, 0]
    s, kv, x, dev, k, v = problem(6, lens, 8, 2, 64, 32, 4, dtype)
    sel = torch.zeros(3, 2, 0, dtype=torch.int32)
    out, ws = run(s, kv, dev, sel, None)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, lens, 2, 32, sel, None, dtype == BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_flags(dtype):
    lens = [100, 70]
    s, kv, x, dev, k, v = problem(7, lens, 4, 2, 64, 16, 2, dtype)
    f16 = dtype == BF16
    sel = selection(gen(8), lens, 2, 16, 3, False)[:, :, :3].contiguous()
    good = sel.clone()
    sel[0, 0, 1], sel[1, 1, 2] = 6, 2 ** 31 - 1  # block 6 of sequence 0 is its partial last one
    good[0, 0, 1] = good[1, 1, 2] = -1
    out, ws = run(s, kv, dev, sel, None)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_BLOCK_INDEX
    compare(out, x, k, v, lens, 2, 16, good, None, f16)
    # a page outside the pool: its keys are left out
    table = kv._tensors[2].clone()
    table[1, 2] = -7
    kv2 = api.make_kv4(*kv._tensors[:2], table, *kv._tensors[3:])
    out, ws = run(s, kv2, dev, None, None)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_PAGE
    left = torch.tensor([[[0, 1, 2, 3, 4, 5]] * 2, [[0, 1, 3, -1, -1, -1]] * 2])
    compare(out, x, k, v, lens, 2, 16, left, None, f16)
    # lengths outside the table are clamped
    ctx = i32([-5, 70])
    kv3 = api.make_kv4(*kv._tensors[:3], ctx, *kv._tensors[4:])
    out, ws = run(s, kv3, dev, None, None)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_LENGTH
    compare(out, x, [k[0][:0], k[1]], [v[0][:0], v[1]], [0, 70], 2, 16, None, None, f16)
    # a sequence without a single page that is there: its drafts alone
    table[1] = -1
    out, ws = run(s, api.make_kv4(*kv._tensors[:2], table, *kv._tensors[3:]), dev, None, None)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_PAGE
    compare(out, x, [k[0], k[1][:0]], [v[0], v[1][:0]], [100, 0], 2, 16, None, None, f16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("q_size", [1e-6, 30.0, 1e30])
def test_attend_sizes_of_queries(dtype, q_size):
    """Rows of very small and very large queries side by side (scores up to some hundreds;
    beyond that the drafts' fp32 products overflow in any form)."""
    lens = [700, 20]
    s, kv, x, dev, k, v = problem(9, lens, 8, 2, 128, 64, 4, dtype, q_size=1.0, size=0.5)
    if q_size == 1e30:  # one row of the batch, orthogonal to everything but its first dim
        x["q"][0, 1, 3] = 0
        x["q"][0, 1, 3, 0] = 8.0
        x["q"][0, 2, 5] *= 1e-30
    else:
        x["q"][:, 1] *= q_size
    dev["q"].copy_(x["q"])
    out, ws = run(s, kv, dev, None, None)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, lens, 2, 64, None, None, dtype == BF16)


@pytest.mark.parametrize("where", ["first", "last", "rising"])
def test_attend_jumps_of_the_scores(where):
    """One key far above the others at the beginning or the end of a long context, and scores
    that rise all the way: the reference of the weights has to move."""
    n, d = 3000, 128
    s, kv, x, dev, k, v = problem(10, [n], 4, 1, d, 64, 2, BF16, q_size=0.5)
    # keys along one dim: rewrite them through the cache
    col = torch.linspace(-6, 6, n) if where == "rising" else torch.full((n,), -1.0)
    if where != "rising":
        col[0 if where == "first" else n - 1] = 6.0
    kk = torch.zeros(n, 1, d)
    kk[:, 0, :16] = col[:, None] * 2
    x["q"][:, :, :, :16] = 3.0
    dev["q"].copy_(x["q"])
    table = kv._tensors[2][0].long()
    i = torch.arange(n, device="cuda")
    slots = (table[i // 64] * 64 + i % 64).to(torch.int32)
    vals = v[0].float().to(BF16).cuda()
    api.sv_write_kv4(s, kk.to(BF16).cuda(), vals, slots, kv)
    code, sb = U.quantise(kk.to(BF16))
    out, ws = run(s, kv, dev, None, None)
    assert api.sv_read_status(ws) == 0
    compare(out, x, [U.values(code, sb)], [U.values(*U.quantise(vals.cpu()))], [n], 1, 64, None, None, True)


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F32)])
def test_attend_nan_of_an_attended_group(d, dtype):
    """A NaN that a token's own scale holds reaches its sequence and head, and no other."""
    lens = [200, 90]
    s, kv, x, dev, k, v = problem(11, lens, 4, 2, d, 16, 2, dtype)
    table = kv._tensors[2]
    kv._tensors[1][table[1, 2].long(), 1, 0, 8 * d + 3] = 0x7f  # V: head 1, first group, token 35
    out, _ = run(s, kv, dev, None, None)
    assert out[1, :, 2:, :16].isnan().all()
    assert out[0].isfinite().all() and out[1, :, :2].isfinite().all() and out[1, :, 2:, 16:].isfinite().all()


def test_attend_large_batch():
    """1024 sequences, most of them short: many segments a CTA."""
    r = random.Random(3)
    lens = [r.choice([0, 1, 5, 16, 40, 200]) for _ in range(1024)]
    s, kv, x, dev, k, v = problem(12, lens, 8, 2, 128, 16, 2, BF16)
    out, ws = run(s, kv, dev, None, None)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, lens, 2, 16, None, None, True, only=range(0, 1024, 37))


def test_attend_long_context():
    n = 150_001
    s, kv, x, dev, k, v = problem(13, [n, 70], 4, 1, 128, 64, 4, BF16)
    out, ws = run(s, kv, dev, None, None)
    assert api.sv_read_status(ws) == 0
    compare(out, x, k, v, [n, 70], 1, 64, None, None, True)


def test_attend_follows_lengths_in_a_graph():
    """A captured step is replayed with other lengths, tables and selections; a second
    graph and an eager call on another stream have workspaces of their own."""
    lens = [300, 77]
    s, kv, x, dev, k, v = problem(14, lens, 8, 2, 128, 16, 4, BF16)
    ctx, outs, graphs = kv._tensors[3], [], []
    side = torch.cuda.Stream()
    for i in range(2):
        ws, out = api.alloc_kv4_workspace(s), torch.zeros_like(dev["q"])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(s, kv, dev, None, None, ws, out=out)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(s, kv, dev, None, None, ws, out=out)
        outs.append((out, ws))
        graphs.append(g)
    for now in ([300, 77], [0, 5], [129, 64], [300, 1]):
        ctx.copy_(i32(now))
        for o, _ in outs:
            o.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager, _ = run(s, kv, dev, None, None)
        torch.cuda.synchronize()
        cut = lambda y: [y[b][:n] for b, n in enumerate(now)]  # noqa: E731
        for o, ws in outs:
            assert api.sv_read_status(ws) == 0
            compare(o, x, cut(k), cut(v), now, 2, 16, None, None, True)
            assert torch.equal(o, eager)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("sparse", [False, True])
def test_serving_loop(sparse):
    """Prompts and verification steps over a 4-bit cache: pages, head norms and rotation,
    rows into the cache, representatives, selection, verification, accepted drafts appended;
    against the same steps in 64 bits on the values the cache holds."""
    B, Hq, Hkv, d, blk, T, norm_eps = 3, 8, 2, 64, 16, 4, 1e-6
    g = gen(21)
    prompts, dtype = [150, 40, 97], BF16
    nb_max, pages = 20, 70
    s = api.make_shape(B, Hq, Hkv, d, blk, T, dtype)
    kv_t = [api.alloc_kv4_pool(s, pages) for _ in range(2)]
    e = [i32([1, -2]), i32([0, 3])]
    table, lens = torch.full((B, nb_max), -1, dtype=torch.int32, device="cuda"), i32([0] * B)
    kv = api.make_kv4(*kv_t, table, lens, *e)
    free, count = torch.randperm(pages, generator=g).to(torch.int32).cuda(), i32([pages])
    w = [(1 + torch.randn(d, generator=g) / 4).to(dtype).cuda() for _ in range(2)]
    rope = api.make_rope(api.rope_table(1024, d), d, False, *w, norm_eps)
    reps = torch.zeros(B, Hkv, nb_max, d, device="cuda")
    ws, status = api.alloc_kv4_workspace(s), status_ws()

    def write(new, k_rows, v_rows):
        """Pages and slots for the lengths `new`, the rows into the cache, representatives."""
        n = k_rows.shape[0]
        cu, slots, pos = i32([0] * (B + 1)), i32([0] * n), i32([0] * n)
        api.sv_build_tables(blk, lens, i32(new), table, free, count, count, cu, slots, pos, ws=status)
        turned = torch.empty_like(k_rows)
        api.sv_norm_rope(s, rope, pos, None, k_rows, None, turned, status)
        api.sv_write_kv4(s, turned, v_rows, slots, kv, status)
        old = lens.clone()
        lens.copy_(i32(new))
        api.sv_build_reps_kv4(s, kv, nb_max, reps, old, status)
        for held, x, exp in ((held_k, turned, e[0]), (held_v, v_rows, e[1])):
            val = U.values(*U.quantise(x.cpu(), exp.cpu()), exp.cpu())
            at = cu.tolist()
            for b in range(B):
                held[b] = torch.cat([held[b], val[at[b]:at[b + 1]]])

    held_k, held_v = [[torch.zeros(0, Hkv, d, dtype=torch.float64)] * B for _ in range(2)]
    n = sum(prompts)
    write(prompts, *[torch.randn(n, Hkv, d, generator=g).to(dtype).cuda() for _ in range(2)])
    now = list(prompts)
    for step in range(3):
        raw = [torch.randn(B, T, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv)]
        pos = torch.tensor([[c + t for t in range(T)] for c in now], dtype=torch.int32, device="cuda").flatten()
        q, dk = torch.empty_like(raw[0]), torch.empty_like(raw[1])
        api.sv_norm_rope(s, rope, pos, raw[0].flatten(0, 1), raw[1].flatten(0, 1), q.flatten(0, 1), dk.flatten(0, 1), status)
        sel = None
        if sparse:
            nb = max(now) // blk
            kept = api.make_kv(kv_t[0], None, table, 0, now)  # the scoring calls read no pool
            sel = i32([[[-1] * 4] * Hkv] * B)
            score_ws = api.alloc_workspace(s, nb_max, 4)
            api.sv_score_select(s, q, reps, kept, W.Budget(W.BUDGET_FIXED, 4), sel, 4, score_ws)
            assert api.sv_read_status(score_ws) == 0
            score = torch.full((B, Hkv, nb), -math.inf, dtype=torch.float64)
            for b in range(B):
                full = now[b] // blk
                mean = held_k[b][:full * blk].view(full, blk, Hkv, d).mean(1)
                score[b, :, :full] = torch.einsum("hd,jhd->hj", q[b, 0].cpu().double().view(Hkv, -1, d).sum(1), mean)
                for h in range(Hkv):
                    want = score[b, h].topk(min(4, full)).indices.sort().values.tolist()
                    assert [j for j in sel[b, h].tolist() if j >= 0] == want
        out = torch.zeros_like(q)
        api.sv_attend_kv4(s, q, kv, sel, dk, raw[2], None, out, ws)
        assert api.sv_read_status(ws) == 0
        x = dict(q=q.cpu(), draft_k=dk.cpu(), draft_v=raw[2].cpu())
        compare(out, x, held_k, held_v, now, Hkv, blk, None if sel is None else sel.cpu(), None, True)
        # the first 1, 2, .. drafts of each sequence are accepted
        take = [1 + (b + step) % T for b in range(B)]
        rows = [torch.cat([y[b, :take[b]] for b in range(B)]) for y in (raw[1], raw[2])]
        now = [c + m for c, m in zip(now, take)]
        write(now, *rows)
    assert api.sv_read_status(status) == 0


def test_captured_step():
    """Pages, rotation, rows, representatives and attention of a step in one graph, which
    follows the lengths and padding in device memory; the same calls one at a time, each
    waited for, give the same bits."""
    B, Hq, Hkv, d, blk, nb_max, pages, rows = 3, 16, 4, 128, 32, 12, 40, 8
    g = gen(31)
    s = api.make_shape(B, Hq, Hkv, d, blk, 1, BF16)
    rope = api.make_rope(api.rope_table(512, d), q_weight=torch.ones(d, dtype=BF16, device="cuda"))
    free = torch.randperm(pages, generator=g).to(torch.int32).cuda()

    class Side:
        def __init__(self):
            self.pools = [api.alloc_kv4_pool(s, pages) for _ in range(2)]
            self.table = torch.full((B, nb_max), -1, dtype=torch.int32, device="cuda")
            self.lens, self.new = i32([0] * B), i32([0] * B)
            self.free, self.count = free.clone(), i32([pages])
            self.reps = torch.zeros(B, Hkv, nb_max, d, device="cuda")
            self.kv = api.make_kv4(*self.pools, self.table, self.lens)
            self.cu, self.slots, self.pos = i32([0] * (B + 1)), i32([-1] * rows), i32([-1] * rows)
            self.qkv = torch.zeros(rows, Hq + 2 * Hkv, d, dtype=BF16, device="cuda")
            self.q, self.k, self.v = self.qkv.split([Hq, Hkv, Hkv], 1)
            self.out = torch.zeros(B, 1, Hq, d, dtype=BF16, device="cuda")
            self.ws, self.status = api.alloc_kv4_workspace(s), status_ws()

        def step(self, wait):
            old = self.lens.clone()
            for call in (
                    lambda: api.sv_build_tables(blk, self.lens, self.new, self.table, self.free, self.count,
                                                self.count, self.cu, self.slots, self.pos, ws=self.status),
                    lambda: api.sv_norm_rope(s, rope, self.pos, self.q, self.k, self.q, self.k, self.status),
                    # every sequence's last row attends to what is there before the rows enter
                    lambda: api.sv_attend_kv4(s, self.q[:B, None].contiguous(), self.kv, None,
                                              self.k[:B, None].contiguous(), self.v[:B, None].contiguous(), None,
                                              self.out, self.ws),
                    lambda: api.sv_write_kv4(s, self.k, self.v, self.slots, self.kv, self.status),
                    lambda: self.lens.copy_(self.new),
                    lambda: api.sv_build_reps_kv4(s, self.kv, nb_max, self.reps, old, self.status)):
                call()
                if wait:
                    torch.cuda.synchronize()

    graph, eager = Side(), Side()
    stream = torch.cuda.Stream()
    captured = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        graph.step(False)  # (nothing grows: lengths of 0)
    torch.cuda.synchronize()
    with torch.cuda.graph(captured):
        graph.step(False)
    now = [0] * B
    for grow in ([3, 2, 0], [1, 1, 1], [0, 7, 1], [1, 0, 0], [0, 0, 8]):
        x = torch.randn(rows, Hq + 2 * Hkv, d, generator=g).to(BF16)
        now = [a + b for a, b in zip(now, grow)]
        for side in (graph, eager):
            side.qkv.copy_(x)
            side.new.copy_(i32(now))
            side.slots.fill_(-1)
            side.pos.fill_(-1)
        torch.cuda.synchronize()
        captured.replay()
        eager.step(True)
        torch.cuda.synchronize()
        for name in ("qkv", "out", "lens", "reps", "table"):
            assert torch.equal(getattr(graph, name), getattr(eager, name)), name
        assert all(torch.equal(x, y) for x, y in zip(graph.pools, eager.pools))
        assert api.sv_read_status(graph.status) == 0 and api.sv_read_status(graph.ws) == 0


def test_prompt_over_a_copy_of_the_cache():
    """A chunk of a prompt over a sequence in 4 bits: its rows read back into a paged bf16
    cache, the chunk's keys rotated into it, attention there."""
    blk, d, Hq, Hkv, have, new = 16, 64, 4, 2, 75, 30
    s4, kv4, _, _, k, v = problem(15, [have], Hq, Hkv, d, blk, 1, BF16, True)
    s = api.make_shape(1, Hq, Hkv, d, blk, 1, BF16)
    i = torch.arange(have, device="cuda")
    slots = (kv4._tensors[2][0].long()[i // blk] * blk + i % blk).to(torch.int32)
    rows = [torch.zeros(have, Hkv, d, dtype=BF16, device="cuda") for _ in range(2)]
    api.sv_read_kv4(s, kv4, slots, *rows)
    assert torch.equal(rows[0].cpu().double(), k[0]) and torch.equal(rows[1].cpu().double(), v[0])
    pages = P.nb(have + new, blk)
    table = torch.randperm(pages, generator=gen(1)).to(torch.int32).cuda()[None]
    pools = [torch.zeros(pages, Hkv, blk, d, dtype=BF16, device="cuda") for _ in range(2)]
    j = torch.arange(have + new, device="cuda")
    to = (table[0].long()[j // blk] * blk + j % blk).to(torch.int32)
    api.sv_write_kv(s, *rows, to[:have], *pools)
    qkv = torch.randn(new, (Hq + 2 * Hkv) * d, generator=gen(2)).to(BF16).cuda()
    q, kn, vn = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    table_rope = api.rope_table(200, d)
    rope = api.make_rope(table_rope, d)
    q_out = torch.zeros(new, Hq, d, dtype=BF16, device="cuda")
    api.sv_rope_write_kv(s, rope, j[have:].to(torch.int32), q, kn, vn, q_out, to[have:], *pools)
    out, ws = torch.zeros_like(q_out), api.alloc_prompt_workspace(s, new)
    api.sv_prompt_attend(s, q_out, *pools, table, i32([have + new]), i32([0, new]), out, ws)
    kn_turned = torch.zeros(new, Hkv, d, dtype=BF16, device="cuda")
    api.sv_norm_rope(s, rope, j[have:].to(torch.int32), None, kn, None, kn_turned)
    kk = torch.cat([k[0].cuda(), kn_turned.double()])
    vv = torch.cat([v[0].cuda(), vn.double()])
    o, tol = P.attend(q_out, kk, vv, P.causal(new, have + new, "cuda"))
    P.check(out, o, tol)
