"""Head norms and rotation, rows to rows and into the paged cache, against the
64-bit form (tests/kv4_util.py, where the tolerances stand)."""
import math

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib
from tests import kv4_util as U

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
    return torch.Generator(device="cuda").manual_seed(seed)


def fused(g, n, Hq, Hkv, d, dtype, scale=1.0):
    """q, k and v rows as slices of one projection's rows."""
    qkv = (torch.randn(n, (Hq + 2 * Hkv) * d, generator=g, device="cuda") * scale).to(dtype)
    return (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))


CASES = [  # n, Hq, Hkv, d, rot, interleaved, norm, dtype
    (1, 32, 8, 128, 128, False, False, BF16), (7, 32, 4, 128, 128, False, True, BF16),
    (130, 8, 2, 96, 48, False, True, F32), (33, 4, 4, 64, 64, True, True, BF16),
    (19, 6, 2, 256, 256, False, True, F32), (5, 3, 3, 256, 40, True, True, BF16),
    (40, 4, 2, 40, 40, False, True, BF16), (9, 2, 1, 8, 8, False, True, F32), (9, 2, 1, 8, 8, True, False, BF16),
    (21, 5, 1, 24, 16, False, True, BF16), (21, 5, 1, 24, 8, True, True, F32), (12, 4, 2, 112, 56, False, True, BF16),
    (17, 4, 2, 64, 0, False, True, F32), (3, 28, 4, 128, 64, True, False, F32), (5000, 2, 1, 64, 64, False, True, BF16)]


def make(case, seed=0, far=5000):
    n, Hq, Hkv, d, rot, inter, norm, dtype = case
    g = gen(seed)
    q, k, v = fused(g, n, Hq, Hkv, d, dtype)
    pos = torch.randint(0, far, (n,), generator=g, device="cuda").to(torch.int32)
    table = api.rope_table(far, rot) if rot else None
    w = [(1 + torch.randn(d, generator=g, device="cuda") / 4).to(dtype) if norm else None for _ in range(2)]
    r = api.make_rope(table, rot, inter, *w, eps=1e-5)
    return q, k, v, pos, r, api.make_shape(1, Hq, Hkv, d, 16, 1, dtype)


def want(case, x, r, side, pos):
    return U.rope(x, r._tensors[1 + side], 1e-5, r._tensors[0], case[4], case[5], pos)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_rope(case):
    q, k, _, pos, r, s = make(case)
    q_out, k_out = torch.full_like(q.contiguous(), 7), torch.full_like(k.contiguous(), 7)
    ws = status_ws()
    api.sv_norm_rope(s, r, pos, q, k, q_out, k_out, ws)
    assert api.sv_read_status(ws) == 0
    U.check(q_out, *want(case, q, r, 0, pos))
    U.check(k_out, *want(case, k, r, 1, pos))
    # in place, and keys alone: the same bits
    q2, k2 = q.clone(), k.clone()
    api.sv_norm_rope(s, r, pos, q2, k2, q2, k2)
    k3 = torch.zeros_like(k_out)
    api.sv_norm_rope(s, r, pos, None, k, None, k3)
    assert torch.equal(q2, q_out) and torch.equal(k2, k_out) and torch.equal(k3, k_out)


def test_one_side_normed():
    case = (11, 4, 2, 64, 64, False, True, F32)
    q, k, _, pos, r, s = make(case)
    for qw, kw in ((r._tensors[1], None), (None, r._tensors[2])):
        one = api.make_rope(r._tensors[0], 64, False, qw, kw, 1e-5)
        q_out, k_out = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
        api.sv_norm_rope(s, one, pos, q, k, q_out, k_out)
        U.check(q_out, *want(case, q, one, 0, pos))
        U.check(k_out, *want(case, k, one, 1, pos))


def test_zero_huge_and_non_finite_rows():
    """Zero rows stay zero under a norm, rows of huge and of tiny elements keep their
    direction, values that are not finite stay in their own pair without a norm."""
    case = (6, 2, 1, 64, 32, False, True, F32)
    q, k, _, pos, r, s = make(case)
    q, k = q.clone(), k.clone()
    q[0] = 0
    q[1] *= 1e15
    q[2] *= 1e-15
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    api.sv_norm_rope(s, r, pos, q, k, q_out, k_out)
    assert not q_out[0].any()
    U.check(q_out[1:], *want(case, q[1:], r, 0, pos[1:]))
    bare = api.make_rope(r._tensors[0], 32)
    q[3, 0, 5], q[3, 1, 40], q[4, 0, 63] = math.inf, math.nan, -math.inf
    api.sv_norm_rope(s, bare, pos, q, k, q_out, k_out)
    odd = ~q_out[3:5].isfinite()
    assert {tuple(x) for x in odd.nonzero().tolist()} <= {(0, 0, 5), (0, 0, 21), (0, 1, 40), (1, 0, 63)}
    assert q_out[4, 0, 63] == -math.inf and q_out[3, 1, 40].isnan()


def test_far_positions_and_padding():
    """The last position of a long table; rows of position -1 stay, others outside the
    table raise a flag and stay."""
    far = 200_003
    case = (8, 4, 2, 128, 128, False, False, BF16)
    q, k, _, pos, r, s = make(case, far=far)
    pos[:6] = i32([far - 1, 0, -1, far, -2, 2 ** 31 - 1])
    q_out, k_out = torch.full_like(q.contiguous(), 7), torch.full_like(k.contiguous(), 7)
    ws = status_ws()
    api.sv_norm_rope(s, r, pos, q, k, q_out, k_out, ws)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_LENGTH
    assert (q_out[2:6] == 7).all() and (k_out[2:6] == 7).all()
    on = torch.tensor([0, 1, 6, 7], device="cuda")
    U.check(q_out[on], *want(case, q[on], r, 0, pos[on]))
    U.check(k_out[on], *want(case, k[on], r, 1, pos[on]))
    ws = status_ws()
    pos[3:6] = -1
    api.sv_norm_rope(s, r, pos, q, k, q_out, k_out, ws)
    assert api.sv_read_status(ws) == 0


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rope_write_kv_is_norm_rope_and_write_kv(case):
    q, k, v, pos, r, s = make(case, seed=1)
    n, Hkv, d, dtype, blk = case[0], case[2], case[3], case[7], 16
    pages = n // blk + 3
    slots = torch.randperm(pages * blk, generator=gen(2), device="cuda")[:n].to(torch.int32)
    skip = torch.rand(n, generator=gen(3), device="cuda") < 0.2
    slots[skip] = -1
    if n > 2:
        pos[1] = -1
    g = gen(4)
    pools = [torch.randn(pages, Hkv, blk, d, generator=g, device="cuda").to(dtype) for _ in range(2)]
    a, b = [x.clone() for x in pools], [x.clone() for x in pools]
    q_out = [torch.full_like(q.contiguous(), 7) for _ in range(3)]
    ws = status_ws()
    api.sv_rope_write_kv(s, r, pos, q, k, v, q_out[0], slots, *a, ws)
    assert api.sv_read_status(ws) == 0
    k_out = torch.zeros_like(k.contiguous())
    api.sv_norm_rope(s, r, pos, q, k, q_out[1], k_out)
    api.sv_write_kv(s, k_out, v, torch.where(pos >= 0, slots, -1), *b)
    assert torch.equal(q_out[0], q_out[1]) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = [x.clone() for x in pools]
    api.sv_rope_write_kv(s, r, pos, None, k, v, None, slots, *c)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_rope_write_kv_bad_slots():
    case = (5, 4, 2, 64, 64, False, True, BF16)
    q, k, v, pos, r, s = make(case)
    pools = [torch.zeros(2, 2, 16, 64, dtype=BF16, device="cuda") for _ in range(2)]
    ws, q_out = status_ws(), torch.zeros_like(q.contiguous())
    api.sv_rope_write_kv(s, r, pos, q, k, v, q_out, i32([3, 32, -5, -1, 2 ** 31 - 1]), *pools, ws)
    assert api.sv_read_status(ws) == api.SV_FLAG_BAD_PAGE
    U.check(q_out, *want(case, q, r, 0, pos))  # the queries are done all the same
    rows = pools[0].transpose(1, 2).flatten(0, 1)
    assert rows[3].any() and not rows[:3].any() and not rows[4:].any()


def test_captured_step_follows_positions_and_slots():
    case = (12, 8, 2, 64, 64, False, True, BF16)
    q, k, v, pos, r, s = make(case)
    pools = [torch.zeros(4, 2, 16, 64, dtype=BF16, device="cuda") for _ in range(2)]
    slots, q_out = i32(list(range(12))), torch.zeros_like(q.contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.sv_rope_write_kv(s, r, pos, q, k, v, q_out, slots, *pools)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sv_rope_write_kv(s, r, pos, q, k, v, q_out, slots, *pools)
    for step in range(2):
        pos.copy_(i32([(997 * i + 31 * step) % 5000 for i in range(12)]))
        slots.copy_(i32([(5 * i + step) % 64 for i in range(12)]))
        for x in pools:
            x.zero_()
        graph.replay()
        w, tol = want(case, k, r, 1, pos)
        rows = pools[0].transpose(1, 2).flatten(0, 1)
        U.check(rows[slots.long()], w, tol)
        assert torch.equal(pools[1].transpose(1, 2).flatten(0, 1)[slots.long()], v)
        U.check(q_out, *want(case, q, r, 0, pos))


def test_rows_past_4_gib():
    """Strides and pools whose offsets pass 32 bits."""
    case = (3, 2, 1, 128, 128, False, False, BF16)
    _, _, _, pos, r, s = make(case)
    stride = 1_200_000_000  # elements: row 2 begins 4.8 GB behind row 0
    big = torch.zeros(2 * stride + 1024, dtype=BF16, device="cuda")
    rows = big.as_strided((3, 4, 128), (stride, 128, 1))
    rows.copy_(torch.randn(3, 4, 128, generator=gen(6), device="cuda").to(BF16))
    q, k, v = rows[:, :2], rows[:, 2:3], rows[:, 3:]
    pages = 1_100_000  # of 16 tokens: 4.5 GB a pool
    pools = [torch.zeros(pages, 1, 16, 128, dtype=BF16, device="cuda") for _ in range(2)]
    slots = i32([5, pages * 16 - 1, pages * 16 - 40])
    q_out = torch.zeros(3, 2, 128, dtype=BF16, device="cuda")
    api.sv_rope_write_kv(s, r, pos, q, k, v, q_out, slots, *pools)
    U.check(q_out, *want(case, q, r, 0, pos))
    got = [x.view(-1, 1, 128)[slots.long()] for x in pools]
    U.check(got[0], *want(case, k, r, 1, pos))
    assert torch.equal(got[1], v)
