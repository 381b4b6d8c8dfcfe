"""Refusals and sizes of the head-norm, rotation and 4-bit cache calls, on the host:
no GPU is touched (a launch attempt would come back as SV_ERR_CUDA)."""
import ctypes as C

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib
from tests import kv4_util as U

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return api.lib()


def refused(L, fn, args, status, word):
    st = fn(*args)
    msg = L.sv_last_error().decode()
    assert st == status and word in msg, (st, msg)


def shape(B=2, Hq=4, Hkv=2, d=64, blk=16, T=4, dtype=torch.float32):
    return api.make_shape(B, Hq, Hkv, d, blk, T, dtype)


def with_arg(args, i, value):
    return args[:i] + [value] + args[i + 1:]


def ref(x):
    return C.byref(x)


INVALID, UNSUPPORTED = api.SV_ERR_INVALID_ARG, api.SV_ERR_UNSUPPORTED


def rope(**kw):
    f = dict(q_weight=None, k_weight=None, table=FAKE, eps=1e-6, max_pos=100, rot=32, interleaved=0)
    return api.Rope(**{**f, **kw})


@pytest.mark.parametrize("bad,word", [
    (dict(rot=-8), "rot"), (dict(rot=12), "rot"), (dict(rot=72), "rot"), (dict(table=None), "table"),
    (dict(max_pos=0), "max_pos"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(q_weight=FAKE + 8), "aligned"), (dict(table=FAKE + 2), "aligned")])
def test_rope_descriptor_refusals(L, bad, word):
    s, r = shape(), rope(**bad)
    refused(L, L.sv_norm_rope, [ref(s), ref(r), FAKE, 5, FAKE, 256, FAKE, 128, FAKE, 256, FAKE, 128, None, None],
            INVALID, word)
    refused(L, L.sv_rope_write_kv, [ref(s), ref(r), FAKE, 5, FAKE, 256, FAKE, 256, FAKE, 128, FAKE, 128, FAKE, FAKE,
                                    FAKE, 8, None, None], INVALID, word)


def test_norm_rope_refusals(L):
    s, r = shape(), rope()
    ok = [ref(s), ref(r), FAKE, 5, FAKE, 256, FAKE, 128, FAKE, 256, FAKE, 128, None, None]
    f = L.sv_norm_rope
    refused(L, f, with_arg(ok, 1, None), INVALID, "rope is NULL")
    refused(L, f, with_arg(ok, 2, None), INVALID, "positions")
    refused(L, f, with_arg(ok, 3, -1), INVALID, "negative")
    for i, name in ((6, "k is"), (8, "q_out is"), (10, "k_out is")):
        refused(L, f, with_arg(ok, i, None), INVALID, name)
    for i in (4, 6, 8, 10):
        refused(L, f, with_arg(ok, i, FAKE + 8), INVALID, "aligned")
    for i in (5, 7, 9, 11):
        refused(L, f, with_arg(ok, i, 127), INVALID, "apart")
        refused(L, f, with_arg(ok, i, 258), INVALID, "multiple of 16 bytes")
    refused(L, f, with_arg(ok, 12, FAKE + 2), INVALID, "aligned")
    refused(L, f, with_arg(ok, 0, ref(shape(d=60))), UNSUPPORTED, "head dim")
    assert f(*with_arg(ok, 3, 0)) == api.SV_OK  # no rows: nothing launched


def test_rope_write_kv_refusals(L):
    s, r = shape(), rope()
    ok = [ref(s), ref(r), FAKE, 5, FAKE, 256, FAKE, 256, FAKE, 128, FAKE, 128, FAKE, FAKE, FAKE, 8, None, None]
    f = L.sv_rope_write_kv
    for i in (6, 8, 10, 12, 13, 14):
        refused(L, f, with_arg(ok, i, None), INVALID, "NULL")
    for i in (4, 6, 8, 10, 13, 14):
        refused(L, f, with_arg(ok, i, FAKE + 8), INVALID, "aligned")
    for i in (9, 11):
        refused(L, f, with_arg(ok, i, 127), INVALID, "apart")
    refused(L, f, with_arg(ok, 15, 0), INVALID, "num_pages")
    refused(L, f, with_arg(ok, 15, 1 << 26), UNSUPPORTED, "too large")
    refused(L, f, with_arg(ok, 3, -1), INVALID, "negative")
    assert f(*with_arg(ok, 3, 0)) == api.SV_OK


def kv4(**kw):
    f = dict(k_pool=FAKE, v_pool=FAKE, block_table=FAKE, seq_ctx=FAKE, k_exp=None, v_exp=None, nb_max=10, num_pages=64)
    return api.KV4(**{**f, **kw})


def calls4(L, s, kv):
    """Every call over a 4-bit cache, with arguments that only the cache can spoil."""
    n = max(L.sv_kv4_workspace_bytes(ref(s)), 1)
    return [(L.sv_write_kv4, [ref(s), FAKE, 4096, FAKE, 4096, FAKE, 5, ref(kv), None, None]),
            (L.sv_read_kv4, [ref(s), ref(kv), FAKE, 5, FAKE, 4096, FAKE, 4096, None, None]),
            (L.sv_build_reps_kv4, [ref(s), ref(kv), None, 3, FAKE, None, None]),
            (L.sv_attend_kv4, [ref(s), FAKE, ref(kv), None, 0, 0, FAKE, FAKE, None, FAKE, FAKE, n, None])]


@pytest.mark.parametrize("bad,status,word", [
    (dict(k_pool=None), INVALID, "NULL"), (dict(v_pool=None), INVALID, "NULL"),
    (dict(k_pool=FAKE + 8), INVALID, "aligned"), (dict(v_pool=FAKE + 4), INVALID, "aligned"),
    (dict(num_pages=0), INVALID, "num_pages"), (dict(num_pages=1 << 26), UNSUPPORTED, "too large"),
    (dict(k_exp=FAKE + 2), INVALID, "aligned"), (dict(v_exp=FAKE + 1), INVALID, "aligned")])
def test_cache_refusals(L, bad, status, word):
    for f, args in calls4(L, shape(), kv4(**bad)):
        refused(L, f, args, status, word)


@pytest.mark.parametrize("bad,status,word", [
    (dict(block_table=None), INVALID, "NULL"), (dict(seq_ctx=None), INVALID, "NULL"),
    (dict(nb_max=0), INVALID, "nb_max"), (dict(nb_max=1 << 27), UNSUPPORTED, "too large"),
    (dict(seq_ctx=FAKE + 2), INVALID, "aligned")])
def test_sequence_refusals(L, bad, status, word):
    for f, args in calls4(L, shape(), kv4(**bad))[2:]:
        refused(L, f, args, status, word)


@pytest.mark.parametrize("kw,word", [(dict(d=24), "multiple of 16"), (dict(blk=24), "multiple of 16"),
                                     (dict(d=272), "head dim"), (dict(T=65), "T=65"),
                                     (dict(Hq=4097, Hkv=4097), "exceed"), (dict(B=65536), "exceed")])
def test_shapes_without_a_4bit_cache(L, kw, word):
    s = shape(**kw)
    for f, args in calls4(L, s, kv4()):
        refused(L, f, args, UNSUPPORTED, word)
    assert L.sv_kv4_page_bytes(ref(s)) == 0 and L.sv_kv4_workspace_bytes(ref(s)) == 0


def test_row_call_refusals(L):
    s, kv = shape(), kv4()
    w = [ref(s), FAKE, 128, FAKE, 128, FAKE, 5, ref(kv), None, None]
    r = [ref(s), ref(kv), FAKE, 5, FAKE, 128, FAKE, 128, None, None]
    for f, ok, rows, slots, n in ((L.sv_write_kv4, w, (1, 3), 5, 6), (L.sv_read_kv4, r, (4, 6), 2, 3)):
        for i in rows + (slots,):
            refused(L, f, with_arg(ok, i, None), INVALID, "NULL")
        for i in rows:
            refused(L, f, with_arg(ok, i, FAKE + 8), INVALID, "aligned")
            refused(L, f, with_arg(ok, i + 1, 124), INVALID, "apart")
            refused(L, f, with_arg(ok, i + 1, 130), INVALID, "multiple of 16 bytes")
        refused(L, f, with_arg(ok, n, -1), INVALID, "negative")
        refused(L, f, with_arg(ok, slots, FAKE + 2), INVALID, "aligned")
        assert f(*with_arg(ok, n, 0)) == api.SV_OK


def test_reps_refusals(L):
    s, kv = shape(), kv4()
    ok = [ref(s), ref(kv), None, 3, FAKE, None, None]
    f = L.sv_build_reps_kv4
    refused(L, f, with_arg(ok, 3, -1), INVALID, "max_blocks")
    refused(L, f, with_arg(ok, 3, 11), INVALID, "max_blocks")
    refused(L, f, with_arg(ok, 4, None), INVALID, "reps")
    refused(L, f, with_arg(ok, 4, FAKE + 4), INVALID, "reps")
    refused(L, f, with_arg(ok, 2, FAKE + 2), INVALID, "aligned")
    assert f(*with_arg(ok, 3, 0)) == api.SV_OK


def test_attend_refusals(L):
    s, kv = shape(), kv4()
    n = L.sv_kv4_workspace_bytes(ref(s))
    ok = [ref(s), FAKE, ref(kv), FAKE, 4, 6, FAKE, FAKE, None, FAKE, FAKE, n, None]
    f = L.sv_attend_kv4
    for i in (1, 2, 6, 7, 9, 10):
        refused(L, f, with_arg(ok, i, None), INVALID, "NULL")
    for i in (1, 6, 7, 9, 10):
        refused(L, f, with_arg(ok, i, FAKE + 8), INVALID, "aligned")
    refused(L, f, with_arg(ok, 3, FAKE + 2), INVALID, "aligned")
    refused(L, f, with_arg(ok, 4, 7), INVALID, "n_sel")
    refused(L, f, with_arg(ok, 4, -1), INVALID, "n_sel")
    refused(L, f, with_arg(with_arg(ok, 4, 11), 5, 20), INVALID, "nb_max")
    refused(L, f, with_arg(ok, 11, n - 1), api.SV_ERR_WORKSPACE, "needs")
    refused(L, f, with_arg(ok, 8, (C.c_int32 * 4)(-1, 0, 2, 1)), INVALID, "draft_parent")
    refused(L, f, with_arg(ok, 0, ref(shape(B=1025))), UNSUPPORTED, "1025 sequences")


def test_sizes(L):
    assert L.sv_kv4_page_bytes(ref(shape())) == 2 * 16 * 64 * 9 // 16  # 4.5 bits an element
    w = lambda **kw: L.sv_kv4_workspace_bytes(ref(shape(**kw)))  # noqa: E731
    assert 0 < w() < w(B=64) and w(T=1) < w(T=64) and w(d=64) < w(d=128) and w(B=1025) == 0


def test_binding_refuses_what_it_cannot_pass(L):
    s = shape()
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    q, k, pos = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), i32(3)
    table = torch.zeros(10, 32)
    r = api.make_rope(table)
    assert (r.rot, r.max_pos) == (32, 10)
    for bad in (dict(table=table.double()), dict(table=table, rot=64), dict(table=table.t()), dict(rot=32)):
        with pytest.raises(ValueError):
            api.make_rope(**bad)
    good = dict(rope=r, positions=pos, q=q, k=k, q_out=q, k_out=k)
    for name, bad in (("positions", i32(4)), ("positions", pos.long()), ("q", q[:2]), ("q", q.double()),
                      ("q", None), ("q_out", q[:, :2]), ("k", k[:2]), ("k_out", k[:2]), ("k", k[:, :, ::2]),
                      ("rope", api.make_rope(table, q_weight=torch.zeros(32))),
                      ("rope", api.make_rope(table, k_weight=torch.zeros(64).bfloat16())), ("k", k)):
        with pytest.raises(ValueError):  # the last: right, but not on a GPU
            api.sv_norm_rope(s, **{**good, name: bad})
    pool = torch.zeros(5, 2, 16, 64)
    good = dict(rope=r, positions=pos, q=q, k=k, v=k, q_out=q, slot_map=i32(3), k_pool=pool, v_pool=pool)
    for name, bad in (("v", k[:2]), ("slot_map", i32(2)), ("k_pool", pool[:, :1]), ("v_pool", pool[:3]),
                      ("q_out", None), ("v", k)):
        with pytest.raises(ValueError):
            api.sv_rope_write_kv(s, **{**good, name: bad})
    p4 = api.alloc_kv4_pool(s, 5, device="cpu")
    assert p4.shape == (5, 2, 1, 576)
    mk = lambda **kw: api.make_kv4(**{**dict(k_pool=p4, v_pool=p4, block_table=i32(2, 3), seq_ctx=i32(2)), **kw})  # noqa: E731
    ws, q4, dk = torch.zeros(4096, dtype=torch.uint8), torch.zeros(2, 4, 4, 64), torch.zeros(2, 4, 2, 64)
    for name, bad in (("k_pool", p4[:, :1]), ("v_pool", p4[:4]), ("k_pool", p4.int()), ("v_pool", p4[..., :570]),
                      ("k_exp", i32(3)), ("v_exp", torch.zeros(2)), ("block_table", i32(3, 3)),
                      ("block_table", None), ("seq_ctx", None), ("seq_ctx", i32(3)), ("seq_ctx", i32(2).long())):
        with pytest.raises(ValueError):
            api.sv_attend_kv4(s, q4, mk(**{name: bad}), None, dk, dk, None, q4, ws)
        with pytest.raises(ValueError):
            api.sv_build_reps_kv4(s, mk(**{name: bad}), 1, torch.zeros(2, 2, 3, 64))
        if name in ("k_pool", "v_pool", "k_exp", "v_exp"):
            with pytest.raises(ValueError):
                api.sv_write_kv4(s, k, k, i32(3), mk(**{name: bad}))
            with pytest.raises(ValueError):
                api.sv_read_kv4(s, mk(**{name: bad}), i32(3), k, k)
    for sel, par, out in ((i32(2, 3, 4), None, q4), (i32(2, 2, 4).long(), None, q4), (None, [-1, 0], q4),
                          (None, None, q4[:1]), (None, None, q4)):
        with pytest.raises(ValueError):
            api.sv_attend_kv4(s, q4, mk(), sel, dk, dk, par, out, ws)
    with pytest.raises(ValueError):
        api.sv_build_reps_kv4(s, mk(), 1, torch.zeros(2, 2, 4, 64))
    with pytest.raises(api.SvError):
        api.alloc_kv4_pool(shape(d=24), 5, device="cpu")


def test_plain_forms_agree_with_the_layout():
    """The tests' own two ways of laying rows out give the same bytes, and read back what was put."""
    g = torch.Generator().manual_seed(3)
    e = torch.tensor([2, -1], dtype=torch.int32)
    kp, vp, table, k, v = U.pools(g, [37, 0, 16], 2, 32, 48, hole=0, k_exp=e, v_exp=e)
    g = torch.Generator().manual_seed(3)
    torch.randperm(kp.shape[0], generator=g)
    for pool, rows, is_v in ((kp, k, False), (vp, v, True)):
        mine = torch.zeros_like(pool)
        for b, n in enumerate([37, 0, 16]):
            code, sb = U.quantise(torch.randn(n, 2, 48, generator=g), e)
            assert torch.equal(U.values(code, sb, e), rows[b])
            U.put_rows(mine, [int(table[b, i // 32]) * 32 + i % 32 for i in range(n)], 32, code, sb, is_v)
        assert torch.equal(mine, pool)


def test_nearest_even_halfway():
    v = torch.tensor(U.LEVELS, dtype=torch.float64)
    x = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.26, 4.99], dtype=torch.float64)
    assert U.nearest_even(x, v).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 1, 6]
