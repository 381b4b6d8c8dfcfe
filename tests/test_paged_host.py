"""Refusals of the paged-cache operators, and their workspace sizes, on the
host: no GPU is touched (a launch attempt would come back as SV_ERR_CUDA)."""
import ctypes as C

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib

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


def test_build_tables_refusals(L):
    ok = [2, 16, FAKE, FAKE, None, FAKE, 8, 32, FAKE, FAKE, FAKE, FAKE, FAKE, None, 10, None, None]
    f = L.sv_build_tables
    for i in (0, 1, 6, 7):
        refused(L, f, with_arg(ok, i, 0), api.SV_ERR_INVALID_ARG, "need B")
    refused(L, f, with_arg(ok, 14, -1), api.SV_ERR_INVALID_ARG, "n_max")
    refused(L, f, with_arg(ok, 0, 4097), api.SV_ERR_UNSUPPORTED, "4097 requests")
    refused(L, f, with_arg(ok, 14, (1 << 30) + 1), api.SV_ERR_UNSUPPORTED, "too large")
    refused(L, f, with_arg(with_arg(ok, 0, 4096), 6, 1 << 19), api.SV_ERR_UNSUPPORTED, "too large")
    refused(L, f, with_arg(ok, 7, 1 << 27), api.SV_ERR_UNSUPPORTED, "2^31")
    refused(L, f, with_arg(ok, 6, 1 << 27), api.SV_ERR_UNSUPPORTED, "2^31")
    for i in (2, 3, 5, 8, 9, 10, 11, 12):
        refused(L, f, with_arg(ok, i, None), api.SV_ERR_INVALID_ARG, "NULL")


def test_write_kv_refusals(L):
    s = shape()
    ok = [C.byref(s), FAKE, 128, FAKE, 128, FAKE, 5, FAKE, FAKE, 8, None, None]
    f = L.sv_write_kv
    for i in (1, 3, 5, 7, 8):
        refused(L, f, with_arg(ok, i, None), api.SV_ERR_INVALID_ARG, "NULL")
    for i in (1, 3, 7, 8):
        refused(L, f, with_arg(ok, i, FAKE + 8), api.SV_ERR_INVALID_ARG, "aligned")
    for i in (2, 4):
        refused(L, f, with_arg(ok, i, 127), api.SV_ERR_INVALID_ARG, "apart")
        refused(L, f, with_arg(ok, i, 130), api.SV_ERR_INVALID_ARG, "multiple of 16 bytes")
    refused(L, f, with_arg(ok, 6, -1), api.SV_ERR_INVALID_ARG, "negative")
    refused(L, f, with_arg(ok, 9, 0), api.SV_ERR_INVALID_ARG, "num_pages")
    refused(L, f, with_arg(ok, 9, 1 << 26), api.SV_ERR_UNSUPPORTED, "too large")
    assert f(*with_arg(ok, 6, 0)) == api.SV_OK  # nothing to write, nothing launched


def test_prompt_attend_refusals(L):
    s = shape()
    n = api.lib().sv_prompt_workspace_bytes(C.byref(s), 50)
    ok = [C.byref(s), FAKE, 256, 50, FAKE, FAKE, FAKE, 8, 32, FAKE, FAKE, FAKE, FAKE, n, None]
    f = L.sv_prompt_attend
    for i in (1, 4, 5, 6, 9, 10, 11, 12):
        refused(L, f, with_arg(ok, i, None), api.SV_ERR_INVALID_ARG, "NULL")
    for i in (1, 4, 5, 11, 12):
        refused(L, f, with_arg(ok, i, FAKE + 8), api.SV_ERR_INVALID_ARG, "aligned")
    refused(L, f, with_arg(ok, 2, 255), api.SV_ERR_INVALID_ARG, "apart")
    refused(L, f, with_arg(ok, 2, 258), api.SV_ERR_INVALID_ARG, "multiple of 16 bytes")
    refused(L, f, with_arg(ok, 3, -1), api.SV_ERR_INVALID_ARG, "n_rows")
    refused(L, f, with_arg(ok, 7, 0), api.SV_ERR_INVALID_ARG, "nb_max")
    refused(L, f, with_arg(ok, 7, 1 << 27), api.SV_ERR_UNSUPPORTED, "block table")
    refused(L, f, with_arg(ok, 8, 0), api.SV_ERR_INVALID_ARG, "num_pages")
    refused(L, f, with_arg(ok, 13, n - 1), api.SV_ERR_WORKSPACE, "needs")
    many = shape(B=1025)
    refused(L, f, with_arg(ok, 0, C.byref(many)), api.SV_ERR_UNSUPPORTED, "1025 sequences")
    bad = shape(d=60)
    refused(L, f, with_arg(ok, 0, C.byref(bad)), api.SV_ERR_UNSUPPORTED, "head dim")
    assert f(*with_arg(ok, 3, 0)) == api.SV_OK  # no rows: nothing launched


def test_prefix_attend_refusals(L):
    s = shape()
    n = api.lib().sv_prefix_workspace_bytes(C.byref(s))
    kv = api.KV(FAKE, FAKE, FAKE, 10, 64, 100)
    ok = [C.byref(s), FAKE, C.byref(kv), 6, FAKE, FAKE, None, FAKE, FAKE, n, None]
    f = L.sv_prefix_attend
    for i in (1, 4, 5, 7, 8):
        refused(L, f, with_arg(ok, i, None), api.SV_ERR_INVALID_ARG, "NULL")
        refused(L, f, with_arg(ok, i, FAKE + 8), api.SV_ERR_INVALID_ARG, "aligned")
    refused(L, f, with_arg(ok, 2, None), api.SV_ERR_INVALID_ARG, "kv")
    refused(L, f, with_arg(ok, 3, 7), api.SV_ERR_INVALID_ARG, "n_shared=7")  # 100 = 6 * 16 + 4
    refused(L, f, with_arg(ok, 3, -1), api.SV_ERR_INVALID_ARG, "n_shared")
    refused(L, f, with_arg(ok, 9, n - 1), api.SV_ERR_WORKSPACE, "needs")
    refused(L, f, with_arg(ok, 6, (C.c_int32 * 4)(-1, 0, 2, 1)), api.SV_ERR_INVALID_ARG, "draft_parent")
    lens = (C.c_int32 * 2)(160, 95)  # the second sequence holds 5 full blocks
    kv2 = api.KV(FAKE, FAKE, FAKE, 10, 64, 0)
    kv2.seq_ctx = C.cast(lens, C.POINTER(C.c_int32))
    refused(L, f, with_arg(ok, 2, C.byref(kv2)), api.SV_ERR_INVALID_ARG, "sequence 1")
    many = shape(B=1025)
    refused(L, f, with_arg(ok, 0, C.byref(many)), api.SV_ERR_UNSUPPORTED, "1025 sequences")


def test_workspace_sizes_grow_with_what_they_hold(L):
    w = lambda s, n: L.sv_prompt_workspace_bytes(C.byref(s), n)  # noqa: E731
    assert w(shape(), 1) <= w(shape(), 100) <= w(shape(), 10 ** 6)
    assert w(shape(d=64), 100) < w(shape(d=128), 100)
    assert w(shape(Hq=5), 1) == 0 and w(shape(), -1) == 0
    p = lambda s: L.sv_prefix_workspace_bytes(C.byref(s))  # noqa: E731
    assert p(shape(B=2)) < p(shape(B=64)) and p(shape(T=1)) < p(shape(T=64))
    assert p(shape(Hq=5)) == 0


def test_binding_refuses_what_it_cannot_pass(L):
    """Tensors of another type, shape or layout than the call reads, and
    tensors outside the GPU, never reach the library."""
    s = shape()
    pool = torch.zeros(4, 2, 16, 64)
    rows = torch.zeros(3, 2, 64)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    for k, v, slots in ((rows, rows, i32(4)), (rows, rows[:2], i32(3)), (rows.double(), rows, i32(3)),
                        (rows, rows, i32(3).long()), (rows.transpose(1, 2), rows, i32(3)),
                        (rows[:, :1], rows, i32(3)), (rows[:, :, ::2], rows, i32(3)),
                        (rows, rows, i32(3))):  # the last: right, but not on a GPU
        with pytest.raises(ValueError):
            api.sv_write_kv(s, k, v, slots, pool, pool)
    q, out, ws = torch.zeros(5, 4, 64), torch.zeros(5, 4, 64), torch.zeros(1 << 10, dtype=torch.uint8)
    good = dict(q=q, k_pool=pool, v_pool=pool, block_table=i32(2, 3), seq_ctx=i32(2), cu_q=i32(3),
                out=out, ws=ws)
    for name, bad in (("q", q[:, :2]), ("out", out[:4]), ("k_pool", pool[:, :, :8]),
                      ("v_pool", pool[:2]), ("block_table", i32(3, 3)), ("seq_ctx", i32(3)),
                      ("cu_q", i32(2)), ("cu_q", i32(3).float()), ("out", out.bfloat16()),
                      ("ws", ws)):
        with pytest.raises(ValueError):
            api.sv_prompt_attend(s, **{**good, name: bad})
    q4 = torch.zeros(2, 4, 4, 64)
    dk = torch.zeros(2, 4, 2, 64)
    kv = api.make_kv(pool, pool, i32(2, 3), 16)
    for q_, dk_, par in ((q4[:1], dk, None), (q4, dk[:, :3], None), (q4, dk, [-1, 0]), (q4, dk, None)):
        with pytest.raises(ValueError):
            api.sv_prefix_attend(s, q_, kv, 1, dk_, dk, par, torch.zeros(2, 4, 4, 64), ws)
    one = dict(old_len=i32(2), new_len=i32(2), block_table=i32(2, 3), free_pages=i32(9),
               free_count=i32(1), free_count_out=i32(1), cu_new=i32(3), slot_map=i32(4))
    for name, bad in (("old_len", i32(3)), ("new_len", i32(2).long()), ("cu_new", i32(2)),
                      ("free_count", i32(2)), ("block_table", i32(3, 2).t()), ("slot_map", i32(2, 2)),
                      ("positions", i32(3)), ("pinned", i32(1)), ("slot_map", i32(4))):
        with pytest.raises(ValueError):
            api.sv_build_tables(16, **{**one, name: bad})
