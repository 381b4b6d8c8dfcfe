"""What the paged-cache calls take and refuse, on the host: no GPU is touched."""
import ctypes as C

import pytest
import torch

from sparse_verification_attention_gb300 import api, build_lib


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return api.lib()


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def test_prefix_refuses_a_cache_of_another_shape(L):
    """A descriptor made for fewer sequences, other heads, pages or types than the call's
    would be read past its ends."""
    B, T, Hq, Hkv, d, blk = 3, 2, 4, 2, 64, 16
    s = api.make_shape(B, Hq, Hkv, d, blk, T, torch.float32)
    q, dk = torch.zeros(B, T, Hq, d), torch.zeros(B, T, Hkv, d)
    ws = torch.zeros(1 << 10, dtype=torch.uint8)

    def call(k, v, table, seq_ctx=None):
        kv = api.make_kv(k, v, table, 16, seq_ctx)
        api.sv_prefix_attend(s, q, kv, 0, dk, dk, None, torch.zeros_like(q), ws)

    pool, table = torch.zeros(5, Hkv, blk, d), i32(B, 4)
    for name, bad in (("block_table", dict(table=i32(B - 1, 4))),
                      ("block_table", dict(table=i32(B - 1, 4), seq_ctx=[16] * (B - 1))),
                      ("block_table", dict(table=i32(B, 4).long())),
                      ("block_table", dict(table=i32(4, B).t())),
                      ("k_pool", dict(k=torch.zeros(5, Hkv, 8, d))),
                      ("k_pool", dict(k=torch.zeros(5, 1, blk, d))),
                      ("k_pool", dict(k=pool.bfloat16())),
                      ("k_pool", dict(k=torch.zeros(5, Hkv, d, blk).transpose(2, 3))),
                      ("v_pool", dict(v=pool[:4])),
                      ("v_pool", dict(v=torch.zeros(5, Hkv, blk, 32))),
                      ("v_pool", dict(v=pool.double()))):
        with pytest.raises(ValueError, match=name):
            call(**{**dict(k=pool, v=pool, table=table), **bad})
    for good in ({}, dict(table=i32(B + 1, 4)), dict(seq_ctx=[16, 0, 7])):
        with pytest.raises(ValueError, match="one CUDA device"):  # right, but not on a GPU
            call(**{**dict(k=pool, v=pool, table=table), **good})


def test_prefix_takes_as_many_contexts_as_sequences(L):
    """Per-sequence contexts for all of the 1024 sequences that a call may have."""
    fake = 1 << 20  # never dereferenced: the workspace is refused
    for B in (64, 65, 1024, 1025):
        s = api.make_shape(B, 4, 2, 64, 16, 4, torch.float32)
        lens = (C.c_int32 * B)(*[16 + b % 50 for b in range(B)])
        kv = api.KV(fake, fake, fake, 10, 64, 0)
        kv.seq_ctx = lens
        st = L.sv_prefix_attend(C.byref(s), fake, C.byref(kv), 1, fake, fake, None, fake, fake, 0, None)
        assert st == (api.SV_ERR_WORKSPACE if B <= 1024 else api.SV_ERR_UNSUPPORTED), B
        st = L.sv_sparse_attend(C.byref(s), fake, C.byref(kv), None, 0, 0, fake, fake, None, fake, fake, 0, None)
        assert st == (api.SV_ERR_WORKSPACE if B <= 64 else api.SV_ERR_UNSUPPORTED), B


def test_misaligned_words_are_refused(L):
    """int32 arrays and the status word off a 4-byte boundary would fault in the kernels."""
    fake = 1 << 20
    s = api.make_shape(2, 4, 2, 64, 16, 4, torch.float32)

    def refused(f, args, at, step=2):
        args = list(args)
        args[at] = fake + step
        st = f(*args)
        msg = L.sv_last_error().decode()
        assert st == api.SV_ERR_INVALID_ARG and "aligned" in msg, (at, st, msg)

    tables = [2, 16, fake, fake, fake, fake, 8, 32, fake, fake, fake, fake, fake, fake, 10, fake, None]
    for i in (2, 3, 4, 5, 8, 9, 10, 11, 12, 13, 15):
        refused(L.sv_build_tables, tables, i)
    write = [C.byref(s), fake, 128, fake, 128, fake, 5, fake, fake, 8, fake, None]
    for i in (5, 10):
        refused(L.sv_write_kv, write, i)
    n = L.sv_prompt_workspace_bytes(C.byref(s), 50)
    prompt = [C.byref(s), fake, 256, 50, fake, fake, fake, 8, 32, fake, fake, fake, fake, n, None]
    for i in (6, 9, 10):
        refused(L.sv_prompt_attend, prompt, i)
    n = L.sv_prefix_workspace_bytes(C.byref(s))
    kv = api.KV(fake, fake, fake + 1, 10, 64, 100)
    prefix = [C.byref(s), fake, C.byref(kv), 6, fake, fake, None, fake, fake, n, None]
    refused(L.sv_prefix_attend, prefix, 1, 0)  # (the table's address is off)


def test_workspaces_must_be_dense(L):
    """A strided or expanded workspace spans other bytes than its size says."""
    s = api.make_shape(2, 4, 2, 64, 16, 4, torch.float32)
    pool, rows = torch.zeros(4, 2, 16, 64), torch.zeros(3, 2, 64)
    q, out = torch.zeros(5, 4, 64), torch.zeros(5, 4, 64)
    q4, dk = torch.zeros(2, 4, 4, 64), torch.zeros(2, 4, 2, 64)
    kv = api.make_kv(pool, pool, i32(2, 3), 16)
    one = torch.zeros(1, dtype=torch.uint8)
    for ws in (torch.zeros(1 << 11, dtype=torch.uint8)[::2], one.expand(1 << 30), one[:0]):
        for call in (lambda: api.sv_prompt_attend(s, q, pool, pool, i32(2, 3), i32(2), i32(3), out, ws),
                     lambda: api.sv_prefix_attend(s, q4, kv, 1, dk, dk, None, torch.zeros_like(q4), ws),
                     lambda: api.sv_write_kv(s, rows, rows, i32(3), pool, pool, ws),
                     lambda: api.sv_build_tables(16, i32(2), i32(2), i32(2, 3), i32(9), i32(1), i32(1),
                                                 i32(3), i32(4), ws=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()


def test_prefix_workspace_follows_the_batch(L):
    """The partial rows of a small batch are few: a cut run holds no more rows than there are."""
    size = lambda **k: L.sv_prefix_workspace_bytes(C.byref(api.make_shape(**k)))  # noqa: E731
    base = dict(Hq=8, Hkv=2, d=128, blk=64, dtype=torch.bfloat16)
    assert size(B=2, T=1, **base) < 16 << 20
    assert size(B=2, T=1, **{**base, "dtype": torch.float32}) < 16 << 20
    last = 0
    for B in (1, 2, 8, 64, 512, 1024):
        assert size(B=B, T=4, **base) > last
        last = size(B=B, T=4, **base)
