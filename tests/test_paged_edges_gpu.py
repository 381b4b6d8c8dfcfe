"""The paged-cache operators where calls of the documentation meet edges: plans
of very many sequences, rows that are not part of a tile, empty caches, pools
that ran out, large batches."""
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
