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
        assert torch.equal(c["out"], first)
    assert api.sv_read_status(ws) == 0
