"""GPU tests of trees whose items follow one another in a CTA in every kind of turn: both row blocks' (more than 128 rows),
one row block's (up to 128 rows and one key block), and of rows that the row blocks share."""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import Cache
from _support import need_gpu
from test_gpu_tree import both, run

pytestmark = pytest.mark.gpu

# (tokens, keys) of sequences with 8 rows a token
WIDE, LONG_WIDE, SINGLE, SHARED = (20, 90), (20, 400), (3, 70), (9, 300)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def again(c, counts, times):
    """The same bits call after call, with the results against 64 bits first."""
    n = sum(counts)
    q = torch.randn((n, c.heads, 128), generator=torch.Generator(device="cuda").manual_seed(90), device="cuda").to(torch.bfloat16)
    masks = [np.tri(m, dtype=bool) for m in counts]
    first = run(c, counts, masks=masks, q=q)
    for _ in range(times):
        out, lse = run(c, counts, masks=masks, q=q, check=False)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@both
@pytest.mark.parametrize("turns", [[WIDE, SINGLE, SINGLE, SHARED], [LONG_WIDE, SINGLE, SINGLE, WIDE], [SINGLE, WIDE, SINGLE, SHARED],
                                   [SHARED, SINGLE, SINGLE, SINGLE], [WIDE, SINGLE, SHARED, SINGLE]])
def test_four_pieces_to_a_cta(dtype, turns):
    """152 items of each kind, of which every CTA has one."""
    seqs = [s for s in turns for _ in range(38)]
    c = Cache([keys for _, keys in seqs], kv_heads=4, heads=32, dtype=dtype, device="cuda", seed=91)
    assert skv.splitkv_tree_workspace_size(c.desc, sum(n for n, _ in seqs)) > 0
    again(c, [n for n, _ in seqs], 20)


@both
def test_a_line_of_all_kinds(dtype):
    seqs = [WIDE, SINGLE, SINGLE, SHARED, LONG_WIDE, SINGLE, SINGLE, SINGLE, SHARED, SINGLE] * 80
    c = Cache([keys for _, keys in seqs], kv_heads=1, heads=8, dtype=dtype, device="cuda", seed=92)
    again(c, [n for n, _ in seqs], 20)
