"""GPU tests of items of more than 128 rows without keys that a CTA takes behind items with them: their zeros pass through the
shared memory that the results before may still be leaving from."""
import numpy as np
import pytest
import torch

import test_gpu_cross as cross
import test_gpu_tree as trees
from _cache_ops import Cache
from _support import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# sequences' keys in turn; each sequence is four items of 160 rows, 152 to a round of CTAs
ORDERS = pytest.mark.parametrize("keys", [[100] * 38 + [0] * 38, ([60] * 38 + [0] * 38) * 2, [0] * 38 + [100] * 38 + [0] * 76])


def same(first, again):
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@ORDERS
@pytest.mark.parametrize("heads", [32, 20])  # (eight heads share one: rows by boxes; five: by lanes)
def test_cross_attention(keys, heads):
    c = Cache(keys, kv_heads=4, heads=heads, device="cuda", seed=95)
    counts = [160 * 4 // heads] * len(keys)
    first = cross.run(c, counts)
    for _ in range(20):
        same(first, cross.run(c, counts, check=False))


@ORDERS
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_trees(keys, dtype):
    c = Cache(keys, kv_heads=4, heads=32, dtype=dtype, device="cuda", seed=96)
    counts = [20] * len(keys)
    masks = [np.tri(20, dtype=bool)] * len(keys)
    first = trees.run(c, counts, masks=masks)
    for _ in range(20):
        same(first, trees.run(c, counts, masks=masks, check=False))
