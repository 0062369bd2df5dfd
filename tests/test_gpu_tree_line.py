"""GPU tests of tree attention where unlike items share a line of work, and with query rows that are not ordinary."""
import numpy as np
import pytest
import torch

from _cache_ops import Cache
from _support import need_gpu
from test_gpu_tree import both, run, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@both
@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("heads,kv_heads,batch", [(32, 4, 14), (8, 8, 120), (40, 2, 30)])
def test_wide_and_narrow_items_in_turn(heads, kv_heads, batch, seed, dtype):
    """Sequences without tokens or keys, items of one block, of up to 128 rows, of 256 and of a few more, long and short."""
    rng = np.random.default_rng(100 + seed)
    counts = [int(x) for x in rng.choice([0, 1, 3, 15, 16, 17, 33, 70], batch, p=[.15, .2, .15, .1, .1, .1, .1, .1])]
    lens = [n + int(x) for n, x in zip(counts, rng.choice([0, 1, 60, 127, 130, 900, 2500], batch))]
    lens = [0 if rng.random() < 0.1 else x for x in lens]
    c = Cache(lens, kv_heads=kv_heads, heads=heads, page=int(rng.choice([16, 64, 256])), dtype=dtype, device="cuda", seed=seed)
    run(c, counts)


@both
def test_a_query_that_is_not_finite_spoils_its_row_alone(dtype):
    c = Cache([700, 40, 260], kv_heads=2, heads=16, dtype=dtype, device="cuda", seed=60)
    counts = [20, 33, 9]
    masks = [tree(np.random.default_rng(i), n) for i, n in enumerate(counts)]
    g = torch.Generator(device="cuda").manual_seed(61)
    q = torch.randn((62, 16, 128), generator=g, device="cuda").to(torch.bfloat16)
    first = run(c, counts, masks=masks, q=q)
    bad = q.clone()
    rows = [(3, 1, "nan"), (3, 15, "inf"), (19, 0, "-inf"), (21, 4, "nan"), (50, 9, "inf"), (61, 15, "nan")]
    good = torch.ones((62, 16), dtype=torch.bool, device="cuda")
    for token, head, x in rows:
        bad[token, head, 5 * head] = float(x)
        good[token, head] = False
    out, lse = run(c, counts, masks=masks, q=bad, check=False)
    assert out[~good].isnan().all() and lse[~good].isnan().all()
    assert torch.equal(out[good], first[0][good]) and torch.equal(lse[good], first[1][good])


@pytest.mark.parametrize("most", [2.0 ** 9, 2.0 ** 120, 2.0 ** -100])
def test_components_far_below_the_largest(most):
    """e4m3: one component of a row is `most`, the others a part of it down to nothing; scores of the usual size."""
    c = Cache([300, 77], kv_heads=2, heads=8, dtype="e4m3", device="cuda", seed=62)
    g = torch.Generator(device="cuda").manual_seed(63)
    q = torch.randn((30, 8, 128), generator=g, device="cuda").double()
    q *= 2.0 ** -torch.randint(0, 30, q.shape, generator=g, device="cuda").double()
    q[:, :, 7] = 1
    run(c, [20, 10], q=(q * most).to(torch.bfloat16), scales=([8 / 64 / most] * 2, [1 / 64] * 2))
