"""GPU tests of trees that see keys which are not finite: the formula decides which results are NaN (a row whose scores
hold NaN or +inf is NaN throughout, with its log-sum-exp), and every other row keeps the bits that it has without."""
import numpy as np
import pytest
import torch

from _cache_ops import Cache
from _support import need_gpu
from test_gpu_tree import latent, run, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def set_key(c, b, j, value, values=False):
    pools = [c.k] if c.shares or not values else [c.k, c.v]
    for pool in pools:
        pool[int(c.table[b, j // c.P]), :, j % c.P] = 127 if c.dtype == "e4m3" else value


@pytest.mark.parametrize("dtype,shares", [("bf16", True), ("bf16", False), ("e4m3", True)])
@pytest.mark.parametrize("tokens,lens,cap_pages", [(8, [100, 60], None), (5, [1500, 700], 64), (1, [4000, 3000], 64)])
def test_a_nan_among_latent_rows(dtype, shares, tokens, lens, cap_pages):
    """In one split, in one of several, and in one of so many that ways share the merge."""
    c = latent(lens, tokens, 64, dtype, shares, seed=80, cap_pages=cap_pages)
    masks = [tree(np.random.default_rng(81 + b), tokens) for b in range(2)]
    clean, clean_l = run(c, [tokens] * 2, masks=masks, cu=False, check=False)
    assert clean.isfinite().all() and clean_l.isfinite().all()
    for j in sorted({0, 7, lens[0] // 2, lens[0] - tokens - 1, lens[0] - tokens, lens[0] - (tokens + 1) // 2, lens[0] - 1}):
        kept = c.k.clone()
        set_key(c, 0, j, float("nan"))
        out, lse = run(c, [tokens] * 2, masks=masks, cu=False, check=False)
        i = j - (lens[0] - tokens)  # the drafted token whose key it is
        for t in range(2 * tokens):
            if t < tokens and (i < 0 or masks[0][t, i]):
                assert out[t].isnan().all() and lse[t].isnan().all(), (j, t)
            else:
                assert torch.equal(out[t], clean[t]) and torch.equal(lse[t], clean_l[t]), (j, t)
        c.k.copy_(kept)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("tokens,heads,kv_heads,keys", [(30, 4, 1, 90), (9, 4, 1, 3000), (60, 16, 2, 700)])
def test_an_infinite_key(tokens, heads, kv_heads, keys, sign):
    """One component: +inf in some rows' scores, which are NaN; -inf in the others', where the key has no weight."""
    c = Cache([keys], kv_heads=kv_heads, heads=heads, device="cuda", seed=82)
    sees = tree(np.random.default_rng(83), tokens)
    g = torch.Generator(device="cuda").manual_seed(84)
    q = torch.randn((tokens, heads, 128), generator=g, device="cuda").to(torch.bfloat16)
    clean, clean_l = run(c, [tokens], masks=[sees], q=q)
    j = keys - tokens + 7
    c.k[int(c.table[0, j // 16]), 0, j % 16, 5] = sign * float("inf")
    out, lse = run(c, [tokens], masks=[sees], q=q, check=False)
    # without that key at all, for the rows that get -inf
    hidden = sees.copy()
    hidden[:, 7] = False
    c.k[int(c.table[0, j // 16]), 0, j % 16, 5] = 0
    without, without_l = run(c, [tokens], masks=[hidden], q=q)
    G = heads // kv_heads
    for t in range(tokens):
        for h in range(heads):
            if not sees[t, 7] or h >= G:
                assert torch.equal(out[t, h], clean[t, h]) and lse[t, h] == clean_l[t, h]
            elif sign * float(q[t, h, 5]) > 0:
                assert out[t, h].isnan().all() and lse[t, h].isnan()
            else:
                assert torch.equal(out[t, h], without[t, h]) and lse[t, h] == without_l[t, h]
