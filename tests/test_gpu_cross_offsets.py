"""Cross attention with token offsets that the header rules out: out of order, negative, beyond the tokens.

The kernel clamps every sequence's tokens to those of the call, however the items are dealt.  What the results are is
not said; nothing outside of the outputs and the workspace is written, and what is written comes from a softmax.
"""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import Cache
from _support import need_gpu

pytestmark = pytest.mark.gpu

LOW, HIGH = -(1 << 31), (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Guarded:
    """A buffer of `numel` elements between two margins that must not change."""

    MARGIN = 1 << 16

    def __init__(self, numel, dtype, value):
        self.all = torch.full((numel + 2 * self.MARGIN,), 77, dtype=dtype, device="cuda")
        self.view = self.all[self.MARGIN:self.MARGIN + numel]
        self.view.fill_(value)

    def untouched(self):
        return bool((self.all[:self.MARGIN] == 77).all() and (self.all[-self.MARGIN:] == 77).all())


def run(desc, c, q, cu):
    n, heads = q.shape[:2]
    out, ls = Guarded(q.numel(), torch.bfloat16, 0), Guarded(n * heads, torch.float32, 0)
    size = skv.splitkv_cross_workspace_size(desc, n)
    ws = Guarded(max(size, 16), torch.uint8, 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.splitkv_cross_attend(desc, torch.tensor(cu, dtype=torch.int32, device="cuda"), q, c["k"], c["v"], c["table"], c["lens"],
                             0.1, out.view.view(q.shape), ls.view.view(n, heads), ws.view if size else None, status=status)
    assert status.item() == 0
    assert out.untouched() and ls.untouched() and ws.untouched()
    assert torch.isfinite(out.view).all() and out.view.abs().max() <= c["most"]
    assert not torch.isnan(ls.view).any()


def offsets(counts, n, rng):
    """The right ones, then wrong ones of every kind."""
    right = np.concatenate([[0], np.cumsum(counts)])
    yield right
    yield right[::-1].copy()
    yield rng.permutation(right)
    yield rng.integers(0, n + 1, len(right))
    yield rng.integers(-n, 2 * n, len(right))
    yield np.where(np.arange(len(right)) % 2, n, 0)         # every other sequence has all tokens
    yield np.where(np.arange(len(right)) % 2, LOW, n)
    yield np.where(np.arange(len(right)) % 2, HIGH, LOW)
    yield rng.choice([LOW, -1, 0, 1, n // 2, n - 1, n, n + 1, HIGH], len(right))


DEALS = {  # lengths, tokens, KV heads, query heads
    "pieces, few rows": ([2000, 50, 700], [1, 2, 1], 2, 4),
    "pieces, many rows": ([4000, 300], [150, 20], 1, 2),
    "pieces, many sequences": ([300, 900] * 25, [1, 40] * 25, 4, 8),
    "line of few items": ([1500] * 10, [1] * 10, 16, 16),
    "line": ([400, 0, 130] * 30, [1, 2, 0] * 30, 8, 16),
    "an item per CTA": ([300, 20] * 35, [60, 64] * 35, 8, 32),
}


@pytest.mark.parametrize("deal", DEALS)
def test_wrong_offsets_write_nothing_else(deal):
    lens, counts, kv, heads = DEALS[deal]
    c = Cache(lens, kv_heads=kv, heads=heads, device="cuda", seed=5)
    n = sum(counts)
    q = torch.randn((n, heads, 128), device="cuda").to(torch.bfloat16)
    state = dict(k=c.k, v=c.v, table=c.table, lens=c.lens, most=float(c.v.abs().max()))
    for cu in offsets(counts, n, np.random.default_rng(6)):
        run(c.desc, state, q, cu)


def test_more_pieces_than_32_bits_count():
    """One token, which the offsets give to every other one of 240,000 sequences of 608 heads: 2.3e9 pieces if each is cut
    into 32."""
    B, heads, P = 240000, 608, 4112  # 33 key blocks
    k = torch.randn((1, heads, P, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.rand((1, heads, P, 128), device="cuda").to(torch.bfloat16)
    state = dict(k=k, v=v, table=torch.zeros((B, 1), dtype=torch.int32, device="cuda"),
                 lens=torch.full((B,), P, dtype=torch.int32, device="cuda"), most=1.0)
    q = torch.randn((1, heads, 128), device="cuda").to(torch.bfloat16)
    run(skv.make_desc(B, 1, heads, heads, 128, 128, P, 1, 1), state, q, np.arange(B + 1) % 2)
