"""Cross attention where a key, a query or a value that is attended to is NaN or infinite.

The formula decides which results are NaN: a row whose scores hold NaN or +inf is NaN throughout, with its
log-sum-exp; a NaN value column is NaN in the rows of its KV head.  Every other row keeps the bits that it has
without them.  The same must come out however the call's items are dealt to the SMs: in whole items, cut into pieces
that are merged, in a line.
"""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import Cache
from _support import need_gpu

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
#: name: lengths, query tokens, KV heads, query heads
DEALS = {
    "cut, few rows": ([2000, 700], [1, 3], 1, 2),
    "cut, many rows": ([4000, 300], [150, 20], 1, 2),
    "one key block": ([100, 128], [1, 150], 2, 4),
    "whole, few rows": ([300] * 40, [1] * 40, 8, 8),
    "line of few items": ([1500] * 10, [1] * 10, 16, 16),
    "line": ([400] * 90, [1] * 90, 8, 16),
    "an item per CTA": ([300] * 70, [60] * 70, 8, 32),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def call(c, q, cu):
    n = q.shape[0]
    out, ls = torch.zeros_like(q), torch.zeros((n, c.heads), device="cuda")
    ws = torch.full((max(16, skv.splitkv_cross_workspace_size(c.desc, n)),), 255, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.splitkv_cross_attend(c.desc, cu, q, c.k, c.v, c.table, c.lens, 0.1, out, ls, ws, status=status)
    assert status.item() == 0
    return out, ls


def same_bits(a, b):
    kind = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


@pytest.mark.parametrize("where", ["key", "last key", "infinite key", "query", "value"])
@pytest.mark.parametrize("deal", DEALS)
def test_nan_stays(deal, where):
    lens, counts, kv, heads = DEALS[deal]
    c = Cache(lens, kv_heads=kv, heads=heads, device="cuda", seed=7)
    n, G = sum(counts), heads // kv
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn((n, heads, 128), generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    clean, clean_l = call(c, q, cu)
    assert torch.isfinite(clean).all() and torch.isfinite(clean_l).all()
    nan, nan_l = torch.zeros_like(clean, dtype=torch.bool), torch.zeros_like(clean_l, dtype=torch.bool)
    at = 0
    for b, (L, m) in enumerate(zip(lens, counts)):
        if b % 3 == 0:  # (other sequences stay as they are)
            h = b % kv
            heads_of = slice(h * G, (h + 1) * G)
            j = L - 1 if where == "last key" else L // 2
            page, row = int(c.table[b, j // 16]), j % 16
            if where in ("key", "last key"):
                c.k[page, h, row, 77] = NAN
                nan[at:at + m, heads_of] = nan_l[at:at + m, heads_of] = True
            elif where == "infinite key":
                c.k[page, h, row, 77] = INF
                hit = q[at:at + m, heads_of, 77] > 0  # a score of +inf; -inf weighs nothing
                nan_l[at:at + m, heads_of] |= hit
                nan[at:at + m, heads_of] |= hit[..., None]
            elif where == "query":
                q[at + m - 1, h * G, 5] = NAN
                nan[at + m - 1, h * G] = nan_l[at + m - 1, h * G] = True
            else:
                c.v[page, h, row, 9] = NAN
                nan[at:at + m, heads_of, 9] = True
        at += m
    out, ls = call(c, q, cu)
    assert torch.equal(torch.isnan(out), nan), "out"
    assert torch.equal(torch.isnan(ls), nan_l), "lse"
    if where != "infinite key":  # (whose other rows lose a key's weight)
        assert same_bits(out[~nan], clean[~nan]) and same_bits(ls[~nan_l], clean_l[~nan_l])
