"""GPU tests of append with norms: what is stored of values in e4m3, and rows that are not finite in long
calls.

A value's code is round(x / scale), the quotient rounded to fp32 first: both have one right result.
"""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import Cache
from _support import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def inputs(c, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, c.heads + 2 * c.Hkv, 128), generator=g, device="cuda")
    x = (x * torch.exp(3 * torch.randn((n, 1, 1), generator=g, device="cuda"))).to(torch.bfloat16)
    return x[:, :c.heads], x[:, c.heads:c.heads + c.Hkv], x[:, c.heads + c.Hkv:]


def call(c, q, k, v, counts, **kw):
    n = q.shape[0]
    out = torch.zeros((n, c.heads, 128), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    skv.splitkv_append_norm(c.desc, skv.splitkv_rope_create(128), pos, q, k, v, c.table, c.lens, out, c.k, c.v, cu_tokens=cu, **kw)
    torch.cuda.synchronize()
    return out


def stored(c, pool, counts):
    """What the pool holds of the new tokens, [n][Hkv][128]."""
    pool = pool if c.layout == "HND" else pool.transpose(1, 2)
    rows = []
    for b, m in enumerate(counts):
        j = torch.arange(c.lens_host[b] - m, c.lens_host[b], device="cuda")
        rows.append(pool[c.table[b].long()[j // c.P], :, j % c.P])
    return torch.cat(rows)


# (short calls; long ones, whose rows come through a ring)
@pytest.mark.parametrize("heads,kv_heads,counts", [(6, 2, [5, 0, 40]), (3, 1, [1]), (8, 4, [4300, 17]), (64, 8, [1, 900])])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("kv_scale", [0.25, 0.3, 2.0 ** -20, 1e-3, 7.0, None])
def test_values_in_e4m3(heads, kv_heads, counts, layout, kv_scale):
    c = Cache([m + 9 for m in counts], kv_heads=kv_heads, heads=heads, dtype="e4m3", layout=layout, device="cuda", seed=20)
    q, k, v = inputs(c, sum(counts), 21)
    if kv_scale is None:  # a scale for each head, keys' and values' apart; powers of two among them
        vs = torch.tensor([0.01, 0.5, 3.0, 2.0 ** -9, 0.125, 0.3, 1.0, 11.0][:kv_heads], device="cuda")
        call(c, q, k, v, counts, k_scale=torch.full_like(vs, 0.02), v_scale=vs)
    else:
        vs = torch.full((kv_heads,), kv_scale, device="cuda")
        call(c, q, k, v, counts, kv_scale=kv_scale)
    want = (v.float() / vs[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(stored(c, c.v, counts), want)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_row_that_is_not_finite_spoils_no_other_in_a_ring(dtype, bad):
    n = 5500
    c = Cache([n + 3], kv_heads=4, heads=8, dtype=dtype, device="cuda", seed=22)
    q, k, v = (x.contiguous() for x in inputs(c, n, 23))
    first = call(c, q, k, v, [n]), stored(c, c.k, [n]), stored(c, c.v, [n])
    rows = [(0, 0), (3, 3), (1717, 2), (n - 1, 1)]
    for t, h in rows:
        q[t, 2 * h, 17 * h] = k[t, h, 5] = bad
    out, keys, values = call(c, q, k, v, [n]), stored(c, c.k, [n]), stored(c, c.v, [n])
    good_q, good_k = torch.ones((n, 8), dtype=torch.bool, device="cuda"), torch.ones((n, 4), dtype=torch.bool, device="cuda")
    for t, h in rows:
        good_q[t, 2 * h] = good_k[t, h] = False
        assert out[t, 2 * h].isnan().any()
        key = keys[t, h].view(torch.float8_e4m3fn).float() if dtype == "e4m3" else keys[t, h]
        assert key.isnan().any()
    assert torch.equal(out[good_q], first[0][good_q]) and torch.equal(keys[good_k], first[1][good_k])
    assert torch.equal(values, first[2])
