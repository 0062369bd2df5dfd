"""GPU tests of trees over e4m3 caches whose keys have a small share of the weight each: one key (a sink at the
sequence's start) takes nearly all of it, and the values of the many others are what comes out.

Tolerances.  As in the tests of tree attention, but for the weights that are multiplied with V: they are f16 times 2^7
where the largest of a piece's first keys is 1, so that their steps of 2^-24 below 2^-14 are off by half of one, 2^-32 of
that: n_keys * 2^-32 * max |V| at most, beside 2^-11 (here 2^-8 is allowed) of each.
"""
import numpy as np
import pytest
import torch

from _cache_ops import EPS16, Cache
from _support import need_gpu
from test_gpu_tree import latent, run

pytestmark = pytest.mark.gpu
KV_SCALE = 1 / 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def codes(x):
    return (x / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def check(c, counts, q, out, lse):
    """Chains of drafted tokens against 64 bits."""
    got, got_l, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    kp, vp = c.values(c.k), None if c.shares else c.values(c.v)
    G, at, scale = c.heads // c.Hkv, 0, c.dim ** -0.5
    for b, m in enumerate(counts):
        L = c.lens_host[b]
        k = c.rows(kp, b, L) * KV_SCALE
        v = k[..., :c.v_dim] if c.shares else c.rows(vp, b, L) * KV_SCALE
        seen = np.arange(L)[None] <= np.arange(L - m, L)[:, None]
        for h in range(c.heads):
            qs, kh, vh = q64[at:at + m, h], k[:, h // G], v[:, h // G]
            x = np.where(seen, qs @ kh.T * scale, -np.inf)
            e = c.dim * 2.0 ** -23 * (np.abs(qs) @ np.abs(kh).T * scale).max() + 2.0 ** -22 * np.abs(np.where(seen, x, 0)).max()
            if c.dim == 128:
                most = np.abs(qs).max(1)[:, None]
                e += 2.0 ** -16 * scale * (most * ((np.abs(qs) < 2.0 ** -9 * most) @ np.abs(kh).T)).max()
            top = x.max(1, keepdims=True)
            z = top + np.log(np.exp(x - top).sum(1, keepdims=True))
            p = np.exp(x - z)
            want, size = p @ vh, p @ np.abs(vh)
            tol = (2.0 ** -8 + 2 * e) * size + EPS16 * np.abs(want) + L * 2.0 ** -32 * np.abs(vh).max()
            d = np.abs(got[at:at + m, h] - want)
            assert (d <= tol).all(), (b, h, float((d / tol).max()), float(np.abs(want).mean()))
            assert np.abs(want).mean() > 4 * tol.mean()  # (the others' share is seen)
            assert (np.abs(got_l[at:at + m, h] - z[:, 0]) <= e + 2.0 ** -20 * (1 + np.abs(z[:, 0]))).all()
        at += m


def sink(c, counts, share, seed):
    """Each sequence's first key is a sink: 16 columns that no other key has, and no value.  Returns queries whose other
    keys have 2^share of its weight each, about."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    first = 512 if c.dim == 576 else 0  # of the columns: behind the values
    k = 0.2 * torch.randn(c.k.shape, generator=g, device="cuda")
    k[..., first:first + 16] = 0
    v = k if c.shares else torch.empty(c.v.shape, device="cuda")
    v[..., :c.v_dim] = 1 + 0.25 * torch.randn(v[..., :c.v_dim].shape, generator=g, device="cuda")
    for b in range(c.B):
        page = int(c.table[b, 0])
        k[page, :, 0] = 0
        k[page, :, 0, first:first + 16] = 4
        v[page, :, 0, :512] = 0
    c.k.copy_(codes(k))
    if not c.shares:
        c.v.copy_(codes(v))
    q = torch.randn((sum(counts), c.heads, c.dim), generator=g, device="cuda")
    if first:
        q[..., :512] *= 0.02
    q[..., first:first + 16] = -share * np.log(2) / (16 * 4 * c.dim ** -0.5)
    return q.to(torch.bfloat16)


SHARES = pytest.mark.parametrize("share", [-20, -24, -27])


@SHARES
@pytest.mark.parametrize("batch,tokens,heads,kv_heads,keys", [(20, 40, 64, 16, 500), (40, 9, 64, 16, 400), (12, 5, 8, 8, 260),
                                                              (1, 7, 4, 1, 900), (90, 2, 8, 8, 400)])
def test_a_sink_and_a_long_tail(batch, tokens, heads, kv_heads, keys, share):
    """Items of 160 rows, of 36 (a CTA each), of a few (a piece each, cut, and in a line)."""
    counts = [tokens] * batch
    c = Cache([keys - 3 * (b % 7) for b in range(batch)], kv_heads=kv_heads, heads=heads, dtype="e4m3", device="cuda", seed=70)
    q = sink(c, counts, share, 71)
    out, lse = run(c, counts, masks=[np.tri(n, dtype=bool) for n in counts], q=q, check=False)
    check(c, counts, q, out, lse)


@SHARES
@pytest.mark.parametrize("batch,tokens,page", [(4, 3, 64), (2, 16, 32)])
def test_a_sink_and_a_long_tail_of_latent_rows(batch, tokens, page, share):
    counts = [tokens] * batch
    c = latent([600 - 3 * b for b in range(batch)], tokens, page, "e4m3", seed=72)
    q = sink(c, counts, share, 73)
    out, lse = run(c, counts, masks=[np.tri(n, dtype=bool) for n in counts], q=q, cu=False, check=False)
    check(c, counts, q, out, lse)
