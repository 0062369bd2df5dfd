"""GPU tests of tree attention against a plain 64-bit implementation.

Tolerances.  A score is a sum of fp32 additions of exact products, off by at most e = D * 2^-23 * sum |q_d K_d| * scale for
rows of D (the tensor cores may truncate).  Over e4m3 caches a query component times a power of two, the row's largest in
[2^7, 2^8), is the sum of two e4m3 codes: its four leading bits, and the rest, of four bits too.  Both are exact from 2^-2
on, as codes have steps of 2^-9 and less; below, each is off by half such a step, so that components below 2^-9 of the
row's largest are off by 2^-16 of it, and e has 2^-16 * max |q| * sum |K_d| over those d besides.  A score's exponent's argument rounds a few times more at its size; a weight is off by that factor, and by 2^-8
where it is rounded to bf16 for the product with V (f16: 2^-11, and 2^-25 of a piece's largest weight below 2^-14).  With
A = sum_j p_j |V_j| the output is off by at most (2^-8 + 2 e) A, in f16 by n_keys * 2^-25 * max |V| too, and by half a step of
bf16, 2^-8 |out|, where it is rounded itself.  The log-sum-exp is off by e and a few roundings of fp32 at its size.
"""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import EPS16, Cache
from _support import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def tree(rng, n, near=9):
    """[n][n]: which tokens a token of a random tree sees."""
    sees = np.zeros((n, n), bool)
    for i in range(n):
        if i:
            p = int(rng.integers(max(0, i - near), i))
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


def words(sees, n_words, spare_bits=False):
    """The masks as int32 [n][n_words]; bits of tokens that there are not are set with `spare_bits`."""
    n = sees.shape[0]
    bits = np.full((n, 32 * n_words), spare_bits, bool)
    m = min(n, 32 * n_words)
    bits[:, :m] = sees[:, :m]
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32).reshape(n, n_words)


def run(c, counts, masks=None, n_words=None, pad=0, before=0, cu=True, stride=0, std=1.0, seed=41, status=0, lse=True, check=True,
        kv_scale=None, scales=None, spare_bits=False, q=None, lens=None, graph=False):
    rng = np.random.default_rng(seed)
    masks = [tree(rng, n) for n in counts] if masks is None else masks
    n_words = n_words or max(1, -(-max(counts) // 32))
    n = before + sum(counts) + pad
    fp8 = c.dtype == "e4m3"
    kv_scale = (1 / 64 if fp8 else 1.0) if kv_scale is None else kv_scale
    g = torch.Generator(device="cuda").manual_seed(seed)
    if q is None:
        wide = torch.randn((n, c.heads * c.dim + stride), generator=g, device="cuda") * std
        q = wide.to(torch.bfloat16)[:, :c.heads * c.dim].view(n, c.heads, c.dim)
    mask = np.full((n, n_words), -1, np.int32)
    at = before
    for m in masks:
        mask[at:at + len(m)] = words(m, n_words, spare_bits)
        at += len(m)
    mask = torch.from_numpy(mask).cuda()
    out = torch.full((n, c.heads, c.v_dim), 9.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((n, c.heads), 9.0, device="cuda")
    size = skv.splitkv_tree_workspace_size(c.desc, n)
    ws = torch.full((max(16, size),), 255, dtype=torch.uint8, device="cuda")  # NaN
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cut = torch.tensor(before + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    scale = c.dim ** -0.5
    ks, vs = (None, None) if scales is None else (torch.tensor(x, dtype=torch.float32, device="cuda") for x in scales)

    def call():
        skv.splitkv_tree_attend(c.desc, cut if cu else None, mask, q, c.k, c.v, c.table, c.lens, scale, out, ls if lse else None,
                                ws, kv_scale=kv_scale, k_scale=ks, v_scale=vs, status=st)

    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            call()
        captured.replay()
    else:
        call()
    torch.cuda.synchronize()
    assert int(st) == status
    if not check:
        return out, ls
    got, got_l, q64 = out.double().cpu().numpy(), ls.double().cpu().numpy(), q.double().cpu().numpy()
    kp, vp = c.values(c.k), None if c.shares else c.values(c.v)
    G, at = c.heads // c.Hkv, before
    lens = c.lens_host if lens is None else lens
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for b, m in enumerate(counts):
            L = lens[b]
            k = c.rows(kp, b, L)
            v = k[..., :c.v_dim] if c.shares else c.rows(vp, b, L)
            seen = np.concatenate([np.ones((m, L - m), bool), masks[b][:, :m] & (np.arange(m) < 32 * n_words)], 1) if L else None
            for h in range(c.heads):
                if L == 0:
                    assert (got[at:at + m, h] == 0).all() and (not lse or (got_l[at:at + m, h] == -np.inf).all())
                    continue
                kh = k[:, h // G] * (np.float32(scales[0][h // G]) if scales else kv_scale)
                vh = v[:, h // G] * (np.float32(scales[1][h // G]) if scales else kv_scale)
                used = seen.any(0)  # (what no token sees may hold anything)
                kh, vh = np.where(used[:, None], kh, 0), np.where(used[:, None], vh, 0)
                qs = q64[at:at + m, h]
                x = np.where(seen, qs @ kh.T * scale, -np.inf)
                top = np.where(seen, x, 0)
                e = (c.dim * 2.0 ** -23 * (np.abs(qs) @ np.abs(kh).T * scale).max(initial=0) +
                     4 * 2.0 ** -24 * np.abs(top).max(initial=0))
                if fp8 and c.dim == 128:
                    most = np.abs(qs).max(1, initial=0)[:, None]
                    e += 2.0 ** -16 * scale * (most * ((np.abs(qs) < 2.0 ** -9 * most) @ np.abs(kh).T)).max(initial=0)
                peak = x.max(1, initial=-np.inf)
                empty = peak == -np.inf
                z = np.where(empty, -np.inf, np.where(empty, 0, peak) + np.log(np.exp(x - np.where(empty, 0, peak)[:, None]).sum(1)))
                p = np.where(empty[:, None], 0, np.exp(x - np.where(empty, 0, z)[:, None]))
                want, size = p @ vh, p @ np.abs(vh)
                tol = (2.0 ** -8 + 2 * e) * size + EPS16 * np.abs(want) + 1e-30
                if fp8:
                    tol = tol + L * 2.0 ** -25 * np.abs(vh).max()
                d = np.abs(got[at:at + m, h] - want)
                assert (d <= tol).all(), (b, h, float(np.nanmax(d)), float(np.nanmax(d / tol)))
                if lse:
                    assert ((got_l[at:at + m, h] == -np.inf) == empty).all()
                    dl = np.abs(got_l[at:at + m, h] - z)[~empty]
                    assert (dl <= e + 2.0 ** -20 * (1 + np.abs(z[~empty]))).all(), (b, h, float(dl.max()))
                assert (got[at:at + m, h][empty] == 0).all()
            at += m
    for x in (got, got_l) if lse else (got,):
        assert (x[:before] == 9).all() and (x[at:] == 9).all()  # tokens of no sequence
    return out, ls


both = pytest.mark.parametrize("dtype", ["bf16", "e4m3"])


@both
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_ragged_trees(dtype, layout, page):
    c = Cache([300, 5, 40, 128, 700, 77, 0], kv_heads=2, heads=8, page=page, dtype=dtype, layout=layout, device="cuda", seed=42)
    run(c, [40, 0, 3, 33, 1, 64, 4], pad=3, before=2)


@both
@pytest.mark.parametrize("context", [0, 1, 31, 100, 127, 128, 129, 250])
@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 64])
def test_where_the_drafted_keys_lie(dtype, context, tokens):
    """Their first key at every kind of place in a key block, with and without keys before them."""
    c = Cache([context + tokens], kv_heads=1, heads=4, dtype=dtype, device="cuda", seed=43)
    run(c, [tokens])


@both
@pytest.mark.parametrize("tokens,n_words", [(130, 5), (200, 7), (300, 10), (300, 4), (97, 32), (60, 1)])
def test_long_and_short_masks(dtype, tokens, n_words):
    """Trees over several key blocks; masks of fewer bits than tokens, and of more."""
    c = Cache([tokens + 70, tokens], kv_heads=1, heads=2, dtype=dtype, device="cuda", seed=44)
    run(c, [tokens, tokens], n_words=n_words, spare_bits=True)


@both
def test_masks_that_are_no_trees(dtype):
    """Random ones, none at all (with keys before: those alone; without: empty rows), and everything."""
    rng = np.random.default_rng(45)
    n = 45
    masks = [rng.random((n, n)) < 0.3, np.zeros((n, n), bool), np.zeros((n, n), bool), np.ones((n, n), bool), np.tri(n, dtype=bool)]
    c = Cache([n + 200, n + 90, n, n, n + 1], kv_heads=2, heads=6, dtype=dtype, device="cuda", seed=45)
    run(c, [n] * 5, masks=masks)


@both
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 1), (8, 8), (64, 2), (300, 1)])
def test_shared_heads(dtype, heads, kv_heads):
    c = Cache([260, 40], kv_heads=kv_heads, heads=heads, dtype=dtype, device="cuda", seed=46)
    run(c, [9, 21])


@both
def test_many_rows_and_keys(dtype):
    c = Cache([3000, 1111], kv_heads=2, heads=16, page=64, dtype=dtype, device="cuda", seed=47)
    run(c, [120, 37], stride=256)


@both
@pytest.mark.parametrize("cap_pages", [2, 9, 100, 3000])
def test_splits_by_capacity(cap_pages, dtype):
    lens = [min(cap_pages * 16, x) for x in (16, 130, 1500)]
    c = Cache(lens, kv_heads=1, heads=2, cap_pages=cap_pages, dtype=dtype, device="cuda", seed=48)
    run(c, [1, 16, 10])


@both
def test_many_sequences(dtype):
    """As a line that the CTAs share (few rows a sequence), and a CTA for each item."""
    rng = np.random.default_rng(49)
    counts = [int(x) for x in rng.integers(0, 5, 90)]
    lens = [n + int(x) for n, x in zip(counts, rng.integers(0, 300, 90))]
    c = Cache(lens, kv_heads=8, heads=8, dtype=dtype, device="cuda", seed=49)
    run(c, counts)
    counts = [int(x) for x in rng.integers(20, 64, 40)]
    lens = [n + int(x) for n, x in zip(counts, rng.integers(0, 200, 40))]
    run(Cache(lens, kv_heads=4, heads=32, dtype=dtype, device="cuda", seed=49), counts)
    c = Cache(lens, kv_heads=16, heads=64, dtype=dtype, device="cuda", seed=49)
    assert skv.splitkv_tree_workspace_size(c.desc, sum(counts)) == 0
    run(c, counts)


@both
def test_tokens_without_cu_and_without_lse(dtype):
    c = Cache([150, 40, 0], tokens=5, dtype=dtype, device="cuda", seed=50)
    run(c, [5, 5, 5], cu=False)
    run(c, [5, 5, 5], lse=False)
    run(c, [5, 5, 5], cu=False, graph=True)


@both
@pytest.mark.parametrize("std", [1e-6, 1e-3, 30.0, 1000.0])
def test_flat_and_sharp_scores(std, dtype):
    c = Cache([500], kv_heads=1, heads=2, dtype=dtype, device="cuda", seed=51)
    run(c, [70], std=std)
    run(c, [60], std=std, masks=[np.tri(60, dtype=bool)])


def test_query_rows_of_unlike_sizes():
    """e4m3: each row's power of two is its own; components far below the row's largest, and rows of zeros."""
    c = Cache([300, 200], kv_heads=2, heads=10, dtype="e4m3", device="cuda", seed=52)
    g = torch.Generator(device="cuda").manual_seed(53)
    for counts in ([20, 9], [60, 40]):
        q = torch.randn((sum(counts), 10, 128), generator=g, device="cuda")
        q *= torch.exp(6 * torch.randn((sum(counts), 10, 1), generator=g, device="cuda")).clamp(max=300)
        q *= torch.exp(-3 * torch.rand((1, 1, 128), generator=g, device="cuda"))
        q[3, 2] = 0
        run(c, counts, q=q.to(torch.bfloat16))


def test_scales_of_heads():
    c = Cache([300, 60], kv_heads=3, heads=6, dtype="e4m3", device="cuda", seed=54)
    run(c, [30, 5], scales=([0.01, 0.03, 0.002], [0.5, 0.01, 2.0]))


@both
def test_what_no_token_sees_may_hold_anything(dtype):
    """NaN behind the length, in pages of no sequence, and in padding of the trees: queries whose keys no other sees."""
    counts = [20, 7, 66]
    rng = np.random.default_rng(55)
    masks = [tree(rng, n) for n in counts]
    spare = [[5, 6, 19], [0], list(range(40, 66))]
    for m, ids in zip(masks, spare):
        m[:, ids] = False
    c = Cache([150, 90, 130], kv_heads=2, heads=8, page=64, dtype=dtype, device="cuda", seed=55)
    first = run(c, counts, masks=masks)
    t = c.table.cpu().numpy()
    nan = 127 if dtype == "e4m3" else float("nan")
    for pool in (c.k, c.v):
        for b, L in enumerate(c.lens_host):
            if L % 64:
                pool[t[b, L // 64], :, L % 64:] = nan
            for i in spare[b]:
                j = L - counts[b] + i
                pool[t[b, j // 64], :, j % 64] = nan
    used = {int(t[b, i]) for b, L in enumerate(c.lens_host) for i in range(-(-L // 64))}
    for page in set(range(c.N)) - used:
        c.k[page] = c.v[page] = nan
    again = run(c, counts, masks=masks, check=False)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@both
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_a_key_that_is_not_finite_reaches_those_that_see_it(dtype, bad):
    if dtype == "e4m3" and bad == "inf":
        pytest.skip("e4m3 has no infinity")
    c = Cache([90], kv_heads=1, heads=4, dtype=dtype, device="cuda", seed=56)
    sees = tree(np.random.default_rng(56), 30)
    first = run(c, [30], masks=[sees])
    j = 60 + 7
    c.k[int(c.table[0, j // 16]), 0, j % 16] = 127 if dtype == "e4m3" else float(bad)
    out, lse = run(c, [30], masks=[sees], check=False)
    for i in range(30):
        if sees[i, 7]:
            assert bad == "inf" or (out[i].isnan().all() and lse[i].isnan().all())
        else:
            assert torch.equal(out[i], first[0][i]) and torch.equal(lse[i], first[1][i])


def test_lengths_and_pages_are_reported():
    for dtype in ("bf16", "e4m3"):
        c = Cache([60, 40, 30, 200], dtype=dtype, device="cuda", seed=57)
        c.lens[0] = 9           # fewer keys than tokens
        c.lens[1] = c.cap + 1
        c.lens[2] = -1
        run(c, [10, 10, 10, 10], lens=[0, 0, 0, 200], status=skv.SPLITKV_DEVERR_SEQLEN)
        c.table[3, 2] = c.N
        c.table[3, 5] = -1
        want = c.table.clone()
        out, lse = run(c, [10, 10, 10, 10], status=skv.SPLITKV_DEVERR_SEQLEN | skv.SPLITKV_DEVERR_PAGE, check=False)
        want[3, 2] = want[3, 5] = 0
        c.table = want
        again = run(c, [10, 10, 10, 10], lens=[0, 0, 0, 200], status=skv.SPLITKV_DEVERR_SEQLEN)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


# ------------------------------------------------------------------ latent rows

def latent(lens, tokens, page=64, dtype="bf16", shares=True, seed=0, **kw):
    return Cache(lens, kv_heads=1, heads=128, page=page, dim=576, v_dim=512, shares=shares, dtype=dtype, tokens=tokens,
                 device="cuda", seed=seed, std=0.5, **kw)


@pytest.mark.parametrize("dtype,shares", [("bf16", True), ("bf16", False), ("e4m3", True)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens", [1, 7, 16])
def test_latent_trees(dtype, shares, page, tokens):
    c = latent([300, 0, tokens, 64 + tokens // 2 + 1], tokens, page, dtype, shares, seed=60)
    run(c, [tokens] * 4, cu=False)


@pytest.mark.parametrize("dtype,shares", [("bf16", True), ("bf16", False), ("e4m3", True)])
@pytest.mark.parametrize("page", [32, 64])
def test_latent_masks(dtype, shares, page):
    """Everything, nothing (an empty row without keys before), random ones, bits behind the tokens, two words."""
    rng = np.random.default_rng(61)
    n = 11
    masks = [np.ones((n, n), bool), np.zeros((n, n), bool), np.zeros((n, n), bool), rng.random((n, n)) < 0.4]
    c = latent([200, 130, n, 65], n, page, dtype, shares, seed=61)
    run(c, [n] * 4, masks=masks, cu=False, spare_bits=True, n_words=2)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shares", [True, False])
def test_latent_keys_that_a_token_does_not_see_may_hold_anything(dtype, shares):
    if dtype == "e4m3" and not shares:
        pytest.skip("no such cache")
    c = latent([100], 8, 64, dtype, shares, seed=62)
    sees = tree(np.random.default_rng(62), 8)
    first = run(c, [8], masks=[sees], cu=False)
    j = 92 + 5
    for pool in (c.k,) if shares else (c.k, c.v):
        pool[int(c.table[0, j // 64]), 0, j % 64] = 127 if dtype == "e4m3" else float("nan")
    out, lse = run(c, [8], masks=[sees], cu=False, check=False)
    for i in range(8):
        assert (torch.equal(out[i], first[0][i]) and torch.equal(lse[i], first[1][i])) or (sees[i, 5] and out[i].isnan().any())


def test_latent_splits_and_reports():
    c = latent([1500, 700], 5, 64, seed=63, cap_pages=64)
    assert skv.splitkv_tree_workspace_size(c.desc, 10) > 2 * 5 * 128 * 512 * 4  # several splits
    run(c, [5, 5], cu=False)
    run(c, [5, 5], cu=False, graph=True)
    c.lens[1] = 4
    run(c, [5, 5], cu=False, lens=[1500, 0], status=skv.SPLITKV_DEVERR_SEQLEN)
