"""GPU tests of cross attention against a plain 64-bit implementation.

Tolerances.  A score is a sum of 128 fp32 additions of exact products, off by at most e = 128 * 2^-23 * sum
|q_d K_d| * scale (the tensor cores may truncate), and its exponent's argument rounds twice more at its size; a
weight is off by that factor, and by 2^-8 where it is rounded to bf16 for the product with V.  With A = sum_j p_j
|V_j| the output is off by at most (2^-8 + 2 e) A, and by half a step of bf16, 2^-8 |out|, where it is rounded
itself.  The log-sum-exp is off by e and a few roundings of fp32 at its size.
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


def run(c, counts, pad=0, before=0, cu=True, stride=0, std=1.0, seed=41, status=0, lse=True, check=True):
    n = before + sum(counts) + pad
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.randn((n, c.heads * 128 + stride), generator=g, device="cuda") * std
    q = wide.to(torch.bfloat16)[:, :c.heads * 128].view(n, c.heads, 128)
    out = torch.full((n, c.heads, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((n, c.heads), 9.0, device="cuda")
    ws = torch.full((max(16, skv.splitkv_cross_workspace_size(c.desc, n)),), 255, dtype=torch.uint8, device="cuda")  # NaN
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cut = torch.tensor(before + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    scale = 128 ** -0.5
    skv.splitkv_cross_attend(c.desc, cut if cu else None, q, c.k, c.v, c.table, c.lens, scale, out, ls if lse else None, ws,
                             status=st)
    torch.cuda.synchronize()
    assert int(st) == status
    if not check:
        return out, ls
    got, got_l, q64 = out.double().cpu().numpy(), ls.double().cpu().numpy(), q.double().cpu().numpy()
    kp, vp = c.values(c.k), c.values(c.v)
    G, at = c.heads // c.Hkv, before
    for b, m in enumerate(counts):
        L = c.lens_host[b]
        k, v = c.rows(kp, b, L), c.rows(vp, b, L)
        for h in range(c.heads):
            qs = q64[at:at + m, h]
            if L == 0:
                assert (got[at:at + m, h] == 0).all() and (not lse or (got_l[at:at + m, h] == -np.inf).all())
                continue
            x = qs @ k[:, h // G].T * scale
            e = 128 * 2.0 ** -23 * (np.abs(qs) @ np.abs(k[:, h // G]).T * scale).max(initial=0) + 4 * 2.0 ** -24 * np.abs(x).max(initial=0)
            z = x.max(1, initial=-np.inf) + np.log(np.exp(x - x.max(1, initial=-np.inf)[:, None]).sum(1))
            p = np.exp(x - z[:, None])
            want, size = p @ v[:, h // G], p @ np.abs(v[:, h // G])
            tol = (2.0 ** -8 + 2 * e) * size + EPS16 * np.abs(want) + 1e-30
            d = np.abs(got[at:at + m, h] - want)
            assert (d <= tol).all(), (b, h, float(d.max()), float((d / tol).max()))
            if lse:
                dl = np.abs(got_l[at:at + m, h] - z)
                assert (dl <= e + 2.0 ** -20 * (1 + np.abs(z))).all(), (b, h, float(dl.max()))
        at += m
    for x in (got, got_l) if lse else (got,):
        assert (x[:before] == 9).all() and (x[at:] == 9).all()  # tokens of no sequence
    return out, ls


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_one_token(layout, page):
    c = Cache([1, 127, 128, 129, 1000, 0], kv_heads=2, heads=6, page=page, layout=layout, device="cuda", seed=42)
    run(c, [1] * 6)


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("page", [16, 32, 96, 128])
def test_ragged_prompts(layout, page):
    c = Cache([300, 5, 0, 128, 700, 77], kv_heads=2, heads=16, page=page, layout=layout, device="cuda", seed=43)
    run(c, [40, 0, 3, 33, 1, 100], pad=3, before=2)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (8, 8), (130, 2), (600, 1)])
def test_shared_heads(heads, kv_heads):
    c = Cache([260, 40], kv_heads=kv_heads, heads=heads, device="cuda", seed=44)
    run(c, [3, 5])


def test_many_tokens_and_keys():
    c = Cache([2000, 1111], kv_heads=1, heads=4, page=64, device="cuda", seed=45)
    run(c, [700, 350], stride=256)


@pytest.mark.parametrize("cap_pages", [1, 9, 100, 3000])
def test_splits_by_capacity(cap_pages):
    """The split count goes by the capacity, the key ranges by the device lengths: parts without keys."""
    lens = [min(cap_pages * 16, x) for x in (16, 130, 1500)]
    c = Cache(lens, kv_heads=1, heads=2, cap_pages=cap_pages, device="cuda", seed=46)
    run(c, [1, 2, 1])


def test_tokens_without_cu_and_without_lse():
    c = Cache([150, 40, 0], tokens=5, device="cuda", seed=47)
    run(c, [5, 5, 5], cu=False)
    run(c, [5, 5, 5], lse=False)


@pytest.mark.parametrize("std", [1e-3, 30.0, 1000.0])
def test_flat_and_sharp_scores(std):
    c = Cache([500], kv_heads=1, heads=2, device="cuda", seed=48)
    run(c, [130], std=std)


def test_growing_scores_rescale():
    """Every key block's scores exceed the ones before by far more than 2^8."""
    c = Cache([1024], kv_heads=1, heads=1, device="cuda", seed=49)
    t = c.table.cpu().numpy()[0]
    ramp = torch.linspace(0.0, 3.0, 1024)
    for j in range(1024):
        c.k[t[j // 16], 0, j % 16] = (ramp[j] * torch.ones(128)).to(torch.bfloat16).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    c.k += torch.randn(c.k.shape, generator=g, device="cuda").to(torch.bfloat16) * 0.1
    run(c, [64], std=4.0)


def test_what_lies_behind_the_length_is_not_read():
    c = Cache([21, 130, 250], kv_heads=2, page=64, device="cuda", seed=50)
    first = run(c, [2, 1, 40])
    t = c.table.cpu().numpy()
    for pool in (c.k, c.v):
        for b, L in enumerate(c.lens_host):
            if L % 64:
                pool[t[b, L // 64], :, L % 64:] = float("nan")
    used = {int(t[b, i]) for b, L in enumerate(c.lens_host) for i in range(-(-L // 64))}
    for page in set(range(c.N)) - used:
        c.k[page] = c.v[page] = float("nan")
    again = run(c, [2, 1, 40], check=False)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_order_of_runs_does_not_matter():
    c = Cache([3000, 200], kv_heads=2, heads=8, device="cuda", seed=51)
    a, b = run(c, [1, 1], check=False), run(c, [1, 1], check=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_reports_lengths_and_pages():
    c = Cache([100, 100, 100], device="cuda", seed=52)
    c.lens.copy_(torch.tensor([-1, c.cap + 1, 100]))
    out, ls = run(c, [2, 2, 2], status=skv.SPLITKV_DEVERR_SEQLEN, check=False)
    assert (out[:4] == 0).all() and (ls[:4] == -float("inf")).all() and torch.isfinite(out[4:]).all()
    c.lens.fill_(100)
    c.table[1, 3] = c.N
    run(c, [2, 2, 2], status=skv.SPLITKV_DEVERR_PAGE, check=False)


def test_bad_token_offsets_stay_in_bounds():
    c = Cache([50, 60], device="cuda", seed=53)
    q = torch.randn((6, c.heads, 128), device="cuda").to(torch.bfloat16)
    for cut in ([0, 9, 6], [-4, 3, 6], [5, 2, 6], [7, 8, 9]):
        out, ls = torch.zeros_like(q), torch.zeros((6, c.heads), device="cuda")
        ws = torch.zeros(max(16, skv.splitkv_cross_workspace_size(c.desc, 6)), dtype=torch.uint8, device="cuda")
        skv.splitkv_cross_attend(c.desc, torch.tensor(cut, dtype=torch.int32, device="cuda"), q, c.k, c.v, c.table, c.lens, 0.1,
                                 out, ls, ws)
    torch.cuda.synchronize()


def test_captured_calls_follow_the_device_lengths():
    c = Cache([500, 500], cap_pages=40, device="cuda", seed=54)
    q = torch.zeros((8, c.heads, 128), dtype=torch.bfloat16, device="cuda")
    cu, lens = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"), c.lens.clone()
    out, ls = torch.zeros_like(q), torch.zeros((8, c.heads), device="cuda")
    ws = torch.zeros(max(16, skv.splitkv_cross_workspace_size(c.desc, 8)), dtype=torch.uint8, device="cuda")

    def call():
        skv.splitkv_cross_attend(c.desc, cu, q, c.k, c.v, c.table, lens, 0.1, out, ls, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for trial, (cut, ln) in enumerate([([0, 4, 8], [500, 3]), ([0, 0, 8], [1, 129]), ([1, 7, 7], [0, 500])]):
        g = torch.Generator(device="cuda").manual_seed(trial)
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        cu.copy_(torch.tensor(cut))
        lens.copy_(torch.tensor(ln))
        results = []
        for go in (graph.replay, call):
            out.fill_(3)
            ls.fill_(3)
            go()
            torch.cuda.synchronize()
            results.append((out.clone(), ls.clone()))
        assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
        assert (results[0][0][:cut[0]] == 3).all() and (results[0][0][cut[2]:] == 3).all()


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_several_items_per_cta(seed):
    """Between one and four items per SM, of all kinds in a row: one row and hundreds, no key, one block, many."""
    rng = np.random.default_rng(seed)
    B = 50
    lens = [int(x) for x in rng.choice([0, 1, 100, 128, 129, 257, 400, 900], B)]
    counts = [int(x) for x in rng.choice([0, 1, 2, 40, 64, 70, 140], B)]
    c = Cache(lens, kv_heads=4, heads=8, device="cuda", seed=55 + seed)
    run(c, counts)


@pytest.mark.parametrize("keys", [1, 128, 129, 256, 257, 1000, 5000])
@pytest.mark.parametrize("tokens", [1, 64, 65])
def test_one_head(keys, tokens):
    """A single item: up to 128 rows its key blocks go to both row blocks in turn, cut or not."""
    c = Cache([keys], kv_heads=1, heads=2, page=32, device="cuda", seed=59)
    run(c, [tokens])


@pytest.mark.parametrize("batch,kv_heads,heads,tokens", [(10, 16, 16, 1), (12, 16, 32, 3), (170, 1, 1, 1), (21, 8, 64, 8)])
def test_slightly_more_items_than_sms(batch, kv_heads, heads, tokens):
    """Items of like lengths that would leave the last round of CTAs nearly empty: cut anywhere, pieces of several
    items in a CTA."""
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(900, 1700, batch)]
    counts = [int(x) for x in rng.integers(1, tokens + 1, batch)]
    c = Cache(lens, kv_heads=kv_heads, heads=heads, device="cuda", seed=70 + batch)
    run(c, counts)
    c.lens_host = [min(x, -(-y // c.P) * c.P) for x, y in zip(lens[::-1], lens)]
    c.lens.copy_(torch.tensor(c.lens_host))
    run(c, counts, pad=3, before=2)


@pytest.mark.parametrize("seed", [1, 2])
def test_many_items_of_few_rows(seed):
    """More than four items per SM, of half a row tile on average: dealt as a line, cut at the CTAs' bounds; lengths,
    tokens and empty sequences of all kinds, more than 32 sequences, some of several row tiles."""
    rng = np.random.default_rng(seed)
    B = 90
    lens = [int(x) for x in rng.choice([0, 1, 100, 128, 129, 257, 400, 700], B)]
    counts = [int(x) for x in rng.choice([0, 1, 2, 9, 40, 65], B, p=[.2, .4, .2, .1, .05, .05])]
    counts[7] = 150
    c = Cache(lens, kv_heads=8, heads=32, device="cuda", seed=80 + seed)
    assert sum(counts) * 4 <= 128 * B and (sum(counts) * 4 // 256 + B) * 8 > 4 * 152
    run(c, counts, before=2, pad=1)


def test_many_items_but_few_tokens():
    """The bound on the items is high, most sequences have no token: fewer key blocks than SMs in the line."""
    B = 100
    counts = [0] * B
    counts[3], counts[50], counts[97] = 1, 90, 9
    lens = [40] * B
    lens[50], lens[97] = 300, 0
    c = Cache(lens, kv_heads=8, heads=8, device="cuda", seed=85)
    run(c, counts)


@pytest.mark.parametrize("seed,G", [(1, 4), (2, 3)])
def test_many_items_of_many_rows(seed, G):
    """More than four items per SM, of more than half a row tile on average: a CTA for each, found by a search."""
    rng = np.random.default_rng(seed)
    B = 70
    lens = [int(x) for x in rng.choice([0, 1, 100, 129, 300], B)]
    counts = [int(x) for x in rng.choice([0, 1, 60, 64, 86, 130], B)]
    c = Cache(lens, kv_heads=8, heads=8 * G, device="cuda", seed=90 + seed)
    assert sum(counts) * G > 128 * B and skv.splitkv_cross_workspace_size(c.desc, sum(counts)) == 0
    run(c, counts, before=3, pad=2)
    c = Cache([200] * B, kv_heads=8, heads=8 * G, tokens=60, device="cuda", seed=92 + seed)
    run(c, [60] * B, cu=False)
