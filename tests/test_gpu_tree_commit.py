"""GPU tests of the commit of accepted paths: rows and state move as they are, so everything is compared for equality."""
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


def bits(pool):
    return pool.view(torch.int16 if pool.dtype == torch.bfloat16 else torch.uint8).cpu().numpy().copy()


def run(c, counts, paths, cu=True, state=True, max_path=None, in_place=False, status=0, lens=None, graph=False, before=0, broken=()):
    """`broken`: sequences that have to be left as they are."""
    width = max_path or max([1] + [len(p) for p in paths])
    path = torch.tensor([(p + [-7] * width)[:width] for p in paths], dtype=torch.int32, device="cuda")
    n = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.rand((c.B, c.Hkv, c.cap), generator=g, device="cuda") if state else None
    p = torch.randint(0, 1 << 30, (c.B, c.Hkv, c.cap), generator=g, device="cuda", dtype=torch.int32) if state else None
    old_w, old_p = (w.cpu().numpy().copy(), p.cpu().numpy().copy()) if state else (None, None)
    before_lens = c.lens.cpu().numpy().copy()
    out = c.lens if in_place else torch.full((c.B,), -5, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cut = torch.tensor(before + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda") if cu else None
    kp, vp = bits(c.k), None if c.shares else bits(c.v)

    def call():
        skv.splitkv_tree_commit(c.desc, path, n, c.k, c.v, c.table, c.lens, out, cu_tokens=cut, key_weights=w, key_positions=p,
                                status=st)

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
    t = c.table.cpu().numpy()
    want_k, want_v, want_w, want_p = kp.copy(), None if vp is None else vp.copy(), None, None
    if state:
        want_w, want_p = old_w.copy(), old_p.copy()
    want_lens = before_lens.copy()
    for b, count in enumerate(counts):
        L = int(before_lens[b])
        if b in broken or L == 0:
            continue
        first = L - count
        want_lens[b] = first + len(paths[b])
        for i, x in enumerate(paths[b]):
            d, s = first + i, first + x
            where = [(t[b, y // c.P], y % c.P) for y in (d, s)]
            for new, old in ((want_k, kp), (want_v, vp)):
                if new is not None:
                    (dp, do), (sp, so) = where
                    if c.layout == "HND":
                        new[dp, :, do] = old[sp, :, so]
                    else:
                        new[dp, do] = old[sp, so]
            if state:
                want_w[b, :, d], want_p[b, :, d] = old_w[b, :, s], old_p[b, :, s]
    assert np.array_equal(bits(c.k), want_k) and (c.shares or np.array_equal(bits(c.v), want_v))
    assert np.array_equal(out.cpu().numpy(), want_lens)
    if state:
        assert np.array_equal(w.cpu().numpy(), want_w) and np.array_equal(p.cpu().numpy(), want_p)


def rising(rng, count, n):
    return sorted(int(x) for x in rng.choice(count, n, replace=False))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_paths(dtype, layout, page):
    c = Cache([70, 5, 40, 200, 64, 33], page=page, dtype=dtype, layout=layout, device="cuda", seed=1)
    rng = np.random.default_rng(2)
    counts = [12, 5, 1, 64, 64, 20]
    paths = [[0, 3, 4, 11], [0, 1, 2, 3, 4], [0], rising(rng, 64, 20), rising(rng, 64, 33), []]
    run(c, counts, paths)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shares", [True, False])
def test_latent_rows(dtype, shares):
    c = Cache([70, 16, 130], kv_heads=1, heads=128, page=32, dim=576, v_dim=512, shares=shares, dtype=dtype, device="cuda", seed=3)
    run(c, [16, 16, 9], [[1, 2, 9, 15], list(range(1, 16)), [8]])


@pytest.mark.parametrize("count,n", [(300, 299), (700, 400), (257, 257)])
def test_long_paths(count, n):
    """More tokens than are looked up at a time; every row's old place is another's new one."""
    c = Cache([count + 5], kv_heads=2, page=16, device="cuda", seed=4)
    run(c, [count], [rising(np.random.default_rng(5), count, n)])
    c = Cache([count], kv_heads=1, page=16, dtype="e4m3", device="cuda", seed=4)
    run(c, [count], [list(range(count - n, count))])


@pytest.mark.parametrize("kv_heads", [1, 3, 8, 40])
def test_heads(kv_heads):
    c = Cache([50, 21], kv_heads=kv_heads, heads=kv_heads, layout="NHD", device="cuda", seed=6)
    run(c, [17, 21], [[2, 5, 6, 9, 10, 11, 12, 13, 14, 16], [20]])


def test_uniform_counts_in_place_and_without_state():
    c = Cache([30, 9, 0, 64], tokens=9, device="cuda", seed=7)
    run(c, [9] * 4, [[0, 8], [4], [], list(range(9))], cu=False, state=False)
    c = Cache([30, 9, 0, 64], tokens=9, device="cuda", seed=7)
    run(c, [9] * 4, [[0, 8], [4], [3, 5], list(range(9))], cu=False, in_place=True)
    c = Cache([30, 9, 3, 64], device="cuda", seed=7)
    run(c, [9, 2, 0, 1], [[0, 8], [1], [], [0]], before=11, max_path=40)


def test_what_does_not_rise_or_fit_is_refused():
    c = Cache([30] * 9, device="cuda", seed=8)
    paths = [[0, 2, 2], [3, 1], [0, 10], [-1, 2], list(range(10)), [0], [1], [2], [0, 9]]
    counts = [10] * 9
    path_bit, length_bit = skv.SPLITKV_DEVERR_PATH, skv.SPLITKV_DEVERR_SEQLEN
    c.lens[5] = 9           # fewer keys than tokens
    c.lens[6] = c.cap + 1
    c.lens[7] = -3
    run(c, counts, paths, max_path=9, status=path_bit | length_bit, broken=(0, 1, 2, 3, 4, 5, 6, 7))


def test_negative_path_length():
    c = Cache([30, 30], device="cuda", seed=9)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    path = torch.tensor([[3], [2]], dtype=torch.int32, device="cuda")
    n = torch.tensor([-1, 1], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda")
    skv.splitkv_tree_commit(c.desc, path, n, c.k, c.v, c.table, c.lens, c.lens, cu_tokens=cu, status=st)
    assert int(st) == skv.SPLITKV_DEVERR_PATH and c.lens.tolist() == [30, 26]


def test_pages_out_of_range():
    """The rows of such a page do not move; the others do."""
    c = Cache([40], page=16, device="cuda", seed=10)
    c.table[0, 2] = c.N
    k, t = bits(c.k), c.table.cpu().numpy()[0]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    path = torch.tensor([[2, 5, 19]], dtype=torch.int32, device="cuda")  # slots 22 -> 20, 25 -> 21, 39 -> 22
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    skv.splitkv_tree_commit(c.desc, path, torch.tensor([3], dtype=torch.int32, device="cuda"), c.k, c.v, c.table, c.lens, c.lens,
                            cu_tokens=cu, status=st)
    assert int(st) == skv.SPLITKV_DEVERR_PAGE and c.lens.tolist() == [23]
    k[t[1], :, 4], k[t[1], :, 5] = k[t[1], :, 6].copy(), k[t[1], :, 9].copy()
    assert np.array_equal(bits(c.k), k)


def test_captured_and_on_another_stream():
    c = Cache([70, 40], device="cuda", seed=11)
    run(c, [30, 12], [[1, 4, 29], [0, 11]], graph=True, in_place=True)
    c = Cache([70, 40], device="cuda", seed=11)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        run(c, [30, 12], [[1, 4, 29], [0, 11]])
