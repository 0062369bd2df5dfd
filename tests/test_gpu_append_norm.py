"""GPU tests of append with norms against a plain 64-bit implementation.

Tolerances.  In fp32 a row's sum of squares is off by at most 20 roundings of 2^-24 (16 squares added in turn, then
three or five sums), its reciprocal root by half of that and two units in the last place, 2^-22, and two products by
2^-24 each: 18 * 2^-24 < 1.2e-6 of the component.  The rotation mixes a pair (u, v), and adds 4e-7 (|u| + |v|) (as in the
tests of the plain append).  Then one rounding: half a step of bf16, 2^-8 of the value, or of e4m3, 2^-4 or 2^-10 among
the subnormals.
"""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import EPS16, Cache, rotated
from _support import need_gpu

pytestmark = pytest.mark.gpu
FP32 = 1.2e-6 + 4e-7


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def normed(x, weight, eps, columns):
    y = x.copy()
    part = x[..., :columns]
    y[..., :columns] = part / np.sqrt((part * part).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y[..., :columns] *= weight
    return y


def run(c, counts, rot=128, offset=0, pairing=0, sections=None, eps=1e-6, which="qk", weights="qk", per_head="", scales=None,
        kv_scale=0.5, seed=3, in_place=False, queries=True, rope=True, pad=0, spread=2.0, cu=True, rows=None, graph=False):
    n, latent = sum(counts) + pad, c.dim == 576
    columns = 512 if latent else 128
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    widths = (c.heads * c.dim, c.Hkv * c.dim, 0 if c.shares else c.Hkv * c.v_dim)
    if rows is None:
        rows = torch.randn((n, sum(widths) + 64), generator=g, device="cuda")
        rows = rows * torch.exp(spread * torch.randn((n, 1), generator=g, device="cuda"))
    rows = rows.to(torch.bfloat16)
    q = rows[:, :widths[0]].view(n, c.heads, c.dim)
    k = rows[:, widths[0]:widths[0] + widths[1]].view(n, c.Hkv, c.dim)
    v = None if c.shares else rows[:, widths[0] + widths[1]:sum(widths)].view(n, c.Hkv, c.v_dim)
    sections = sections or (rot // 2,)
    freqs = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    pos = rng.integers(0, 100000, (len(sections), n)).astype(np.int32)
    r = skv.splitkv_rope_create(rot, sections, freqs=freqs, rot_offset=offset, pairing=pairing) if rope else None

    def weight(name, heads):
        if name not in weights or name not in which:
            return None
        shape = (heads, columns) if name in per_head else (columns,)
        return 1.0 + 0.3 * torch.randn(shape, generator=g, device="cuda")

    wq, wk = weight("q", c.heads), weight("k", c.Hkv)
    q64, k64 = q.double().cpu().numpy(), k.double().cpu().numpy()
    v64 = None if v is None else v.double().cpu().numpy()
    kp, vp = c.values(c.k), None if c.shares else c.values(c.v)
    q_out = q if in_place else torch.full((n, c.heads, c.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cut = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda") if cu else None
    ks, vs = (None, None) if scales is None else (torch.tensor(x, dtype=torch.float32, device="cuda") for x in scales)
    positions = torch.from_numpy(pos).cuda()

    def call():
        skv.splitkv_append_norm(c.desc, r, positions, q if queries else None, k, v, c.table, c.lens,
                                q_out if queries else None, c.k, c.v, norm_q="q" in which, norm_k="k" in which, q_weight=wq,
                                k_weight=wk, eps=eps, cu_tokens=cut, kv_scale=kv_scale, k_scale=ks, v_scale=vs, status=st)

    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            call()
        captured.replay()
    else:
        call()
    torch.cuda.synchronize()
    assert int(st) == 0

    def finished(x, name, w):
        """The exact row, and what its fp32 errors are measured by: |u| + |v| of the pairs that turn."""
        y = normed(x, None if w is None else w.double().cpu().numpy(), eps, columns) if name in which else x
        size = np.abs(y)
        if rope:
            half = rot // 2
            iu = offset + (np.arange(half) if pairing == 0 else 2 * np.arange(half))
            iv = iu + (half if pairing == 0 else 1)
            size[..., iu] = size[..., iv] = np.abs(y[..., iu]) + np.abs(y[..., iv])
            y = rotated(y, pos, freqs, sections, offset, pairing)
        return y, size

    m = sum(counts)

    def close(got, want, size, e4m3=False):
        half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) if e4m3 else EPS16 * np.abs(want)
        err = np.abs(got - want) - half - FP32 * size
        assert err.max(initial=-1) <= 0, err.max()

    got = q_out.double().cpu().numpy()
    if queries:
        want, size = finished(q64, "q", wq)
        close(got[:m], want[:m], size[:m])
        assert np.array_equal(got[m:], q64[m:] if in_place else np.full_like(got[m:], 7))
    table = c.table.cpu().numpy()
    want, size = finished(k64, "k", wk)
    new_k, new_v = c.values(c.k), None if c.shares else c.values(c.v)
    at = 0
    for b, count in enumerate(counts):
        for i in range(count):
            j = c.lens_host[b] - count + i
            page, off = table[b, j // c.P], j % c.P
            for h in range(c.Hkv):
                x = new_k[page, h, off]
                if c.dtype == "e4m3":
                    sc = np.float32(scales[0][h] if scales else kv_scale)
                    close(x, np.clip(want[at + i, h] / sc, -448, 448), size[at + i, h] / sc, True)
                else:
                    close(x, want[at + i, h], size[at + i, h])
                kp[page, h, off] = x
                if new_v is not None:
                    if c.dtype != "e4m3":
                        assert np.array_equal(new_v[page, h, off], v64[at + i, h])
                    vp[page, h, off] = new_v[page, h, off]
        at += count
    assert np.array_equal(new_k, kp) and (c.shares or np.array_equal(new_v, vp))  # nothing else was written
    return q_out


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("pairing", [0, 1])
def test_ragged_prompts(dtype, layout, pairing):
    c = Cache([5, 3, 30, 40, 100], dtype=dtype, layout=layout, device="cuda", seed=1)
    run(c, [5, 0, 1, 40, 17], sections=(24, 20, 20), pairing=pairing, pad=2)


@pytest.mark.parametrize("rot,offset,sections", [(64, 0, None), (64, 64, (10, 11, 11)), (16, 48, None), (128, 0, (1, 2, 3, 58))])
@pytest.mark.parametrize("pairing", [0, 1])
def test_rows_that_turn_in_part(rot, offset, sections, pairing):
    """The lanes that hold a row's chunks change with the rotated columns; the sum over them does not."""
    c = Cache([33, 7], kv_heads=1, heads=3, page=32, device="cuda", seed=2)
    run(c, [9, 7], rot=rot, offset=offset, sections=sections, pairing=pairing)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shares", [True, False])
@pytest.mark.parametrize("offset", [512, 16])  # (rotated columns among the normalised ones)
def test_latent_rows(dtype, shares, offset):
    c = Cache([70, 6], kv_heads=1, heads=128, page=64, dim=576, v_dim=512, shares=shares, dtype=dtype, device="cuda", seed=3)
    run(c, [7, 6], rot=64, offset=offset, pairing=1, which="k", weights="k")
    c = Cache([70, 6], kv_heads=1, heads=5, page=64, dim=576, v_dim=512, shares=shares, dtype=dtype, device="cuda", seed=3)
    run(c, [70, 6], rot=64, offset=offset, which="k", weights="", queries=False)


@pytest.mark.parametrize("which,weights,per_head", [("q", "q", ""), ("k", "k", ""), ("qk", "", ""), ("qk", "k", "k"),
                                                    ("qk", "qk", "q"), ("qk", "qk", "qk")])
def test_which_rows_and_weights(which, weights, per_head):
    c = Cache([20, 9], kv_heads=3, heads=6, device="cuda", seed=4)
    run(c, [4, 9], which=which, weights=weights, per_head=per_head)


def test_in_place_uniform_and_without_queries_or_rotation():
    c = Cache([3, 50, 16], device="cuda", tokens=3, seed=5)
    run(c, [3, 3, 3], in_place=True, cu=False)
    run(c, [2, 1, 0], queries=False)
    run(c, [2, 1, 0], rope=False, pad=5, in_place=True)


@pytest.mark.parametrize("eps", [1e-6, 1e-3, 10.0])
def test_small_and_empty_rows(eps):
    """Rows whose squares are below eps, rows of zeros, and rows of one large component."""
    c = Cache([12], kv_heads=1, heads=2, device="cuda", seed=6)
    rows = torch.randn((12, 4 * 128 + 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    rows[0] = 0
    rows[1] *= 1e-5
    rows[2] *= 1e-20
    rows[3] *= 1e8
    rows[4] = 0
    rows[4, 5::128] = 2.0 ** 59
    rows[5, 130] = -3e4
    run(c, [12], rows=rows, eps=eps)


def test_a_row_with_a_nan_or_infinity_spoils_no_other():
    c = Cache([8], kv_heads=1, heads=2, device="cuda", seed=8)
    rows = torch.randn((8, 4 * 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)).to(torch.bfloat16)
    outs = []
    for bad in (None, float("nan"), float("inf")):
        x = rows.clone()
        if bad is not None:
            x[3, 7] = bad          # first query head
            x[5, 2 * 128 + 1] = bad  # key
        q, k, v = (x[:, a * 128:b * 128].view(8, b - a, 128) for a, b in ((0, 2), (2, 3), (3, 4)))
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        kp, vp = torch.zeros_like(c.k), torch.zeros_like(c.v)
        skv.splitkv_append_norm(c.desc, skv.splitkv_rope_create(128), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8),
                                q, k, v, c.table, c.lens, out, kp, vp,
                                cu_tokens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
        outs.append((out, kp))
    t = int(c.table[0, 0])
    for out, kp in outs[1:]:
        assert out[3, 0].isnan().any() and kp[t, 0, 5].isnan().any()
        same = torch.ones((8, 2), dtype=torch.bool, device="cuda")
        same[3, 0] = False
        assert torch.equal(out[same], outs[0][0][same])
        keys = torch.arange(8, device="cuda") != 5
        assert torch.equal(kp[t, 0, :8][keys], outs[0][1][t, 0, :8][keys])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_long_calls_and_many_heads(dtype):
    """Two units per thread, several tokens to a CTA (bf16: 40 rows), and a token of several CTAs."""
    c = Cache([700, 300], kv_heads=4, heads=32, dtype=dtype, device="cuda", seed=10)
    run(c, [700, 300])
    c = Cache([2], kv_heads=70, heads=140, dtype=dtype, device="cuda", seed=11)
    run(c, [2], per_head="q")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv_heads,per_head,tokens", [(8, 4, "", 4300), (32, 4, "qk", 1800), (64, 8, "qk", 900),
                                                            (6, 2, "k", 7500), (128, 8, "", 470)])
def test_calls_of_a_ring(dtype, heads, kv_heads, per_head, tokens):
    """More than 2^16 rows: stages of four tokens, two or one, weights in shared memory or (64 heads of their own) not; an odd
    number of tokens, sequences that end within a stage, padding behind them."""
    counts = [tokens // 2 + 1, 0, 1, 2, tokens // 2 - 8]
    c = Cache([n + 5 for n in counts], kv_heads=kv_heads, heads=heads, dtype=dtype, layout="NHD", device="cuda", seed=16)
    run(c, counts, per_head=per_head, pad=3, sections=(24, 20, 20), kv_scale=0.25)
    run(c, counts, per_head=per_head, rot=64, offset=32, pairing=1, kv_scale=0.3, which="qk", weights="k", in_place=True)


def test_a_ring_of_keys_alone_and_many_sequences():
    rng = np.random.default_rng(17)
    counts = [int(x) for x in rng.integers(0, 30, 600)]
    lens = [n + int(x) for n, x in zip(counts, rng.integers(0, 20, 600))]
    c = Cache(lens, kv_heads=4, heads=4, device="cuda", seed=17)
    run(c, counts, queries=False, weights="")


def test_a_ring_reports_slots_and_pages_and_writes_the_state():
    n = 8300
    c = Cache([n, 40], kv_heads=4, heads=4, page=64, device="cuda", seed=18)
    x = torch.randn((n + 40, 12, 128), device="cuda").to(torch.bfloat16)
    w = torch.full((2, 4, c.cap), 5.0, device="cuda")
    p = torch.full((2, 4, c.cap), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lens[1] = 37         # the first three tokens of the second sequence have no slot
    c.table[0, 100] = c.N  # nor a page those of keys 6400 to 6463
    k0 = c.k.clone()
    pos = torch.arange(n + 40, dtype=torch.int32, device="cuda").view(1, -1)
    out = torch.zeros((n + 40, 4, 128), dtype=torch.bfloat16, device="cuda")
    skv.splitkv_append_norm(c.desc, None, pos, x[:, :4], x[:, 4:8], x[:, 8:], c.table, c.lens, out, c.k, c.v,
                            cu_tokens=torch.tensor([0, n, n + 40], dtype=torch.int32, device="cuda"), key_weights=w, key_positions=p,
                            status=st)
    torch.cuda.synchronize()
    assert int(st) == skv.SPLITKV_DEVERR_SEQLEN | skv.SPLITKV_DEVERR_PAGE
    want = torch.zeros((2, c.cap), dtype=torch.bool, device="cuda")
    want[0, :n], want[1, :37] = True, True
    want[0, 6400:6464] = False
    assert torch.equal(w == 0, want[:, None].expand(2, 4, -1))
    at = torch.where(want[0], torch.arange(c.cap, device="cuda"), -9)
    assert torch.equal(p[0], at.int()[None].expand(4, -1)) and torch.equal(p[1, 0, :37], torch.arange(n + 3, n + 40, device="cuda").int())
    pages = torch.zeros(c.N, dtype=torch.bool, device="cuda")
    pages[c.table[0].long()[torch.arange(c.width, device="cuda") != 100][:130 - 1]] = True
    changed = (c.k != k0).flatten(1).any(1)
    assert not changed[[i for i in range(c.N) if not pages[i] and i != int(c.table[1, 0])]].any()
    assert (out != 0).any(-1).all()  # the queries come whole


def test_per_head_scales():
    c = Cache([10, 31], dtype="e4m3", device="cuda", seed=12)
    run(c, [10, 4], scales=([0.25, 0.001], [0.001, 3.0]))


def test_same_results_as_norms_apart_and_captured():
    c = Cache([40, 11], device="cuda", seed=13)
    first = run(c, [21, 11], seed=14)
    again = run(c, [21, 11], seed=14, graph=True)
    assert torch.equal(first, again)


def test_nothing_normalised_is_the_plain_append():
    c = Cache([30], device="cuda", seed=15)
    x = torch.randn((30, c.heads + 2 * c.Hkv, 128), device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :c.heads], x[:, c.heads:c.heads + c.Hkv], x[:, c.heads + c.Hkv:]
    rope, pos = skv.splitkv_rope_create(128), torch.arange(30, dtype=torch.int32, device="cuda").view(1, 30)
    cu = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
    outs = [torch.zeros((30, c.heads, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pools = [torch.zeros_like(c.k) for _ in range(4)]
    skv.splitkv_append(c.desc, rope, pos, q, k, v, c.table, c.lens, outs[0], *pools[:2], cu_tokens=cu)
    skv.splitkv_append_norm(c.desc, rope, pos, q, k, v, c.table, c.lens, outs[1], *pools[2:], norm_q=False, norm_k=False,
                            cu_tokens=cu)
    assert torch.equal(*outs) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
