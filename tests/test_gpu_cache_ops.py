"""GPU tests of append, key weights and eviction against plain 64-bit implementations.

Tolerances.  bf16: half a step, 2^-8 of the value; e4m3: half a step, 2^-4 of the value or 2^-10 among the
subnormals.  Rotation in fp32 adds, per component of a pair (u, v), at most (|u| + |v|) times the error of a
sine or cosine (the angle to 2^-25 half turns = 9.4e-8 rad, the function to 2 ulp = 1.2e-7) and of two products
and a sum (1.8e-7): 4e-7 (|u| + |v|).  Key weights: see `weight_tolerance`.  Eviction moves bits: equality.
"""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import EPS16, Cache, evict_moves, key_weights, lse_of, rotated
from _support import need_gpu

pytestmark = pytest.mark.gpu
SINE = 4e-7


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

def close(got, want, about, e4m3=False):
    """`about`: |u| + |v| of each component's pair."""
    half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) if e4m3 else EPS16 * np.abs(want)
    err = np.abs(got - want) - half - SINE * about
    assert err.max(initial=-1) <= 0, err.max()


def run_append(c, counts, rot=128, sections=None, pairing=0, offset=0, pos_base=0, seed=3, in_place=False, cu=True,
               kv_scale=0.5, scales=None, wide=True, rope=True, queries=True, pad=0, state=True, n_heads=None):
    n = sum(counts) + pad
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    heads = c.heads
    widths = (heads * c.dim, c.Hkv * c.dim, 0 if c.shares else c.Hkv * c.v_dim)
    rows = torch.randn((n, sum(widths) + (64 if wide else 0)), generator=g, device="cuda").to(torch.bfloat16)
    q = rows[:, :widths[0]].view(n, heads, c.dim) if wide else rows[:, :widths[0]].reshape(n, heads, c.dim).contiguous()
    k = rows[:, widths[0]:widths[0] + widths[1]].view(n, c.Hkv, c.dim)
    v = None if c.shares else rows[:, widths[0] + widths[1]:sum(widths)].view(n, c.Hkv, c.v_dim)
    sections = sections or (rot // 2,)
    freqs = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    pos = rng.integers(0, 4096, (len(sections), n)).astype(np.int32) + np.int32(pos_base)
    positions = torch.from_numpy(pos).cuda()
    r = skv.splitkv_rope_create(rot, sections, freqs=freqs, rot_offset=offset, pairing=pairing) if rope else None
    q0, k0 = q.double().cpu().numpy(), k.double().cpu().numpy()
    v0 = None if v is None else v.double().cpu().numpy()
    kp0, vp0 = c.values(c.k), None if c.shares else c.values(c.v)
    q_out = q if in_place else torch.full((n, heads, c.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    w = torch.full((c.B, c.Hkv, c.cap), 5.0, device="cuda") if state else None
    kpos = torch.full((c.B, c.Hkv, c.cap), -9, dtype=torch.int32, device="cuda") if state else None
    st = status_word()
    cut = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda") if cu else None
    ks = vs = None
    if scales is not None:
        ks, vs = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in scales)
    skv.splitkv_append(c.desc, r, positions, q if queries else None, k, v, c.table, c.lens, q_out if queries else None,
                       c.k, c.v, cu_tokens=cut, kv_scale=kv_scale, k_scale=ks, v_scale=vs, key_weights=w,
                       key_positions=kpos, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0

    def turned(x):
        return rotated(x, pos, freqs, sections, offset, pairing) if rope else x

    m = sum(counts)

    def about(x):  # |u| + |v| of every component's pair, 0 where nothing turns
        a = np.zeros_like(x)
        if rope:
            half = rot // 2
            iu = offset + (np.arange(half) if pairing == 0 else 2 * np.arange(half))
            iv = iu + (half if pairing == 0 else 1)
            a[..., iu] = a[..., iv] = np.abs(x[..., iu]) + np.abs(x[..., iv])
        return a

    if queries:
        got = q_out.double().cpu().numpy()
        close(got[:m], turned(q0)[:m], about(q0)[:m])
        if not in_place:
            assert (got[m:] == 7).all()  # rows behind the last sequence
        else:
            assert np.array_equal(got[m:], q0[m:])
    # every row of the pools: the new ones, and all others as they were
    e4m3 = c.dtype == "e4m3"
    table = c.table.cpu().numpy()
    kt, at = turned(k0), 0
    want_w, want_p = np.full((c.B, c.Hkv, c.cap), 5.0), np.full((c.B, c.Hkv, c.cap), -9)
    new_k, new_v = c.values(c.k), None if c.shares else c.values(c.v)
    for b, cnt in enumerate(counts):
        for i in range(cnt):
            j = c.lens_host[b] - cnt + i
            page, off = table[b, j // c.P], j % c.P
            for h in range(c.Hkv):
                for new, old, val, sc, a in ((new_k, kp0, kt, scales[0][h] if scales else kv_scale, about(k0)),
                                             (new_v, vp0, v0, scales[1][h] if scales else kv_scale, None)):
                    if new is None:
                        continue
                    x, y = new[page, h, off], val[at + i, h]
                    around = 0 if a is None else a[at + i, h]
                    if e4m3:
                        close(x, np.clip(y / np.float32(sc), -448, 448), around / sc, True)
                    else:
                        close(x, y, around)
                        if a is None:
                            assert np.array_equal(x, y)
                    old[page, h, off] = x
            want_w[b, :, j], want_p[b, :, j] = 0, pos[0][at + i]
        at += cnt
    assert np.array_equal(new_k, kp0)
    if not c.shares:
        assert np.array_equal(new_v, vp0)
    if state:
        assert np.array_equal(w.cpu().numpy(), want_w) and np.array_equal(kpos.cpu().numpy(), want_p)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("pairing", [0, 1])
def test_append_ragged_prompts(dtype, layout, pairing):
    counts = [5, 0, 1, 40, 17]
    c = Cache([5, 3, 30, 40, 100], page=16, dtype=dtype, layout=layout, device="cuda", seed=1)
    run_append(c, counts, sections=(24, 20, 20), pairing=pairing)


@pytest.mark.parametrize("rot,offset,sections", [(64, 0, None), (64, 64, (10, 11, 11)), (16, 48, None), (32, 16, (0, 16, 0)),
                                                 (128, 0, (1, 2, 3, 58))])
@pytest.mark.parametrize("pairing", [0, 1])
def test_append_partial_rotation(rot, offset, sections, pairing):
    c = Cache([33, 7], kv_heads=1, heads=3, page=32, device="cuda", seed=2)
    run_append(c, [9, 7], rot=rot, offset=offset, sections=sections, pairing=pairing)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shares", [True, False])
def test_append_latent_rows(dtype, shares):
    c = Cache([70, 6], kv_heads=1, heads=128, page=64, dim=576, v_dim=512, shares=shares, dtype=dtype, device="cuda", seed=3)
    run_append(c, [7, 6], rot=64, offset=512, pairing=1)


@pytest.mark.parametrize("pos_base", [0, 1 << 20, (1 << 31) - 5000, -(1 << 31), -3000])
def test_append_far_positions(pos_base):
    run_append(Cache([20], device="cuda", seed=4), [20], pos_base=pos_base)


def test_append_in_place_uniform_and_bare():
    c = Cache([3, 50, 16], device="cuda", tokens=3, seed=5)
    run_append(c, [3, 3, 3], in_place=True, cu=False)
    run_append(c, [3, 3, 3], wide=False, state=False)
    run_append(c, [2, 1, 0], queries=False, rope=False)  # encoder states
    run_append(c, [2, 1, 0], pad=5)                      # rows behind the last sequence
    run_append(c, [2, 1, 0], pad=5, in_place=True)


def test_append_per_head_scales_and_saturation():
    c = Cache([10, 31], dtype="e4m3", device="cuda", seed=6)
    run_append(c, [10, 4], scales=([0.25, 0.001], [0.001, 3.0]))  # 0.001: most values saturate


def test_append_many_heads_and_tokens():
    c = Cache([200], kv_heads=8, heads=64, page=16, device="cuda", seed=7)
    run_append(c, [200], sections=(24, 20, 20))
    c = Cache([1] * 70, kv_heads=1, heads=1, page=16, device="cuda", seed=8)
    run_append(c, [1] * 70)


@pytest.mark.parametrize("batch", [33, 100, 1100])
def test_append_many_sequences(batch):
    rng = np.random.default_rng(batch)
    counts = [int(x) for x in rng.choice([0, 0, 1, 2], batch)]
    counts[-1] = 0
    lens = [n + int(x) for n, x in zip(counts, rng.integers(0, 40, batch))]
    run_append(Cache(lens, kv_heads=1, heads=1, device="cuda", seed=7), counts, pad=3)
    run_append(Cache([1] * batch, kv_heads=1, heads=1, device="cuda", seed=8), [1] * batch)


def test_append_reports_slots_and_pages():
    c = Cache([16, 40, 20], device="cuda", seed=9)
    c.lens[0] = 2         # shorter than its three tokens: the first has no slot
    c.lens[1] = c.cap + 1  # its last token lies behind the cache
    c.table[2, 1] = c.N   # an id out of range
    k0, v0 = c.k.clone(), c.v.clone()
    x = torch.randn((9, c.heads, 128), device="cuda").to(torch.bfloat16)
    k = torch.ones((9, c.Hkv, 128), device="cuda").to(torch.bfloat16)
    st, out = status_word(), torch.zeros_like(x)
    cu = torch.tensor([0, 3, 6, 9], dtype=torch.int32, device="cuda")
    skv.splitkv_append(c.desc, None, None, x, k, k, c.table, c.lens, out, c.k, c.v, cu_tokens=cu, status=st)
    torch.cuda.synchronize()
    assert int(st) == skv.SPLITKV_DEVERR_SEQLEN | skv.SPLITKV_DEVERR_PAGE
    assert torch.equal(out, x)  # the queries come whole
    changed = {(int(p), int(o)) for p, o in torch.nonzero((c.k != k0).any(-1).any(1))}
    t = c.table.cpu().numpy()
    assert changed == {(t[0, 0], 0), (t[0, 0], 1), (t[1, 2], 14), (t[1, 2], 15)}
    assert {(int(p), int(o)) for p, o in torch.nonzero((c.v != v0).any(-1).any(1))} == changed


# ------------------------------------------------------------------ key weights

def weight_tolerance(q, keys, lse, scale, T, w):
    """A score is a sum of 128 fp32 additions of exact products: off by at most 128 * 2^-23 * sum |q_d K_d|
    (the tensor cores may truncate); the exponent's argument rounds twice more at its size, ex2 is good to 2^-22.
    With lse = -inf rows leaving nothing, the weight of one row is off by that factor."""
    L, Hkv = keys.shape[:2]
    size = np.abs(q).max() * np.abs(keys).sum(-1).max() * scale if L else 0.0
    big = size + np.abs(lse[np.isfinite(lse)]).max(initial=0)
    return w * (128 * 2.0 ** -23 * size + 4 * 2.0 ** -24 * big + 2.0 ** -21) + 1e-37


def run_weights(c, T, decay=1.0, kv_scale=1.0, seed=11, out_of_place=True, scales=None, empty=(), std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn((c.B, T, c.heads, 128), generator=g, device="cuda") * std).to(torch.bfloat16)
    q64, kp = q.double().cpu().numpy(), c.values(c.k)
    per_head = np.array(scales if scales is not None else [kv_scale] * c.Hkv, np.float32).astype(np.float64)
    keys = [c.rows(kp, b, L) * per_head[None, :, None] for b, L in enumerate(c.lens_host)]
    scale = 128 ** -0.5
    lse = np.stack([lse_of(q64[b], keys[b], scale, T) for b in range(c.B)]).astype(np.float32)
    for i in empty:
        lse[i] = -np.inf
    w_in = torch.rand((c.B, c.Hkv, c.cap), generator=g, device="cuda")
    out = torch.full_like(w_in, -3.0) if out_of_place else w_in.clone()
    st = status_word()
    skv.splitkv_key_weights(c.desc, q, c.k, c.table, c.lens, torch.from_numpy(lse).cuda(), scale, kv_scale, decay,
                            (w_in if out_of_place else out) if decay else None, out,
                            k_scale=None if scales is None else torch.tensor(scales, dtype=torch.float32, device="cuda"), status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    got, w0 = out.double().cpu().numpy(), w_in.double().cpu().numpy()
    for b, L in enumerate(c.lens_host):
        w = key_weights(q64[b], keys[b], lse[b].astype(np.float64), scale, T)
        want = np.float32(decay) * w0[b, :, :L] + w
        tol = weight_tolerance(q64[b], keys[b], lse[b], scale, T, w) + 2.0 ** -22 * np.abs(want)
        assert (np.abs(got[b, :, :L] - want) <= tol).all(), (b, np.abs(got[b, :, :L] - want).max())
        rest = got[b, :, L:]
        assert (rest == (-3.0 if out_of_place else w0[b, :, L:])).all()  # not written
    return got


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout,page", [("HND", 16), ("NHD", 32), ("HND", 48)])
@pytest.mark.parametrize("heads,T", [(2, 1), (16, 1), (14, 2), (16, 4)])
def test_weights(dtype, layout, page, heads, T):
    c = Cache([T, 0, 17, 333, 16, 1000], kv_heads=2, heads=heads, page=page, dtype=dtype, layout=layout, device="cuda",
              tokens=T, seed=12)
    run_weights(c, T, kv_scale=1 / 64 if dtype == "e4m3" else 1.0)


def test_weights_decay_in_place_scales_and_empty_rows():
    c = Cache([100, 31, 5], device="cuda", seed=13)
    run_weights(c, 1, decay=0.5, out_of_place=False)
    run_weights(c, 1, decay=0.0)
    run_weights(c, 1, decay=-2.0, empty=(1,))
    c = Cache([100, 31, 5], dtype="e4m3", device="cuda", seed=14)
    run_weights(c, 1, scales=[1 / 64, 1 / 200])


def test_weights_of_large_and_tiny_queries():
    """f16 would overflow or vanish: the e4m3 path scales each query row."""
    for std in (1e6, 1e-6):
        c = Cache([50], dtype="e4m3", kv_heads=1, heads=8, device="cuda", seed=15)
        run_weights(c, 1, kv_scale=1 / (64 * std), std=std)


def test_weights_ignore_what_lies_behind_the_length():
    c = Cache([21, 5], device="cuda", seed=16)
    bad = c.k.clone()
    t = c.table.cpu().numpy()
    bad[t[0, 1], :, 5:] = float("nan")
    bad[t[1, 0], :, 5:] = float("inf")
    first = run_weights(c, 1)
    c.k.copy_(bad)
    got = run_weights(c, 1)
    assert np.array_equal(first, got)


def test_weights_report_lengths_and_pages():
    c = Cache([40, 40, 40, 40], device="cuda", tokens=2, seed=17)
    st, q = status_word(), torch.zeros((4, 2, c.heads, 128), dtype=torch.bfloat16, device="cuda")
    c.lens.copy_(torch.tensor([-1, c.cap + 1, 1, 40]))
    out = torch.full((4, c.Hkv, c.cap), 2.0, device="cuda")
    lse = torch.zeros((4, 2, c.heads), device="cuda")
    args = (c.desc, q, c.k, c.table, c.lens, lse, 0.1, 1.0, 1.0, out, out)
    skv.splitkv_key_weights(*args, status=st)
    assert int(st) == skv.SPLITKV_DEVERR_SEQLEN
    assert (out[:3] == 2).all() and (out[3, :, :39] == 2 + 2 * c.heads // c.Hkv).all()
    c.lens.fill_(40)
    c.table[1, 0] = -1
    st.zero_()
    skv.splitkv_key_weights(*args, status=st)
    assert int(st) == skv.SPLITKV_DEVERR_PAGE
    skv.splitkv_key_weights(*args)  # without a status word


@pytest.mark.parametrize("batch", [1, 33, 100])
def test_weights_of_many_and_long_sequences(batch):
    rng = np.random.default_rng(batch)
    lens = [20000] if batch == 1 else list(rng.integers(0, 200, batch))
    run_weights(Cache(lens, kv_heads=1 if batch == 1 else 2, heads=8, device="cuda", seed=18), 1)


# ------------------------------------------------------------------ evict

def run_evict(c, budget, sink=0, recent=0, weights=None, positions="slots", in_place=False, seed=21):
    rng = np.random.default_rng(seed)
    w0 = np.exp(2 * rng.standard_normal((c.B, c.Hkv, c.cap))).astype(np.float32) if weights is None else weights
    if isinstance(positions, str) and positions == "slots":
        p0 = np.broadcast_to(np.arange(c.cap, dtype=np.int32), w0.shape).copy()
    elif isinstance(positions, str):
        p0 = rng.integers(-(1 << 31), 1 << 31, w0.shape).astype(np.int32)
    else:
        p0 = positions
    w = torch.from_numpy(w0).cuda()
    p = None if p0 is None else torch.from_numpy(p0).cuda()
    wo = w if in_place else torch.full_like(w, -1.0)
    po = p if in_place or p is None else torch.full_like(p, -1)
    lens_out = c.lens if in_place else torch.full_like(c.lens, -1)
    kp, vp = c.k.cpu().clone(), None if c.shares else c.v.cpu().clone()
    st = status_word()
    ws = torch.empty(skv.splitkv_evict_workspace_size(c.desc, budget), dtype=torch.uint8, device="cuda")
    skv.splitkv_evict(c.desc, budget, sink, recent, c.k, c.v, c.table, c.lens, w, p, wo, po, lens_out, ws, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    t = c.table.cpu().numpy()
    got_w, got_p = wo.cpu().numpy(), None if po is None else po.cpu().numpy()
    want_w = w0.copy() if in_place else np.full_like(w0, -1)
    want_p = None if p0 is None else p0.copy() if in_place else np.full_like(p0, -1)
    moved = 0
    for b, L in enumerate(c.lens_host):
        assert int(lens_out[b]) == min(L, budget)
        for h in range(c.Hkv):
            n, moves = evict_moves(w0[b, h], None if p0 is None else p0[b, h], L, budget, sink, recent)
            moved += len(moves)
            gone = {d for d, _ in moves}
            for j in range(n):
                if j not in gone:
                    want_w[b, h, j] = w0[b, h, j]
                    if p0 is not None:
                        want_p[b, h, j] = p0[b, h, j]
            for d, s in moves:
                want_w[b, h, d] = w0[b, h, s]
                if p0 is not None:
                    want_p[b, h, d] = p0[b, h, s]
                at, to = (t[b, s // c.P], s % c.P), (t[b, d // c.P], d % c.P)
                for pool in (kp, vp):
                    if pool is not None:
                        if c.layout == "HND":
                            pool[to[0], h, to[1]] = pool[at[0], h, at[1]]
                        else:
                            pool[to[0], to[1], h] = pool[at[0], at[1], h]
    assert np.array_equal(got_w, want_w, equal_nan=True)
    assert p0 is None or np.array_equal(got_p, want_p)
    assert torch.equal(c.k.cpu().view(torch.uint8), kp.view(torch.uint8))
    assert c.shares or torch.equal(c.v.cpu().view(torch.uint8), vp.view(torch.uint8))
    return moved


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget", [1, 31, 64, 500])
def test_evict(dtype, layout, in_place, budget):
    c = Cache([0, 1, 31, 64, 65, 700, 333], page=16, dtype=dtype, layout=layout, device="cuda", seed=22)
    assert run_evict(c, budget, sink=4, recent=20, in_place=in_place) > 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shares", [True, False])
def test_evict_latent_rows(dtype, shares):
    c = Cache([300, 64, 1000], kv_heads=1, heads=128, page=64, dim=576, v_dim=512, shares=shares, dtype=dtype, device="cuda", seed=23)
    assert run_evict(c, 100, sink=2, recent=30)


def test_evict_ties_zeros_and_odd_weights():
    c = Cache([900, 50, 333], device="cuda", seed=24)
    shape = (c.B, c.Hkv, c.cap)
    run_evict(c, 40, weights=np.zeros(shape, np.float32))
    run_evict(c, 40, weights=np.ones(shape, np.float32), recent=10, sink=3)
    rng = np.random.default_rng(0)
    few = rng.integers(0, 3, shape).astype(np.float32)
    run_evict(c, 200, weights=few)
    odd = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, -1, -0.0, 0.0, 1e-45, 1e-39, 3.4e38, 1], np.float32), shape)
    run_evict(c, 100, weights=odd)
    near = (1 + rng.integers(0, 4, shape) * 2.0 ** -23).astype(np.float32)  # the last digits decide
    run_evict(c, 100, weights=near)


def test_evict_protects_by_position():
    c = Cache([300, 300], device="cuda", seed=25)
    run_evict(c, 64, sink=0, recent=64)
    run_evict(c, 64, sink=10, recent=100)       # more protected keys than the budget: the best of them
    run_evict(c, 64, sink=1 << 30, recent=5)    # everything protected
    run_evict(c, 64, sink=5, recent=2 ** 31 - 1)
    run_evict(c, 64, sink=5, recent=1000, positions="random")
    same = np.zeros((c.B, c.Hkv, c.cap), np.int32)
    run_evict(c, 64, recent=1, positions=same)
    run_evict(c, 64, positions=None)


@pytest.mark.parametrize("cap_pages,lens", [(1, [16]), (600, [9000, 5]), (1300, [20000]), (2100, [33001, 100]), (5000, [70001])])
def test_evict_long_sequences(cap_pages, lens):
    """Clusters of 1, 2, 4 and 8 CTAs for a head, and sequences far below the capacity."""
    c = Cache(lens, kv_heads=1, heads=1, cap_pages=cap_pages, device="cuda", seed=26)
    run_evict(c, max(1, lens[0] // 3), sink=4, recent=lens[0] // 20)
    run_evict(Cache([40], kv_heads=2, cap_pages=cap_pages + 3, device="cuda", seed=27), 10)


def test_evict_more_keys_than_shared_memory_holds():
    c = Cache([380001], kv_heads=1, heads=1, page=64, device="cuda", seed=28)  # 47,504 a CTA
    few = np.random.default_rng(1).integers(0, 50, (1, 1, c.cap)).astype(np.float32)
    run_evict(c, 100003, sink=4, recent=1000, weights=few)


def test_evict_reports_lengths_and_pages():
    c = Cache([100, 100, 100], device="cuda", seed=29)
    c.lens.copy_(torch.tensor([-5, c.cap + 1, 100]))
    c.table[2, 6] = c.N + 7  # slots 96 .. 99: their rows cannot move
    k0 = c.k.clone()
    w = torch.zeros((3, c.Hkv, c.cap), device="cuda")
    w[2, :, 90:100] = 1.0
    wo, lens, st = torch.full_like(w, -1.0), torch.zeros_like(c.lens), status_word()
    ws = torch.empty(skv.splitkv_evict_workspace_size(c.desc, 10), dtype=torch.uint8, device="cuda")
    skv.splitkv_evict(c.desc, 10, 0, 0, c.k, c.v, c.table, c.lens, w, None, wo, None, lens, ws, status=st)
    torch.cuda.synchronize()
    assert int(st) == skv.SPLITKV_DEVERR_SEQLEN | skv.SPLITKV_DEVERR_PAGE
    assert lens.tolist() == [-5, c.cap + 1, 10]
    assert (wo[:2] == -1).all() and (wo[2, :, :10] == 1).all()
    t = c.table.cpu().numpy()
    for j in range(10):
        src = c.k[t[2, 5], :, 10 + j] if j < 6 else k0[t[2, 0], :, j]
        assert torch.equal(c.k[t[2, 0], :, j], src)


# ------------------------------------------------------------------ streams and graphs

def test_captured_calls_follow_the_device_lengths():
    """One graph of all three, replayed for other lengths, tokens and weights."""
    c = Cache([200, 90], device="cuda", cap_pages=20, seed=30)
    big = Cache([320, 320], device="cuda", cap_pages=20, seed=31)  # pages for every length up to the capacity
    c.k, c.v, c.table, c.N, c.desc = big.k, big.v, big.table, big.N, big.desc
    n, T = 2, 1
    q = torch.zeros((n, c.heads, 128), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((n, c.Hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    w = torch.rand((2, c.Hkv, c.cap), device="cuda")
    kpos = torch.arange(c.cap, dtype=torch.int32, device="cuda").expand(2, c.Hkv, -1).contiguous()
    q_out, lse = torch.empty_like(q), torch.zeros((2, 1, c.heads), device="cuda")
    rope = skv.splitkv_rope_create(128)
    ws = torch.empty(skv.splitkv_evict_workspace_size(c.desc, 64), dtype=torch.uint8, device="cuda")
    lens_out, wo, po = torch.zeros_like(c.lens), torch.zeros_like(w), torch.zeros_like(kpos)

    def step(stream):
        skv.splitkv_append(c.desc, rope, pos, q, k, v, c.table, c.lens, q_out, c.k, c.v, key_weights=w, key_positions=kpos,
                           stream=stream)
        skv.splitkv_key_weights(c.desc, q_out, c.k, c.table, c.lens, lse, 0.1, 1.0, 0.5, w, w, stream=stream)
        skv.splitkv_evict(c.desc, 64, 2, 8, c.k, c.v, c.table, c.lens, w, kpos, wo, po, lens_out, ws, stream=stream)

    s = torch.cuda.Stream()
    keep = [x.clone() for x in (c.k, c.v, w, kpos)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(torch.cuda.current_stream())
    for trial in range(3):
        g = torch.Generator(device="cuda").manual_seed(trial)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        c.lens.copy_(torch.tensor([[200, 90], [1, 320], [65, 64]][trial]))
        pos.fill_(1000 * trial)
        results = []
        for run in (graph.replay, lambda: step(s)):
            for x, y in zip((c.k, c.v, w, kpos), keep):
                x.copy_(y)
            for x in (wo, po):
                x.zero_()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            results.append([x.clone() for x in (c.k, c.v, w, kpos, wo, po, lens_out, q_out)])
        for x, y in zip(*results):
            assert torch.equal(x, y)
        assert lens_out.tolist() == [min(64, x) for x in c.lens.tolist()]
