"""The cache operators as they are used together: prompts appended, tokens decoded, keys weighed and evicted, and
the decode over what is left, each step against the plain 64-bit implementation on the same state; an encoder's
states appended and attended to.  Tolerances of single steps are those of the operators' own tests; the decode's
are the decode tests'."""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import EPS16, Cache, evict_moves, key_weights, lse_of, rotated
from _support import LSE_TOL, OUT_TOL, need_gpu
from split_kv_paged_splitkv_gb300.runner import CacheSession

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def attend(q, k, v, scale, T):
    """q [T][Hq][128], k and v [L][Hkv][128] (64 bits), causal among the T: (out, lse)."""
    lse = lse_of(q, k, scale, T)
    G, L = q.shape[1] // k.shape[1], k.shape[0]
    out = np.zeros(q.shape)
    for t in range(T):
        seen = L - T + t + 1
        for h in range(q.shape[1]):
            x = k[:seen, h // G] @ q[t, h] * scale
            out[t, h] = np.exp(x - lse[t, h]) @ v[:seen, h // G]
    return out, lse


@pytest.mark.parametrize("dtype,layout,T", [("bf16", "HND", 1), ("bf16", "NHD", 2), ("e4m3", "HND", 1), ("e4m3", "NHD", 3)])
def test_life_of_a_cache(dtype, layout, T):
    B, Hkv, heads, scale = 3, 2, 8, 128 ** -0.5
    c = Cache([200] * B, kv_heads=Hkv, heads=heads, dtype=dtype, layout=layout, tokens=T, device="cuda", seed=60)
    kv_scale = 1 / 64 if dtype == "e4m3" else 1.0
    freqs = [1e4 ** (-i / 64) for i in range(64)]
    rope = skv.splitkv_rope_create(128, (24, 20, 20), freqs=freqs)
    s = CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=scale, rope=rope, kv_scale=kv_scale, num_splits=3, track=True)
    g = torch.Generator(device="cuda").manual_seed(61)
    c.lens.zero_()
    lens, written = [0] * B, [0] * B

    def take(counts):
        """Appends counts[b] new tokens to each sequence; returns their rotated queries, [n][heads][128]."""
        n = sum(counts)
        q, k, v = (torch.randn((n, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (heads, Hkv, Hkv))
        at = np.concatenate([np.arange(w, w + m) for w, m in zip(written, counts)])
        pos = np.stack([at, at // 2 + 5, at % 7]).astype(np.int32)
        for b, m in enumerate(counts):
            lens[b] += m
            written[b] += m
        c.lens.copy_(torch.tensor(lens))
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        out = s.append(torch.from_numpy(pos).cuda(), q, k, v, cu_tokens=cu)
        want = rotated(q.double().cpu().numpy(), pos, freqs, (24, 20, 20), 0, 0)
        assert (np.abs(out.double().cpu().numpy() - want) <= EPS16 * np.abs(want) + 4e-6).all()
        return out, at

    def keys():
        kp, vp = c.values(c.k) * kv_scale, c.values(c.v) * kv_scale
        return [(c.rows(kp, b, L), c.rows(vp, b, L)) for b, L in enumerate(lens)]

    take([50, 1 + T, 120])
    evictions = 0
    for step in range(8):
        q, at = take([T] * B)
        q = q.view(B, T, heads, 128)
        out, lse = s.decode(q)
        before = s.key_weights.double().cpu().numpy()
        s.weigh(q, lse, decay=0.9)
        torch.cuda.synchronize()
        q64, l64 = q.double().cpu().numpy(), lse.double().cpu().numpy()
        after = s.key_weights.double().cpu().numpy()
        for b, (k, v) in enumerate(keys()):
            want, want_l = attend(q64[b], k, v, scale, T)
            assert np.abs(out[b].double().cpu().numpy() - want).max() <= OUT_TOL
            assert np.abs(l64[b] - want_l).max() <= LSE_TOL
            w = np.float32(0.9) * before[b, :, :lens[b]] + key_weights(q64[b], k, l64[b], scale, T)
            assert np.abs(after[b, :, :lens[b]] - w).max() <= 1e-4 * np.abs(w).max()
            assert (s.key_positions[b, :, lens[b] - T:lens[b]].cpu().numpy() == np.arange(written[b] - T, written[b])).all()
        if step % 3 == 2:
            held = [(w.copy(), p.copy()) for w, p in zip(s.key_weights.cpu().numpy(), s.key_positions.cpu().numpy())]
            pools = (c.values(c.k), c.values(c.v))
            s.evict(40, sink=2, recent=10)
            torch.cuda.synchronize()
            assert c.lens.tolist() == [min(40, L) for L in lens]
            t = c.table.cpu().numpy()
            for b in range(B):
                for h in range(Hkv):
                    n, moves = evict_moves(held[b][0][h], held[b][1][h], lens[b], 40, 2, 10)
                    evictions += len(moves)
                    left = {int(p) for p in s.key_positions[b, h, :n].cpu()}
                    assert left >= set(range(max(0, written[b] - 10), written[b])) and (written[b] < 3 or left >= {0, 1})
                    for pool, new in zip(pools, (c.values(c.k), c.values(c.v))):
                        for d, sl in moves:
                            assert np.array_equal(new[t[b, d // c.P], h, d % c.P], pool[t[b, sl // c.P], h, sl % c.P])
            lens[:] = [min(40, L) for L in lens]
    assert evictions > 0
    assert s.read_status() == 0 and skv.splitkv_read_stats(s.plan, s.workspace)[1] == 0


def test_a_captured_step_of_the_whole():
    """append, decode, weigh and evict in one graph, replayed while the lengths grow and shrink on the device."""
    B, Hkv, heads = 2, 2, 8
    results = []
    for captured in (False, True):
        c = Cache([160] * B, kv_heads=Hkv, heads=heads, device="cuda", seed=62)
        s = CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=0.1, rope=skv.splitkv_rope_create(64, rot_offset=64), track=True,
                         num_splits=4)
        g = torch.Generator(device="cuda").manual_seed(63)
        c.lens.copy_(torch.tensor([60, 3]))
        q, k, v = (torch.zeros((B, h, 128), dtype=torch.bfloat16, device="cuda") for h in (heads, Hkv, Hkv))
        pos = torch.zeros((1, B), dtype=torch.int32, device="cuda")
        q_out = torch.empty_like(q)
        out, lse = torch.empty((B, 1, heads, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((B, 1, heads), device="cuda")

        def step():
            s.append(pos, q, k, v, q_out=q_out)
            s.decode(q_out.view(B, 1, heads, 128), out, lse)
            s.weigh(q_out.view(B, 1, heads, 128), lse)
            s.evict(64, sink=1, recent=4)

        keep = [x.clone() for x in (c.k, c.v, c.lens)]
        step()  # plans, workspaces
        for x, y in zip((c.k, c.v, c.lens), keep):
            x.copy_(y)
        s.key_weights.zero_()
        s.key_positions.copy_(torch.arange(c.cap, device="cuda"))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph):
                step()
        seen = []
        for i in range(12):
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            pos.fill_(100 + i)
            c.lens += 1
            graph.replay() if captured else step()
            seen.append([x.clone() for x in (out, lse, c.lens, s.key_weights, s.key_positions)])
        torch.cuda.synchronize()
        assert s.read_status() == 0 and c.lens.tolist() == [64, 15]
        results.append(seen + [[c.k.clone(), c.v.clone()]])
    for a, b in zip(*results):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_encoder_states_and_cross_attention():
    counts, tokens = [70, 0, 33], [5, 2, 40]
    c = Cache(counts, kv_heads=2, heads=6, page=32, device="cuda", seed=64)
    s = CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=0.08)
    g = torch.Generator(device="cuda").manual_seed(65)
    k, v = (torch.randn((sum(counts), 2, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((sum(tokens), 6, 128), generator=g, device="cuda").to(torch.bfloat16)
    cut = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    s.append(None, None, k, v, cu_tokens=cut(counts))
    out, lse = s.cross_attend(q, cu_tokens=cut(tokens))
    torch.cuda.synchronize()
    assert s.read_status() == 0
    k64, v64, q64 = (x.double().cpu().numpy() for x in (k, v, q))
    at = kt = 0
    for m, L in zip(tokens, counts):
        for h in range(6):
            got = out[at:at + m, h].double().cpu().numpy()
            if L == 0:
                assert (got == 0).all() and (lse[at:at + m, h] == -float("inf")).all()
                continue
            x = q64[at:at + m, h] @ k64[kt:kt + L, h // 3].T * 0.08
            p = np.exp(x - x.max(1)[:, None])
            p /= p.sum(1)[:, None]
            want, size = p @ v64[kt:kt + L, h // 3], p @ np.abs(v64[kt:kt + L, h // 3])
            assert (np.abs(got - want) <= (2.0 ** -8 + 1e-3) * size + EPS16 * np.abs(want)).all()
        at, kt = at + m, kt + L


def session_of(seed, lens=(160, 160), **kw):
    c = Cache(list(lens), device="cuda", seed=seed)
    return c, CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=0.1, track=True, num_splits=4, **kw)


def test_a_call_on_another_stream_keeps_its_memory():
    """What a call allocates is not handed out again on the current stream before the call has run."""
    c, s = session_of(66)
    q = torch.randn((2, c.heads, 128), device="cuda").to(torch.bfloat16)
    want = [x.clone() for x in s.cross_attend(q)]
    size = skv.splitkv_cross_workspace_size(c.desc, 2)
    assert size > 0
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    got = s.cross_attend(q, stream=side)
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in others)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_without_a_call_before():
    """The first calls of a session lie in a graph, and eager calls between its replays use the same workspaces."""
    results = []
    for captured in (False, True):
        c, s = session_of(67)
        g = torch.Generator(device="cuda").manual_seed(68)
        q = torch.randn((2, 1, c.heads, 128), generator=g, device="cuda").to(torch.bfloat16)
        out, lse = torch.zeros_like(q), torch.zeros((2, 1, c.heads), device="cuda")

        def step():
            s.decode(q, out, lse)
            s.weigh(q, lse)
            s.evict(30)

        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph):
                step()
        seen = []
        for n in (160, 90):
            s.decode(q, out, lse)
            s.weigh(q, lse)
            s.evict(100)  # (a larger workspace)
            c.lens.fill_(n)
            graph.replay() if captured else step()
            seen += [x.clone() for x in (out, lse, c.lens, s.key_weights)]
        torch.cuda.synchronize()
        assert s.read_status() == 0 and c.lens.tolist() == [30, 30]
        results.append(seen + [c.k.clone(), c.v.clone()])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_a_call_without_tokens():
    c, s = session_of(69)
    none = torch.zeros((0, c.heads, 128), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((0, c.Hkv, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert s.append(torch.zeros((1, 0), dtype=torch.int32, device="cuda"), none, k, k, cu_tokens=cu).shape == none.shape
    out, lse = s.cross_attend(none, cu_tokens=cu)
    assert out.shape == none.shape and lse.shape == (0, c.heads)
