"""Speculative decoding over a paged cache as its operators are used together: prompts appended with norms, then steps of a
drafted tree appended, attended and committed, each against the plain 64-bit implementation on the same state.  Tolerances
are those of the operators' own tests."""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import EPS16, Cache, rotated
from _support import LSE_TOL, OUT_TOL, need_gpu
from split_kv_paged_splitkv_gb300.runner import CacheSession

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def draft(rng, n):
    """(parents, [n][n] sees, depths) of a random tree."""
    parents = [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]
    sees, depth = np.zeros((n, n), bool), np.zeros(n, int)
    for i, p in enumerate(parents):
        if p >= 0:
            sees[i], depth[i] = sees[p], depth[p] + 1
        sees[i, i] = True
    return parents, sees, depth


def words(sees, n_words):
    bits = np.zeros((len(sees), 32 * n_words), bool)
    bits[:, :len(sees)] = sees
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def attend(q, k, v, sees, scale):
    """q [n][Hq][D], the keys before the tree and the drafted ones k, v [L][Hkv][..] in 64 bits: (out, lse)."""
    n, L, G = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    seen = np.concatenate([np.ones((n, L - n), bool), sees], 1)
    out, lse = np.zeros(q.shape[:2] + v.shape[2:]), np.zeros(q.shape[:2])
    for h in range(q.shape[1]):
        x = np.where(seen, q[:, h] @ k[:, h // G].T * scale, -np.inf)
        top = x.max(1)
        lse[:, h] = top + np.log(np.exp(x - top[:, None]).sum(1))
        out[:, h] = np.exp(x - lse[:, h][:, None]) @ v[:, h // G]
    return out, lse


@pytest.mark.parametrize("dtype,layout", [("bf16", "HND"), ("bf16", "NHD"), ("e4m3", "HND"), ("e4m3", "NHD")])
def test_steps_of_drafted_trees(dtype, layout):
    B, Hkv, heads, scale = 3, 2, 8, 128 ** -0.5
    c = Cache([260] * B, kv_heads=Hkv, heads=heads, dtype=dtype, layout=layout, device="cuda", seed=70)
    kv_scale = 1 / 64 if dtype == "e4m3" else 1.0
    freqs = [1e4 ** (-i / 64) for i in range(64)]
    g = torch.Generator(device="cuda").manual_seed(71)
    wq, wk = 1 + 0.2 * torch.randn(128, generator=g, device="cuda"), 1 + 0.2 * torch.randn((Hkv, 128), generator=g, device="cuda")
    s = CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=scale, rope=skv.splitkv_rope_create(128, freqs=freqs),
                     kv_scale=kv_scale, num_splits=3, track=True, q_norm=wq, k_norm=wk)
    rng = np.random.default_rng(72)
    c.lens.zero_()
    lens = [0] * B

    def normed(x, w):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w.double().cpu().numpy()

    def append(counts, positions):
        n = sum(counts)
        q, k, v = (torch.randn((n, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (heads, Hkv, Hkv))
        for b, m in enumerate(counts):
            lens[b] += m
        c.lens.copy_(torch.tensor(lens))
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        pos = np.concatenate(positions)[None].astype(np.int32)
        out = s.append(torch.from_numpy(pos).cuda(), q, k, v, cu_tokens=cu)
        want = rotated(normed(q.double().cpu().numpy(), wq), pos, freqs, (64,), 0, 0)
        assert (np.abs(out.double().cpu().numpy() - want) <= EPS16 * np.abs(want) + 1e-5).all()
        want_k = rotated(normed(k.double().cpu().numpy(), wk), pos, freqs, (64,), 0, 0)
        return out, cu, want_k

    append([50, 3, 120], [np.arange(50), np.arange(3), np.arange(120)])
    history = [list(range(n)) for n in (50, 3, 120)]  # the positions that are kept
    moved = 0
    for step in range(5):
        counts = [int(x) for x in rng.integers(1, 40, B)]
        trees = [draft(rng, n) for n in counts]
        before = list(lens)
        q, cu, want_k = append(counts, [before[b] + trees[b][2] for b in range(B)])
        mask = np.concatenate([words(t[1], 2) for t in trees])
        out, lse = s.tree_attend(q, torch.from_numpy(mask).cuda(), cu_tokens=cu)
        kp, vp = c.values(c.k) * kv_scale, c.values(c.v) * kv_scale
        got, got_l, q64, at = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy(), 0
        paths = []
        for b, n in enumerate(counts):
            k, v = c.rows(kp, b, lens[b]), c.rows(vp, b, lens[b])
            err = np.abs(k[before[b]:] - want_k[at:at + n])
            assert (err <= (2.0 ** -4 if dtype == "e4m3" else EPS16) * np.abs(want_k[at:at + n]) + 1e-4).all()
            want, want_l = attend(q64[at:at + n], k, v, trees[b][1], scale)
            assert np.abs(got[at:at + n] - want).max() <= OUT_TOL and np.abs(got_l[at:at + n] - want_l).max() <= LSE_TOL
            path = [0]  # a way down the tree
            while True:
                children = [i for i, p in enumerate(trees[b][0]) if p == path[-1]]
                if not children or rng.random() < 0.2:
                    break
                path.append(int(rng.choice(children)))
            paths.append(path)
            moved += sum(i != p for i, p in enumerate(path))
            at += n
        width = max(len(p) for p in paths)
        s.commit(torch.tensor([p + [0] * (width - len(p)) for p in paths], dtype=torch.int32, device="cuda"),
                 torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"), cu_tokens=cu)
        new_k, new_v, state = c.values(c.k) * kv_scale, c.values(c.v) * kv_scale, s.key_positions.cpu().numpy()
        for b, path in enumerate(paths):
            keep = list(range(before[b])) + [before[b] + i for i in path]
            history[b] += [before[b] + int(trees[b][2][i]) for i in path]
            for new, old in ((new_k, kp), (new_v, vp)):
                assert np.array_equal(c.rows(new, b, len(keep)), c.rows(old, b, lens[b])[keep])
            lens[b] = len(keep)
            assert (state[b, :, :lens[b]] == history[b]).all()
            assert history[b] == list(range(lens[b]))  # a committed sequence is like one decoded token by token
        assert c.lens.tolist() == lens
    assert moved > 0 and s.read_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_steps_over_latent_rows(dtype):
    B, T, scale = 2, 8, 576 ** -0.5
    c = Cache([200] * B, kv_heads=1, heads=128, page=64, dim=576, v_dim=512, shares=True, dtype=dtype, tokens=T, device="cuda",
              seed=73)
    kv_scale = 1 / 64 if dtype == "e4m3" else 1.0
    g = torch.Generator(device="cuda").manual_seed(74)
    s = CacheSession(c.desc, c.k, None, c.table, c.lens, scale=scale, rope=skv.splitkv_rope_create(64, rot_offset=512, pairing=1),
                     kv_scale=kv_scale, num_splits=2, k_norm=True)
    rng = np.random.default_rng(75)
    c.lens.copy_(torch.tensor([100, 9]))
    lens = [100, 9]
    for step in range(3):
        lens = [n + T for n in lens]
        c.lens.copy_(torch.tensor(lens))
        trees = [draft(rng, T) for _ in range(B)]
        q, k = (torch.randn((B * T, h, 576), generator=g, device="cuda").to(torch.bfloat16) for h in (128, 1))
        pos = np.concatenate([lens[b] - T + trees[b][2] for b in range(B)])[None].astype(np.int32)
        q = s.append(torch.from_numpy(pos).cuda(), q, k, None)
        out, lse = s.tree_attend(q, torch.from_numpy(np.concatenate([words(t[1], 1) for t in trees])).cuda())
        kp = c.values(c.k) * kv_scale
        for b in range(B):
            rows = c.rows(kp, b, lens[b])
            at = slice(b * T, (b + 1) * T)
            want, want_l = attend(q[at].double().cpu().numpy(), rows, rows[..., :512], trees[b][1], scale)
            assert np.abs(out[at].double().cpu().numpy() - want).max() <= OUT_TOL
            assert np.abs(lse[at].double().cpu().numpy() - want_l).max() <= LSE_TOL
        s.commit(torch.tensor([[0, 1, 3], [0, 2, 0]], dtype=torch.int32, device="cuda"),
                 torch.tensor([3, 2], dtype=torch.int32, device="cuda"))
        lens = [lens[0] - T + 3, lens[1] - T + 2]
        assert c.lens.tolist() == lens
        new = c.values(c.k) * kv_scale
        for b, path in enumerate(([0, 1, 3], [0, 2])):
            first = lens[b] - len(path)
            assert np.array_equal(c.rows(new, b, lens[b])[first:], c.rows(kp, b, first + T)[[first + i for i in path]])
    assert s.read_status() == 0


def test_a_captured_step_of_the_whole():
    """append, tree attention and commit in one graph, replayed while the lengths on the device grow: as the eager calls."""
    B, Hkv, heads, n = 2, 2, 8, 6
    results = []
    for captured in (False, True):
        c = Cache([160] * B, kv_heads=Hkv, heads=heads, tokens=n, device="cuda", seed=76)
        s = CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=0.1, rope=skv.splitkv_rope_create(128), track=True, num_splits=4,
                         q_norm=True, k_norm=True)
        g = torch.Generator(device="cuda").manual_seed(77)
        c.lens.copy_(torch.tensor([60, 3]))
        q, k, v = (torch.zeros((B * n, h, 128), dtype=torch.bfloat16, device="cuda") for h in (heads, Hkv, Hkv))
        pos = torch.zeros((1, B * n), dtype=torch.int32, device="cuda")
        mask = torch.zeros((B * n, 1), dtype=torch.int32, device="cuda")
        path = torch.zeros((B, n), dtype=torch.int32, device="cuda")
        count = torch.zeros(B, dtype=torch.int32, device="cuda")

        def step():
            c.lens.add_(n)
            turned = s.append(pos, q, k, v)
            out = s.tree_attend(turned, mask)
            s.commit(path, count)
            return out

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph):
                held = step()
        seen = []
        rng = np.random.default_rng(78)
        for i in range(6):
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            trees = [draft(rng, n) for _ in range(B)]
            mask.copy_(torch.from_numpy(np.concatenate([words(t[1], 1) for t in trees])))
            pos.copy_(torch.from_numpy(np.concatenate([t[2] for t in trees])[None] + 10 * i))
            kept = [sorted({0, *rng.integers(0, n, 3).tolist()}) for _ in range(B)]
            path.copy_(torch.tensor([p + [0] * (n - len(p)) for p in kept]))
            count.copy_(torch.tensor([len(p) for p in kept]))
            torch.cuda.synchronize()
            if captured:
                graph.replay()
                out = held
            else:
                out = step()
            torch.cuda.synchronize()
            seen += [x.clone() for x in out] + [c.lens.clone(), c.k.clone(), c.v.clone()]
        assert s.read_status() == 0
        results.append(seen)
    assert all(torch.equal(x, y) for x, y in zip(*results))


def test_two_sessions_on_two_streams_at_once():
    """Calls that overlap on the GPU, each with its own workspace: as one after the other."""
    cases = []
    for seed in (79, 80):
        c = Cache([3000, 700], kv_heads=2, heads=16, device="cuda", seed=seed)
        s = CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=0.09)
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn((30, 16, 128), generator=g, device="cuda").to(torch.bfloat16)
        mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (30, 1), generator=g, device="cuda", dtype=torch.int32)
        cu = torch.tensor([0, 20, 30], dtype=torch.int32, device="cuda")
        cases.append((s, q, mask, cu, torch.cuda.Stream()))
    torch.cuda.synchronize()
    alone = [s.tree_attend(q, mask, cu) for s, q, mask, cu, _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        both = [s.tree_attend(q, mask, cu, stream=st) for s, q, mask, cu, st in cases]
        torch.cuda.synchronize()
        for x, y in zip(alone, both):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_a_call_without_tokens():
    c = Cache([20, 30], device="cuda", seed=81)
    s = CacheSession(c.desc, c.k, c.v, c.table, c.lens, scale=0.1, q_norm=True)
    none = torch.zeros((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = s.tree_attend(none, torch.zeros((0, 1), dtype=torch.int32, device="cuda"), cu_tokens=cu)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8) and s.read_status() == 0
