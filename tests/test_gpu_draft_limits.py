"""GPU tests of the operators of drafted trees at their limits: pools beyond 2^32 bytes, token offsets that the header
rules out, masks and paths of any bits, and more items than 32 bits count."""
import numpy as np
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import Cache
from _support import need_gpu
from test_gpu_cache_far import moved_far
from test_gpu_cross_offsets import DEALS, Guarded, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("kw", [dict(), dict(layout="NHD"), dict(dtype="e4m3"), dict(dtype="e4m3", layout="NHD"),
                                dict(kv_heads=1, heads=128, dim=576, v_dim=512, page=64),
                                dict(kv_heads=1, heads=128, dim=576, v_dim=512, page=64, dtype="e4m3", shares=True)])
def test_pools_beyond_32_bits(kw):
    c = Cache([700, 90, 333], device="cuda", seed=90, **kw)
    far = moved_far(c)
    latent, T = c.dim != 128, 12
    results = []
    for x in (c, far):
        d = skv.make_desc(x.B, T, x.heads, x.Hkv, x.dim, x.v_dim, x.P, x.width, x.N, x.desc.kv_dtype, int(x.shares),
                          skv.SPLITKV_COMBINE_SEPARATE, x.desc.kv_layout)
        g = torch.Generator(device="cuda").manual_seed(91)
        q, k, v = (torch.randn((3 * T, h, m), generator=g, device="cuda").to(torch.bfloat16)
                   for h, m in ((x.heads, x.dim), (x.Hkv, x.dim), (x.Hkv, x.v_dim)))
        pos = torch.randint(0, 1 << 20, (1, 3 * T), generator=g, device="cuda", dtype=torch.int32)
        mask = torch.randint(0, 1 << T, (3 * T, 1), generator=g, device="cuda", dtype=torch.int32)
        w = torch.rand((x.B, x.Hkv, x.cap), generator=g, device="cuda")
        p = torch.randint(0, 1000, (x.B, x.Hkv, x.cap), generator=g, device="cuda", dtype=torch.int32)
        out, lse = torch.empty((3 * T, x.heads, x.v_dim), dtype=torch.bfloat16, device="cuda"), torch.empty((3 * T, x.heads), device="cuda")
        ws = torch.empty(max(16, skv.splitkv_tree_workspace_size(d, 3 * T)), dtype=torch.uint8, device="cuda")
        st, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros_like(x.lens)
        skv.splitkv_append_norm(d, skv.splitkv_rope_create(64, rot_offset=512 if latent else 0), pos, q, k, None if x.shares else v,
                                x.table, x.lens, q, x.k, x.v, norm_q=not latent, kv_scale=0.01, key_weights=w, key_positions=p,
                                status=st)
        skv.splitkv_tree_attend(d, None, mask, q, x.k, x.v, x.table, x.lens, 0.05, out, lse, ws, kv_scale=0.01, status=st) \
            if not (latent and not x.shares and x.dtype == "e4m3") else None
        skv.splitkv_tree_commit(d, torch.tensor([[1, 5, 11], [0, 2, 3], [7, 8, 9]], dtype=torch.int32, device="cuda"),
                                torch.tensor([3, 2, 3], dtype=torch.int32, device="cuda"), x.k, x.v, x.table, x.lens, lens,
                                key_weights=w, key_positions=p, status=st)
        torch.cuda.synchronize()
        assert int(st) == 0 and lens.tolist() == [691, 80, 324]
        results.append([q, out, lse, w, p] + [y[x.N - c.N:] for y in (x.k, x.v) if y is not None])
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert not far.k[:far.N - c.N].any() and (far.v is None or not far.v[:far.N - c.N].any())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("deal", DEALS)
def test_wrong_offsets_write_nothing_else(deal, dtype):
    """The tree's kernel clamps tokens as cross attention does; sequences with fewer keys than tokens count as empty."""
    lens, counts, kv, heads = DEALS[deal]
    lens = [max(a, b) for a, b in zip(lens, counts)]
    c = Cache(lens, kv_heads=kv, heads=heads, dtype=dtype, device="cuda", seed=92)
    n = sum(counts)
    q = torch.randn((n, heads, 128), device="cuda").to(torch.bfloat16)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, 3), device="cuda", dtype=torch.int32)
    for cu in offsets(counts, n, np.random.default_rng(93)):
        out, ls = Guarded(q.numel(), torch.bfloat16, 0), Guarded(n * heads, torch.float32, 0)
        size = skv.splitkv_tree_workspace_size(c.desc, n)
        ws = Guarded(max(size, 16), torch.uint8, 0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        skv.splitkv_tree_attend(c.desc, torch.tensor(cu, dtype=torch.int32, device="cuda"), mask, q, c.k, c.v, c.table, c.lens, 0.1,
                                out.view.view(q.shape), ls.view.view(n, heads), ws.view if size else None, kv_scale=0.01,
                                status=status)
        assert status.item() in (0, skv.SPLITKV_DEVERR_SEQLEN)
        assert out.untouched() and ls.untouched() and ws.untouched()
        assert torch.isfinite(out.view).all() and not torch.isnan(ls.view).any()


def test_wrong_offsets_and_paths_of_a_commit():
    """Any offsets, lengths and paths: nothing but the sequences' own rows is written, or the status says why."""
    rng = np.random.default_rng(94)
    c = Cache([70, 40, 9, 130], device="cuda", seed=94)
    own = torch.zeros(c.N, dtype=torch.bool, device="cuda")
    for b, L in enumerate(c.lens_host):
        own[c.table[b, :-(-L // c.P)].long()] = True
    k0, v0 = c.k.clone(), c.v.clone()
    for _ in range(40):
        cu = torch.from_numpy(rng.choice([-(1 << 31), -5, 0, 3, 9, 20, 40, (1 << 31) - 1], 5).astype(np.int32)).cuda()
        path = torch.from_numpy(rng.choice([-(1 << 31), -1, 0, 1, 2, 5, 19, 60, (1 << 31) - 1], (4, 6)).astype(np.int32)).cuda()
        path[0] = torch.arange(6)
        n = torch.from_numpy(rng.choice([-(1 << 31), -1, 0, 1, 3, 6, 7, (1 << 31) - 1], 4).astype(np.int32)).cuda()
        out = Guarded(4, torch.int32, 0)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        skv.splitkv_tree_commit(c.desc, path, n, c.k, c.v, c.table, c.lens, out.view, cu_tokens=cu, status=st)
        torch.cuda.synchronize()
        assert int(st) in (0, 2, 8, 10) and out.untouched()
        assert ((out.view >= 0) & (out.view <= c.lens)).all()
        assert torch.equal(c.k[~own], k0[~own]) and torch.equal(c.v[~own], v0[~own])


@pytest.mark.parametrize("heads,kv,tokens", [(1, 1, [3, 0, 40]), (8, 4, [2500, 0, 3300])])
def test_wrong_offsets_of_an_append(heads, kv, tokens):
    """Both kinds of kernels: tokens of no sequence leave everything as it is, others go to a slot or to the status."""
    n = sum(tokens)
    c = Cache([max(t, 1) + 20 for t in tokens], kv_heads=kv, heads=heads, device="cuda", seed=95)
    x = torch.randn((n, heads + 2 * kv, 128), device="cuda").to(torch.bfloat16)
    own = torch.zeros(c.N, dtype=torch.bool, device="cuda")
    own[c.table.flatten().long()] = True
    k0 = c.k.clone()
    for cu in offsets(tokens, n, np.random.default_rng(96)):
        out = Guarded(n * heads * 128, torch.bfloat16, 0)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        skv.splitkv_append_norm(c.desc, skv.splitkv_rope_create(128), torch.arange(n, dtype=torch.int32, device="cuda").view(1, n),
                                x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], c.table, c.lens,
                                out.view.view(n, heads, 128), c.k, c.v, cu_tokens=torch.from_numpy(cu.astype(np.int32)).cuda(), status=st)
        torch.cuda.synchronize()
        assert int(st) in (0, skv.SPLITKV_DEVERR_SEQLEN) and out.untouched() and torch.isfinite(out.view).all()
        assert torch.equal(c.k[~own], k0[~own])


def test_more_pieces_than_32_bits_count():
    """One token, which the offsets give to every other one of 240,000 sequences of 608 heads."""
    B, heads, P = 240000, 608, 4112  # 33 key blocks
    k = torch.randn((1, heads, P, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.rand((1, heads, P, 128), device="cuda").to(torch.bfloat16)
    d = skv.make_desc(B, 1, heads, heads, 128, 128, P, 1, 1)
    q = torch.randn((1, heads, 128), device="cuda").to(torch.bfloat16)
    out, ls = Guarded(q.numel(), torch.bfloat16, 0), Guarded(heads, torch.float32, 0)
    size = skv.splitkv_tree_workspace_size(d, 1)
    ws = Guarded(size, torch.uint8, 0)
    skv.splitkv_tree_attend(d, torch.from_numpy((np.arange(B + 1) % 2).astype(np.int32)).cuda(),
                            torch.ones((1, 1), dtype=torch.int32, device="cuda"), q, k, v,
                            torch.zeros((B, 1), dtype=torch.int32, device="cuda"),
                            torch.full((B,), P, dtype=torch.int32, device="cuda"), 0.1, out.view.view(1, heads, 128),
                            ls.view.view(1, heads), ws.view)
    torch.cuda.synchronize()
    assert out.untouched() and ls.untouched() and ws.untouched()
    assert torch.isfinite(out.view).all() and out.view.abs().max() <= 1 and not torch.isnan(ls.view).any()
