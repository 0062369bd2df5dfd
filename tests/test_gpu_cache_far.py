"""GPU tests of the cache operators in pools beyond 2^32 bytes, and of calls on two streams at once."""
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import Cache
from _support import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def moved_far(c):
    """The same cache with its pages at the end of pools of more than 2^32 bytes."""
    per_page = c.k[0].numel() * c.k.element_size()
    n = (1 << 32) // per_page + 5000
    far = Cache.__new__(Cache)
    far.__dict__.update(c.__dict__)

    def pool(x):
        if x is None:
            return None
        y = torch.zeros((n,) + x.shape[1:], dtype=x.dtype, device="cuda")
        y[n - c.N:] = x
        return y

    far.k, far.v, far.N = pool(c.k), pool(c.v), n
    far.table = c.table + (n - c.N)
    far.desc = skv.make_desc(c.B, 1, c.heads, c.Hkv, c.dim, c.v_dim, c.P, c.width, n, c.desc.kv_dtype, int(c.shares),
                             skv.SPLITKV_COMBINE_SEPARATE, c.desc.kv_layout)
    return far


def life(c, stream=None, seed=0):
    """Append, weigh, evict and cross attention; everything that they write."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    latent = c.dim != 128

    def rows(heads, dim):
        return torch.randn((c.B, heads, dim), generator=g, device="cuda").to(torch.bfloat16)

    q, k, v = rows(c.heads, c.dim), rows(c.Hkv, c.dim), None if c.shares else rows(c.Hkv, c.v_dim)
    w = torch.rand((c.B, c.Hkv, c.cap), generator=g, device="cuda")
    kpos = torch.arange(c.cap, dtype=torch.int32, device="cuda").expand(c.B, c.Hkv, -1).contiguous()
    pos = torch.randint(0, 1 << 20, (1, c.B), generator=g, device="cuda", dtype=torch.int32)
    lse = torch.full((c.B, 1, c.heads), 3.0, device="cuda")
    rope = skv.splitkv_rope_create(64, rot_offset=512 if latent else 0)
    q_out, out, lens_out = torch.empty_like(q), torch.zeros_like(q), torch.zeros_like(c.lens)
    cross_lse, status = torch.zeros((c.B, c.heads), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(skv.splitkv_evict_workspace_size(c.desc, 100), dtype=torch.uint8, device="cuda")
    cross = not latent and c.dtype == "bf16"
    cross_ws = torch.zeros(max(16, skv.splitkv_cross_workspace_size(c.desc, c.B)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def run():
        skv.splitkv_append(c.desc, rope, pos, q, k, v, c.table, c.lens, q_out, c.k, c.v, kv_scale=0.01, key_weights=w,
                           key_positions=kpos, status=status, stream=stream)
        if not latent:
            skv.splitkv_key_weights(c.desc, q_out, c.k, c.table, c.lens, lse, 0.02, 1.0, 0.5, w, w, status=status, stream=stream)
        skv.splitkv_evict(c.desc, 100, 4, 20, c.k, c.v, c.table, c.lens, w, kpos, w, kpos, lens_out, ws, status=status,
                          stream=stream)
        if cross:
            skv.splitkv_cross_attend(c.desc, None, q_out, c.k, c.v, c.table, lens_out, 0.1, out, cross_lse, cross_ws,
                                     status=status, stream=stream)

    run.state = [q_out, w, kpos, lens_out, out, cross_lse, status]
    return run


@pytest.mark.parametrize("kw", [dict(), dict(layout="NHD"), dict(dtype="e4m3"),
                                dict(kv_heads=1, heads=16, dim=576, v_dim=512, page=64),
                                dict(kv_heads=1, heads=16, dim=576, v_dim=512, page=64, dtype="e4m3", shares=True)])
def test_pools_beyond_32_bits(kw):
    c = Cache([700, 90, 333], device="cuda", seed=61, **kw)
    far = moved_far(c)
    results = []
    for x in (c, far):
        run = life(x)
        run()
        torch.cuda.synchronize()
        results.append(run.state + [p[x.N - c.N:] for p in (x.k, x.v) if p is not None])
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert not far.k[:far.N - c.N].any() and (far.v is None or not far.v[:far.N - c.N].any())
    assert int(results[0][6]) == 0 and results[0][3].tolist() == [100, 90, 100]


def test_two_streams_at_once():
    """Two caches, each on its own stream with its own workspaces: the results of one after the other."""
    lens = [[3000, 200], [1500, 900]]

    def start(i, stream=None):
        c = Cache(lens[i], device="cuda", seed=62 + i)
        run = life(c, stream, seed=i)
        return run, run.state + [c.k, c.v]

    alone = []
    for i in range(2):
        run, results = start(i)
        run()
        torch.cuda.synchronize()
        alone.append(results)
    for _ in range(5):
        started = [start(i, torch.cuda.Stream()) for i in range(2)]
        torch.cuda.synchronize()
        for run, _ in started:
            run()
        torch.cuda.synchronize()
        for (_, results), want in zip(started, alone):
            for a, b in zip(results, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
