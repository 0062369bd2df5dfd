"""GPU tests of the norms that a session is told to take and not to take."""
import pytest
import torch

import split_kv_paged_splitkv_gb300 as skv
from _cache_ops import Cache
from _support import need_gpu
from split_kv_paged_splitkv_gb300.runner import CacheSession
from test_gpu_append_norm_values import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("q_norm,k_norm", [(False, False), (False, None), (None, False), (False, True), (True, False)])
def test_a_session_that_takes_no_norm(q_norm, k_norm):
    c = Cache([40], device="cuda", seed=24)
    q, k, v = inputs(c, 40, 25)
    rope = skv.splitkv_rope_create(128)
    pos = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    got = []
    for qn, kn in ((q_norm, k_norm), (q_norm or None, k_norm or None)):
        pools = torch.zeros_like(c.k), torch.zeros_like(c.v)
        s = CacheSession(c.desc, *pools, c.table, c.lens, scale=0.1, rope=rope, q_norm=qn, k_norm=kn)
        got.append((s.append(pos, q, k, v, cu_tokens=cu), *pools))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    s.k_pages.zero_(), s.v_pages.zero_()
    s.q_norm, s.k_norm = q_norm, k_norm  # (changed later)
    for a, b in zip((s.append(pos, q, k, v, cu_tokens=cu), s.k_pages, s.v_pages), got[0]):
        assert torch.equal(a, b)


def test_a_latent_session_whose_queries_take_no_norm():
    c = Cache([20], kv_heads=1, heads=128, page=64, dim=576, v_dim=512, shares=True, device="cuda", seed=26)
    s = CacheSession(c.desc, c.k, None, c.table, c.lens, scale=0.1, q_norm=False, k_norm=True)
    x = torch.randn((20, 129, 576), device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    out = s.append(torch.zeros((1, 20), dtype=torch.int32, device="cuda"), x[:, :128], x[:, 128:], None, cu_tokens=cu)
    torch.cuda.synchronize()
    assert torch.equal(out, x[:, :128]) and s.read_status() == 0
