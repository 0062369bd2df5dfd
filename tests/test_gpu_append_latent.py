"""GPU tests of appends to latent caches whose rotated columns lie anywhere in the row: the queries' other columns are
copied by units of their own."""
import pytest

from _cache_ops import Cache
from _support import need_gpu
from test_gpu_append_norm import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("heads,lens,counts", [(1, [70, 6], [9, 2]), (5, [40, 0, 300], [33, 0, 1]), (40, [120], [110])])
@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("rot,offset", [(64, 512), (64, 0), (16, 288), (128, 448), (128, 0), (112, 16), (48, 496)])
def test_any_rotated_columns(rot, offset, pairing, heads, lens, counts):
    for dtype, which in (("bf16", "k"), ("e4m3", "")):
        c = Cache(lens, kv_heads=1, heads=heads, page=64, dim=576, v_dim=512, shares=True, dtype=dtype, device="cuda", seed=rot)
        run(c, counts, rot=rot, offset=offset, pairing=pairing, which=which, weights=which, pad=2)


@pytest.mark.parametrize("heads,lens,counts", [(3, [70], [9]), (40, [120], [110])])
def test_in_place_and_without_rotation(heads, lens, counts):
    c = Cache(lens, kv_heads=1, heads=heads, page=64, dim=576, v_dim=512, shares=False, device="cuda", seed=5)
    run(c, counts, rot=64, offset=512, which="k", weights="k", in_place=True, pad=1)
    run(c, counts, rope=False, which="k", weights="", pad=1)
