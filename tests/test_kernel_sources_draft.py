"""The rules of the kernels' sources for the kernel that cross attention and drafted trees share, and for the commit (no GPU
needed)."""
import re

import pytest

from test_kernel_sources import code


@pytest.mark.parametrize("name", ["cross_kernel.cuh", "tree_commit.cu"])
def test_no_read_only_loads_beside_a_running_writer(name):
    text = code(name)
    assert "wait_prerequisites" in text
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", text)


def test_a_barrier_that_both_row_blocks_wait_for_has_both_in_every_turn():
    """B may be behind A by any number of pieces that it has no part in, so it waits for no barrier that A also turns in
    those: of A's, for the exponents (pieces of both) and for the joined results (likewise)."""
    text = code("cross_kernel.cuh")
    softmax = text[text.index("const int t = warp >> 2;"):]
    assert sorted(set(re.findall(r"wait_for\(bar\((\w+)( \+ \w+)?\)", softmax))) == [
        ("B_DOWN", ""), ("B_JOINED", ""), ("B_ML", ""), ("B_O", " + 1"), ("B_O", " + t"), ("B_Q", " + t"), ("B_S", " + t")]
    assert re.search(r"if \(FP8 && two\) mbar_arrive\(bar\(B_DOWN\)\)", softmax)
    assert re.search(r"if \(FP8 && t == 1 && two\) {\s*ok = __all_sync\(kFull, wait_for\(bar\(B_DOWN\)", softmax)
