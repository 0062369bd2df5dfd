"""Host-side checks of the sizes that the cache operators are given (no GPU needed).

Tensors on the CPU stand for what is on the device: sizes are looked at before the device, so a refusal names
the size where it is wrong and the device where it is right.
"""
import pytest
import torch

import __graft_entry__

__graft_entry__.build()

import split_kv_paged_splitkv_gb300 as skv  # noqa: E402
from test_cache_ops_host import A, call_cross, call_evict, desc  # noqa: E402


# ------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("given", [-1, -(1 << 40), 257, 1 << 40])
@pytest.mark.parametrize("call", [call_cross, call_evict])
def test_workspace_bytes_beyond_the_workspace(call, given):
    """A count that the tensor does not hold would let the kernels write behind it."""
    with pytest.raises(ValueError, match="workspace_bytes"):
        call(desc(), workspace=torch.zeros(256, dtype=torch.uint8, device="meta"), workspace_bytes=given)


@pytest.mark.parametrize("call", [call_cross, call_evict])
def test_workspace_bytes_of_an_address_are_not_negative(call):
    with pytest.raises(ValueError, match="workspace_bytes"):
        call(desc(), workspace=A, workspace_bytes=-1)


@pytest.mark.parametrize("call", [call_cross, call_evict])
def test_workspace_bytes_within_the_workspace(call):
    for given in (0, 256, None):
        with pytest.raises(ValueError, match="not on the current CUDA device"):
            call(desc(), workspace=torch.zeros(256, dtype=torch.uint8), workspace_bytes=given)
