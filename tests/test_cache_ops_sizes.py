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


# ------------------------------------------------------------------ rows of arrays

INT, FLOAT, BF16, BYTE = torch.int32, torch.float32, torch.bfloat16, torch.uint8


def call_append(d, rope=None, **kw):
    n = d.batch * d.q_tokens
    a = dict(desc=d, rope=rope, positions=A, q=None, k=A, v=A, block_table=A, seq_lens=A, q_out=None, k_pages=A, v_pages=A,
             n_tokens=n, stream=0)
    a.update(kw)
    return skv.splitkv_append(**a)


def call_weights(d, **kw):
    a = dict(desc=d, q=A, k_pages=A, block_table=A, seq_lens=A, lse=A, scale=0.1, kv_scale=1.0, decay=1.0, weights_in=A,
             weights_out=A, stream=0)
    a.update(kw)
    return skv.splitkv_key_weights(**a)


AXES = dict(rope=skv.splitkv_rope_create(128, (24, 20, 20)))
D = dict(B=2, T=2, Hq=8, Hkv=4, maxp=8, N=20)  # 4 tokens; state rows of 128 slots


# an array that is longer than the call needs, in a dimension other than its first: its rows do not begin where the
# kernel, which goes by the descriptor and the number of tokens, looks for them
@pytest.mark.parametrize("call,name,shape,dtype,kw", [
    (call_append, "positions", (3, 5), INT, AXES),
    (call_append, "positions", (15,), INT, AXES),
    (call_append, "positions", (3, 64), INT, AXES),
    (call_append, "block_table", (2, 9), INT, {}),
    (call_append, "key_weights", (2, 4, 144), FLOAT, {}),
    (call_append, "key_weights", (2, 5, 128), FLOAT, {}),
    (call_append, "key_positions", (2, 4, 9, 16), INT, {}),
    (call_append, "k_pages", (20, 4, 32, 128), BF16, {}),
    (call_append, "v_pages", (20, 5, 16, 128), BF16, {}),
    (call_weights, "q", (2, 3, 8, 128), BF16, {}),
    (call_weights, "lse", (2, 3, 8), FLOAT, {}),
    (call_weights, "block_table", (3, 9), INT, {}),
    (call_weights, "weights_in", (3, 4, 144), FLOAT, {}),
    (call_weights, "weights_out", (2, 4, 129), FLOAT, {}),
    (call_evict, "block_table", (2, 16), INT, {}),
    (call_evict, "weights_in", (2, 4, 256), FLOAT, {}),
    (call_evict, "positions_in", (2, 8, 128), INT, {}),
    (call_evict, "weights_out", (1100,), FLOAT, {}),
    (call_evict, "positions_out", (2, 4, 132), INT, {}),
    (call_cross, "block_table", (2, 9), INT, {}),
    (call_cross, "k_pages", (21, 4, 17, 128), BF16, {}),
])
def test_longer_rows_are_refused(call, name, shape, dtype, kw):
    with pytest.raises(ValueError, match=f"{name}.*rows of"):
        call(desc(**D), **{name: torch.zeros(shape, dtype=dtype)}, **kw)


# longer in the first dimension only, or other views of as many elements: the rows lie where the call expects them
@pytest.mark.parametrize("call,name,shape,dtype,kw", [
    (call_append, "positions", (3, 4), INT, AXES),
    (call_append, "positions", (12,), INT, AXES),
    (call_append, "positions", (4, 4), INT, AXES),
    (call_append, "positions", (64,), INT, {}),           # one axis: the first four
    (call_append, "positions", (1, 64), INT, {}),
    (call_append, "block_table", (5, 8), INT, {}),
    (call_append, "block_table", (16,), INT, {}),
    (call_append, "seq_lens", (9,), INT, {}),
    (call_append, "cu_tokens", (9,), INT, {}),
    (call_append, "key_weights", (3, 4, 128), FLOAT, {}),
    (call_append, "key_weights", (12, 128), FLOAT, {}),
    (call_append, "key_positions", (7, 4, 8, 16), INT, {}),
    (call_append, "k_pages", (30, 4, 16, 128), BF16, {}),
    (call_append, "k_pages", (20, 16, 4, 128), BF16, {}),
    (call_weights, "q", (3, 2, 8, 128), BF16, {}),
    (call_weights, "q", (4, 8, 128), BF16, {}),
    (call_weights, "lse", (4, 8), FLOAT, {}),
    (call_weights, "weights_out", (8, 128), FLOAT, {}),
    (call_evict, "seq_lens_out", (3,), INT, {}),
    (call_cross, "out", (9, 8, 128), BF16, {}),
    (call_cross, "lse", (9, 8), FLOAT, {}),
])
def test_rows_in_place_are_taken(call, name, shape, dtype, kw):
    with pytest.raises(ValueError, match=f"{name} is not on the current CUDA device"):
        call(desc(**D), **{name: torch.zeros(shape, dtype=dtype)}, **kw)


def test_one_row_may_be_longer():
    d = desc(B=1, T=1, Hq=4, Hkv=1, maxp=8)
    for call, name, shape, dtype in ((call_append, "block_table", (1, 9), INT), (call_append, "key_weights", (1, 1, 999), FLOAT),
                                     (call_evict, "weights_in", (200,), FLOAT), (call_cross, "block_table", (64,), INT)):
        with pytest.raises(ValueError, match=f"{name} is not on the current CUDA device"):
            call(d, **{name: torch.zeros(shape, dtype=dtype)})


# ------------------------------------------------------------------ the documented bound of a workspace

def test_cross_workspace_bound():
    """No call needs more than the header says, and some need all of it."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "splitkv.h")) as f:
        bound = re.search(r"splitkv_cross_workspace_size bytes \(0: may be NULL;\s*\*?\s*([\d,]+)\s*\*?\s*at\s*\*?\s*most\)", f.read())
    assert bound, "the header names the bound in bytes"
    most = 0
    for kv in (1, 2, 8, 16, 608, 65535):
        for group in (1, 4, 32, 300):
            for batch in (1, 3, 600, 5000):
                d = desc(B=batch, Hq=kv * group, Hkv=kv, maxp=1 << 12, N=16)
                for n in (1, 5, 128, 4000, 1 << 17):
                    most = max(most, skv.splitkv_cross_workspace_size(d, n))
    assert most == int(bound.group(1).replace(",", ""))


@pytest.mark.parametrize("shape", [(4, 3), (2, 6), (6, 2), (12, 1, 1), (1, 4, 3)])
def test_positions_go_by_axis(shape):
    """[tokens][axes] has as many elements as [axes][tokens], in another order."""
    taken = shape == (12, 1, 1)  # (no rows of its own: taken as it lies)
    with pytest.raises(ValueError, match="positions is not on" if taken else "positions.*rows of"):
        call_append(desc(**D), positions=torch.zeros(shape, dtype=INT), **AXES)
