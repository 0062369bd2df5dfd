"""Host-side checks of the operators of drafted trees: refusals happen before any CUDA call (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__

__graft_entry__.build()

import split_kv_paged_splitkv_gb300 as skv  # noqa: E402

A = 1 << 20  # an aligned address that no refused call reads
EINVAL, EUNSUPPORTED, EWORKSPACE = skv.SPLITKV_EINVAL, skv.SPLITKV_EUNSUPPORTED, skv.SPLITKV_EWORKSPACE


def desc(B=2, T=1, Hq=8, Hkv=2, Dk=128, Dv=128, P=16, maxp=8, N=20, fp8=False, shares=0, layout=0):
    return skv.make_desc(B, T, Hq, Hkv, Dk, Dv, P, maxp, N, int(fp8), shares, 1, layout)


def latent(**kw):
    return desc(**{**dict(Hq=128, Hkv=1, Dk=576, Dv=512, shares=1), **kw})


def refused(want, fn, *args, **kw):
    with pytest.raises(skv.SplitKVError) as e:
        fn(*args, **kw)
    assert e.value.status == want and skv.splitkv_last_error(), e.value
    return str(e.value)


# ------------------------------------------------------------------ append with norms

def call_norm(d, **kw):
    a = dict(desc=d, rope=None, positions=A, q=A, k=A, v=A, block_table=A, seq_lens=A, q_out=2 * A, k_pages=A, v_pages=A,
             n_tokens=d.batch * d.q_tokens, stream=0)
    if d.v_shares_k:
        a.update(v=None, v_pages=None)
    a.update(kw)
    return skv.splitkv_append_norm(**a)


@pytest.mark.parametrize("kw", [
    dict(eps=0.0), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(eps=1e39), dict(norm_q=False, q_weight=A),
    dict(norm_k=False, k_weight=A), dict(q_weight=A + 4), dict(k_weight=A + 8), dict(k=None), dict(v_pages=None), dict(q=None),
    dict(q=A + 2), dict(n_tokens=3), dict(n_tokens=-1), dict(k_scale=A, v_scale=A), dict(q_out=A + 256)])
def test_norm_refusals(kw):
    refused(EINVAL, call_norm, desc(), **kw)


def test_norm_refuses_queries_of_latent_caches_and_a_missing_norm():
    assert "norm_q" in refused(EUNSUPPORTED, call_norm, latent())
    refused(EINVAL, call_norm, latent(), norm_q=False, eps=0.0)
    refused(EUNSUPPORTED, call_norm, desc(Dk=64, Dv=64))
    d = desc()
    assert skv._lib.splitkv_append_norm(ctypes.byref(d), None, None, 2, None, None, A, 1024, A, 256, A, 256, A, A, 1.0, None, None,
                                        2 * A, 1024, A, A, None, None, None, 0) == EINVAL


@pytest.mark.parametrize("shape", [(64,), (256,), (4, 128), (2, 128), (8, 64), (1, 128), (8, 1, 128)])
def test_norm_weights_of_other_shapes(shape):
    with pytest.raises(ValueError):
        call_norm(desc(), q_weight=torch.zeros(shape))
    with pytest.raises(ValueError):
        call_norm(desc(), q_weight=torch.zeros((8, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        call_norm(latent(), norm_q=False, k_weight=torch.zeros(576))
    with pytest.raises(ValueError, match="device"):
        call_norm(desc(), k_weight=torch.zeros((2, 128)))


def test_norm_of_no_tokens():
    call_norm(desc(), cu_tokens=A, n_tokens=0, k=None, v=None, q=None, q_out=None, positions=None)


# ------------------------------------------------------------------ commit

def call_commit(d, **kw):
    a = dict(desc=d, path=A, path_lens=A, k_pages=A, v_pages=None if d.v_shares_k else A, block_table=A, seq_lens=A,
             seq_lens_out=A, max_path=4, stream=0)
    a.update(kw)
    return skv.splitkv_tree_commit(**a)


@pytest.mark.parametrize("kw", [
    dict(path=None), dict(path_lens=None), dict(k_pages=None), dict(v_pages=None), dict(block_table=None), dict(seq_lens=None),
    dict(seq_lens_out=None), dict(max_path=0), dict(max_path=-2), dict(k_pages=A + 8), dict(v_pages=A + 4), dict(path=A + 2),
    dict(path_lens=A + 1), dict(cu_tokens=A + 2), dict(key_weights=A + 2), dict(key_positions=A + 1), dict(status=A + 2),
    dict(seq_lens_out=A + 4)])
def test_commit_refusals(kw):
    refused(EINVAL, call_commit, desc(), **kw)


def test_commit_refuses_other_caches_and_arguments():
    refused(EINVAL, call_commit, latent(), v_pages=A)
    refused(EUNSUPPORTED, call_commit, desc(Dk=64, Dv=64))
    refused(EINVAL, call_commit, desc(P=24))
    refused(EINVAL, call_commit, desc(maxp=1 << 27))
    with pytest.raises(TypeError):
        call_commit(desc(), max_path=None)
    with pytest.raises(OverflowError):
        call_commit(desc(), max_path=1 << 31)
    for bad in (torch.zeros((2, 4)), torch.zeros((2, 3), dtype=torch.int32), torch.zeros((3, 5), dtype=torch.int32),
                torch.zeros((2, 4), dtype=torch.int32)):  # the type, too few, rows of another length, the device
        with pytest.raises(ValueError):
            call_commit(desc(), path=bad)


# ------------------------------------------------------------------ tree attention

def call_tree(d, **kw):
    a = dict(desc=d, cu_tokens=None, tree_mask=A, mask_words=1, q=A, k_pages=A, v_pages=None if d.v_shares_k else A, block_table=A,
             seq_lens=A, scale=0.1, out=1 << 40, lse=A, workspace=A, workspace_bytes=1 << 40, n_tokens=d.batch * d.q_tokens, stream=0)
    a.update(kw)
    return skv.splitkv_tree_attend(**a)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(tree_mask=None), dict(k_pages=None), dict(v_pages=None), dict(block_table=None), dict(seq_lens=None),
    dict(out=None), dict(q=A + 8), dict(out=A), dict(out=A + 256), dict(lse=A + 2), dict(cu_tokens=A + 2), dict(tree_mask=A + 2),
    dict(scale=0.0), dict(scale=math.nan), dict(mask_words=0), dict(mask_words=33), dict(mask_words=-1), dict(n_tokens=-1),
    dict(n_tokens=5), dict(n_tokens=1 << 28, cu_tokens=A), dict(k_scale=A, v_scale=A), dict(status=A + 1), dict(v_pages=A + 8),
    dict(workspace=A + 8)])
def test_tree_refusals(kw):
    refused(EINVAL, call_tree, desc(), **kw)


def test_tree_scales():
    refused(EINVAL, call_tree, desc(fp8=True), kv_scale=0.0)
    refused(EINVAL, call_tree, desc(fp8=True), kv_scale=math.inf)
    refused(EINVAL, call_tree, desc(fp8=True), k_scale=A)
    refused(EINVAL, call_tree, desc(fp8=True), k_scale=A + 2, v_scale=A)
    refused(EUNSUPPORTED, call_tree, latent(fp8=True), k_scale=A, v_scale=A)


def test_tree_over_latent_rows():
    refused(EINVAL, call_tree, latent(T=4), cu_tokens=A)
    refused(EINVAL, call_tree, latent(T=4), n_tokens=7)
    refused(EINVAL, call_tree, latent(T=4), v_pages=A)
    for kw in (dict(T=17), dict(Hq=64), dict(P=48), dict(fp8=True, shares=0)):
        refused(EUNSUPPORTED, call_tree, latent(**kw))
        assert skv.splitkv_tree_workspace_size(latent(**kw), latent(**kw).batch * latent(**kw).q_tokens) == 0
    d = latent(T=4, maxp=64, P=64)
    need = skv.splitkv_tree_workspace_size(d, 8)
    assert need > 2 * 4 * 128 * 512 * 4  # more than a split: partial results of every row
    refused(EWORKSPACE, call_tree, d, workspace=None, workspace_bytes=0)
    refused(EWORKSPACE, call_tree, d, workspace_bytes=need - 1)
    lib = skv._lib.splitkv_tree_attend
    for stride in (128 * 576 + 8, 128 * 576 - 8):
        assert lib(ctypes.byref(d), 8, None, A, 1, A, stride, A, None, A, A, 0.1, 1.0, None, None, 1 << 40, None, A, 1 << 40, None,
                   0) == EINVAL


def test_tree_workspaces():
    d = desc(B=1, Hkv=1, maxp=512)
    need = skv.splitkv_tree_workspace_size(d, 1)
    assert need == skv.splitkv_cross_workspace_size(d, 1) > 0
    refused(EWORKSPACE, call_tree, d, workspace=None, workspace_bytes=0)
    refused(EWORKSPACE, call_tree, d, workspace_bytes=need - 1)
    assert skv.splitkv_tree_workspace_size(desc(fp8=True), 2) > 0
    assert skv.splitkv_tree_workspace_size(d, 0) == skv.splitkv_tree_workspace_size(d, -1) == 0
    call_tree(d, cu_tokens=A, n_tokens=0)  # nothing to do, nothing launched
    for stride in (1016, 1025, 1 << 31, 1 << 62, -1024):
        assert skv._lib.splitkv_tree_attend(ctypes.byref(d), 1, None, A, 1, A, stride, A, A, A, A, 0.1, 1.0, None, None, 1 << 40, None,
                                            A, 1 << 40, None, 0) == EINVAL


def test_tree_tensor_arguments():
    d = desc()
    for bad in (torch.zeros((2, 1)), torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32),
                torch.zeros((3, 1), dtype=torch.int64), torch.zeros((2, 1), dtype=torch.int32)):
        with pytest.raises(ValueError):  # the type, too few, rows of another length, the type, the device
            call_tree(d, tree_mask=bad, mask_words=None)
    with pytest.raises(ValueError):  # rows of two words
        call_tree(d, tree_mask=torch.zeros((2, 2), dtype=torch.int32), mask_words=1)
    with pytest.raises(TypeError):
        call_tree(d, mask_words=None)
    with pytest.raises(TypeError):
        call_tree(d, n_tokens=None)
    with pytest.raises(ValueError):
        call_tree(d, out=torch.zeros((2, 8, 64), dtype=torch.bfloat16))


def test_the_norm_struct_is_the_headers():
    assert ctypes.sizeof(skv.splitkv_norm_t) == 40 and skv.splitkv_norm_t.eps.offset == 16
    assert skv.splitkv_norm_t.k_per_head.offset == 32


@pytest.mark.parametrize("name", ["cross_kernel.cuh", "tree_attend.cu", "tree_commit.cu"])
def test_no_read_only_loads_beside_a_running_writer(name):
    """As in the older kernels: what the kernel before may still write is read with plain loads."""
    import os
    import re

    import split_kv_paged_splitkv_gb300._build as build
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert "wait_prerequisites" in text or "cross_kernel.cuh" in text
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", text)
