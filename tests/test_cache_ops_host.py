"""Host-side checks of the cache operators: refusals happen before any CUDA call (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

import __graft_entry__

__graft_entry__.build()

import split_kv_paged_splitkv_gb300 as skv  # noqa: E402

A = 1 << 20  # an aligned address that no refused call reads
EINVAL, EUNSUPPORTED, EWORKSPACE = skv.SPLITKV_EINVAL, skv.SPLITKV_EUNSUPPORTED, skv.SPLITKV_EWORKSPACE


def desc(B=2, T=1, Hq=8, Hkv=2, Dk=128, Dv=128, P=16, maxp=8, N=20, fp8=False, shares=0, layout=0):
    return skv.make_desc(B, T, Hq, Hkv, Dk, Dv, P, maxp, N, int(fp8), shares, 1, layout)


def refused(want, fn, *args, **kw):
    with pytest.raises(skv.SplitKVError) as e:
        fn(*args, **kw)
    assert e.value.status == want and skv.splitkv_last_error(), e.value
    return str(e.value)


# ------------------------------------------------------------------ rope tables

@pytest.mark.parametrize("kw", [
    dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=128, rot_offset=8), dict(rot_dim=128, rot_offset=-16),
    dict(rot_dim=128, sections=(30, 30, 30)), dict(rot_dim=128, sections=(65, -1)), dict(rot_dim=128, sections=(16,) * 5),
    dict(rot_dim=128, base=0.0), dict(rot_dim=128, base=math.inf), dict(rot_dim=128, base=math.nan), dict(rot_dim=128, pairing=2),
    dict(rot_dim=32, freqs=[math.nan] * 16), dict(rot_dim=32, freqs=[1e6] * 16)])
def test_rope_refusals(kw):
    refused(EINVAL, skv.splitkv_rope_create, **kw)


def test_rope_takes_empty_sections_and_one_axis():
    assert skv.splitkv_rope_create(128, (0, 64, 0)).n_axes == 3
    assert skv.splitkv_rope_create(64).n_axes == 1
    with pytest.raises(ValueError):
        skv.splitkv_rope_create(64, freqs=[1.0] * 31)


def test_rope_turns_are_the_frequencies_in_fixed_point():
    """The library's table, read from the host object: freq / 2 pi modulo 1, exact to 2^-62 of a turn."""
    from fractions import Fraction
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    freqs = [1.0, 0.5, 2.0 ** -40, 1e-3, 6.5, 12345.678, -0.25, 0.0, 1e-18, 2 * math.pi, 999999.0, -1e-3, 3.0, 4.0, 5.0, 0.1]
    r = skv.splitkv_rope_create(32, freqs=freqs)
    turns = (ctypes.c_uint64 * 16).from_address(r.handle + 16)  # after four int32 fields
    for f, t in zip(freqs, turns):
        exact = Fraction(f) / (2 * pi) % 1
        d = abs(Fraction(int(t), 1 << 64) - exact)
        # the product's second double is exact to 2^-53 of its own size, 2^-53 |f| / 2 pi
        assert min(d, 1 - d) <= Fraction(1, 1 << 63) + abs(Fraction(f)) / (1 << 105), f


# ------------------------------------------------------------------ append

def call_append(d, **kw):
    a = dict(desc=d, rope=None, positions=A, q=A, k=A, v=A, block_table=A, seq_lens=A, q_out=2 * A, k_pages=A, v_pages=A,
             n_tokens=d.batch * d.q_tokens, stream=0)
    a.update(kw)
    if d.v_shares_k and "v" not in kw:
        a.update(v=None, v_pages=None)
    return skv.splitkv_append(**a)


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(k_pages=None), dict(block_table=None), dict(seq_lens=None), dict(v=None), dict(v_pages=None),
    dict(q=None), dict(q_out=None), dict(k=A + 8), dict(q=A + 2), dict(v_pages=A + 4), dict(cu_tokens=A + 2), dict(positions=A + 1),
    dict(status=A + 2), dict(key_weights=A + 2), dict(n_tokens=-1), dict(n_tokens=3), dict(positions=None, key_positions=A),
    dict(q_out=A + 256), dict(k_scale=A, v_scale=A)])
def test_append_refusals(kw):
    refused(EINVAL, call_append, desc(), **kw)


def test_append_refuses_what_does_not_fit_the_cache():
    rope = skv.splitkv_rope_create(128)
    refused(EINVAL, call_append, desc(), rope=rope, positions=None)
    refused(EINVAL, call_append, desc(), rope=skv.splitkv_rope_create(128, rot_offset=16))
    refused(EINVAL, call_append, desc(Hq=128, Hkv=1, Dk=576, Dv=512, shares=1), v=A)
    refused(EINVAL, call_append, desc(Hq=128, Hkv=1, Dk=576, Dv=512, shares=1), rope=skv.splitkv_rope_create(128, rot_offset=464))
    refused(EUNSUPPORTED, call_append, desc(Dk=64, Dv=64))
    refused(EUNSUPPORTED, call_append, desc(Hq=128, Hkv=2, Dk=576, Dv=512, shares=1))
    refused(EUNSUPPORTED, call_append, desc(Dk=128, Dv=128, shares=1))
    refused(EINVAL, call_append, desc(P=24))
    refused(EINVAL, call_append, desc(maxp=1 << 27))
    refused(EINVAL, call_append, desc(fp8=True), kv_scale=0.0)
    refused(EINVAL, call_append, desc(fp8=True), kv_scale=math.nan)
    refused(EINVAL, call_append, desc(fp8=True), k_scale=A)
    refused(EINVAL, call_append, desc(fp8=True), k_scale=A + 2, v_scale=A)


def test_append_refuses_strides_that_do_not_hold_a_token():
    d = desc()
    lib = skv._lib.splitkv_append

    def status(qs=1024, ks=256, vs=256, os_=1024):
        return lib(ctypes.byref(d), None, 2, None, None, A, qs, A, ks, A, vs, A, A, 1.0, None, None, 2 * A, os_, A, A, None,
                   None, None, 0)

    assert status(qs=1016) == status(ks=248) == status(vs=260) == status(os_=1028) == EINVAL


# ------------------------------------------------------------------ key weights

def call_weights(d, **kw):
    a = dict(desc=d, q=A, k_pages=A, block_table=A, seq_lens=A, lse=A, scale=0.1, kv_scale=1.0, decay=1.0, weights_in=A,
             weights_out=A, stream=0)
    a.update(kw)
    return skv.splitkv_key_weights(**a)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k_pages=None), dict(block_table=None), dict(seq_lens=None), dict(lse=None), dict(weights_out=None),
    dict(weights_in=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(decay=math.nan),
    dict(decay=math.inf), dict(q=A + 8), dict(k_pages=A + 8), dict(lse=A + 2), dict(weights_out=A + 64), dict(weights_in=A + 4),
    dict(k_scale=A), dict(status=A + 1)])
def test_weight_refusals(kw):
    refused(EINVAL, call_weights, desc(), **kw)


def test_weights_refuse_other_shapes():
    refused(EUNSUPPORTED, call_weights, desc(Hq=128, Hkv=1, Dk=576, Dv=512, shares=1))
    refused(EUNSUPPORTED, call_weights, desc(T=9))
    refused(EUNSUPPORTED, call_weights, desc(Hq=66, Hkv=2))
    refused(EINVAL, call_weights, desc(fp8=True), kv_scale=-1.0)
    refused(EINVAL, call_weights, desc(fp8=True), k_scale=A + 2)


# ------------------------------------------------------------------ evict

def call_evict(d, budget=16, **kw):
    a = dict(desc=d, budget=budget, sink=0, recent=0, k_pages=A, v_pages=A, block_table=A, seq_lens=A, weights_in=A,
             positions_in=2 * A, weights_out=A, positions_out=2 * A, seq_lens_out=A, workspace=A,
             workspace_bytes=1 << 30, stream=0)
    a.update(kw)
    return skv.splitkv_evict(**a)


@pytest.mark.parametrize("kw", [
    dict(budget=0), dict(budget=-5), dict(sink=-1), dict(recent=-1), dict(k_pages=None), dict(v_pages=None),
    dict(block_table=None), dict(seq_lens=None), dict(weights_in=None), dict(weights_out=None), dict(seq_lens_out=None),
    dict(positions_in=None), dict(positions_out=None), dict(sink=1, positions_in=None, positions_out=None),
    dict(recent=1, positions_in=None, positions_out=None), dict(k_pages=A + 8), dict(weights_in=A + 2),
    dict(weights_out=A + 4), dict(positions_out=2 * A - 4), dict(seq_lens_out=A + 4), dict(workspace=A + 8)])
def test_evict_refusals(kw):
    refused(EINVAL, call_evict, desc(), **kw)


def test_evict_refuses_more_groups_than_a_grid_holds():
    d = desc(B=1 << 27, Hkv=2, maxp=1)
    assert "2^28" in refused(EINVAL, call_evict, d) and skv.splitkv_evict_workspace_size(d, 1) == 0
    assert skv.splitkv_evict_workspace_size(desc(B=(1 << 27) - 1, Hkv=2, maxp=1), 1) > 0


def test_evict_workspace():
    d = desc(B=3, Hkv=2, maxp=8, P=16)  # 128 slots
    refused(EWORKSPACE, call_evict, d, workspace=None)
    for budget, most in ((16, 16), (64, 64), (100, 28), (128, 0), (1 << 30, 0)):
        need = skv.splitkv_evict_workspace_size(d, budget)
        assert need >= 6 * 8 + 6 * 2 * most * 4
        refused(EWORKSPACE, call_evict, d, budget=budget, workspace_bytes=need - 1)
    assert skv.splitkv_evict_workspace_size(d, 0) == 0
    assert skv.splitkv_evict_workspace_size(desc(Dk=64, Dv=64), 4) == 0
    refused(EINVAL, call_evict, desc(Hq=128, Hkv=1, Dk=576, Dv=512, shares=1))


# ------------------------------------------------------------------ cross attention

def call_cross(d, **kw):
    a = dict(desc=d, cu_tokens=None, q=A, k_pages=A, v_pages=A, block_table=A, seq_lens=A, scale=0.1, out=1 << 40, lse=A,
             workspace=A, workspace_bytes=1 << 40, n_tokens=d.batch * d.q_tokens, stream=0)
    a.update(kw)
    return skv.splitkv_cross_attend(**a)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k_pages=None), dict(v_pages=None), dict(block_table=None), dict(seq_lens=None), dict(out=None),
    dict(q=A + 8), dict(out=A), dict(out=A + 256), dict(lse=A + 2), dict(cu_tokens=A + 2), dict(scale=0.0), dict(scale=math.nan),
    dict(n_tokens=-1), dict(n_tokens=5), dict(n_tokens=1 << 28, cu_tokens=A)])
def test_cross_refusals(kw):
    refused(EINVAL, call_cross, desc(), **kw)


def test_cross_refuses_other_caches_and_small_workspaces():
    refused(EUNSUPPORTED, call_cross, desc(fp8=True))
    refused(EUNSUPPORTED, call_cross, desc(Hq=128, Hkv=1, Dk=576, Dv=512, shares=1))
    d = desc(B=1, Hkv=1, maxp=512)  # one row tile over 8192 slots: split
    need = skv.splitkv_cross_workspace_size(d, 1)
    assert need >= 2 * 8 * 129 * 4  # two partial results at least
    refused(EWORKSPACE, call_cross, d, workspace=None, workspace_bytes=0)
    refused(EWORKSPACE, call_cross, d, workspace_bytes=need - 1)
    refused(EINVAL, call_cross, d, workspace=A + 8)
    assert skv.splitkv_cross_workspace_size(desc(Hkv=2, maxp=512), 1 << 20) == 0  # many rows: not split
    assert skv.splitkv_cross_workspace_size(d, 0) == 0 and skv.splitkv_cross_workspace_size(d, -1) == 0
    call_cross(d, cu_tokens=A, n_tokens=0)  # nothing to do, nothing launched
    lib = skv._lib.splitkv_cross_attend
    for stride in (1016, 1025, 1 << 31, 1 << 62, -1024):
        assert lib(ctypes.byref(d), 1, None, A, stride, A, A, A, A, 0.1, 1 << 40, None, A, 1 << 40, None, 0) == EINVAL


def test_calls_without_tokens():
    import torch
    none = torch.zeros((0, 2, 128), dtype=torch.bfloat16)
    call_append(desc(), cu_tokens=A, n_tokens=0, k=None, v=None, q=None, q_out=None, positions=None)
    assert skv._lib.splitkv_cross_attend(ctypes.byref(desc()), 0, A, none.data_ptr(), 1024, A, A, A, A, 0.1, None, None, None, 0,
                                         None, 0) == skv.SPLITKV_OK
    refused(EINVAL, call_append, desc(), n_tokens=0)  # without cu_tokens: a token per sequence


def test_tensor_arguments_are_checked():
    import torch
    d = desc()
    for bad in (torch.zeros(4, dtype=torch.float32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):  # the type, the size, the device
            call_weights(d, seq_lens=bad)
    with pytest.raises(ValueError):
        call_append(d, k=torch.zeros(2, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        call_append(d, k=torch.zeros(2, 128, 2, dtype=torch.bfloat16).transpose(1, 2))


# ------------------------------------------------------------------ the plain implementations the GPU tests use

def test_plain_evict_by_hand():
    from _cache_ops import evict_moves
    w = np.array([5, 1, 4, 0, 3, 9, 2, 2], np.float32)
    p = np.arange(8)
    assert evict_moves(w, p, 8, 8, 0, 0) == (8, [])
    assert evict_moves(w, p, 8, 4, 0, 0) == (4, [(1, 4), (3, 5)])
    assert evict_moves(w, p, 8, 4, 2, 1) == (4, [(2, 5), (3, 7)])
    assert evict_moves(np.zeros(8, np.float32), p, 8, 3, 0, 0) == (3, [])
    assert evict_moves(np.array([np.nan, -1, 0, 1], np.float32), p, 4, 2, 0, 0) == (2, [(1, 3)])
    assert evict_moves(w, p[::-1], 8, 2, 0, 2) == (2, [])


def test_plain_rotation_is_a_rotation():
    from _cache_ops import rotated
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 32))
    pos = np.array([[0, 5, 7], [1, 2, 3]])
    for pairing in (0, 1):
        y = rotated(x, pos, [1.0, 0.5, 0.25, 0.1] * 2, (3, 5), 16, pairing)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.array_equal(y[..., :16], x[..., :16])
        back = rotated(y, -pos, [1.0, 0.5, 0.25, 0.1] * 2, (3, 5), 16, pairing)
        assert np.allclose(back, x)
    one = np.zeros((1, 1, 16))
    one[0, 0, 0] = 1
    y = rotated(one, np.array([[2]]), [0.3] * 8, (8,), 0, 0)
    assert np.isclose(y[0, 0, 0], math.cos(0.6)) and np.isclose(y[0, 0, 8], math.sin(0.6))


def test_plain_weights_sum_to_the_rows():
    from _cache_ops import key_weights, lse_of
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((3, 4, 128)), rng.standard_normal((20, 2, 128))
    w = key_weights(q, k, lse_of(q, k, 0.1, 3), 0.1, 3)
    assert np.allclose(w.sum(1), 3 * 2)


# ------------------------------------------------------------------ the compiled marshalling

def test_wrong_kinds_of_arguments_raise():
    import torch
    d = desc()
    with pytest.raises(TypeError):
        call_evict(b"not a descriptor")
    with pytest.raises(OverflowError):
        call_evict(d, budget=1 << 40)
    with pytest.raises(TypeError):
        call_evict(d, budget="a")
    for bad in ("q", np.zeros(8), object()):
        with pytest.raises(TypeError):
            call_cross(d, q=bad)
    with pytest.raises(TypeError):
        call_cross(d, scale=None)
    with pytest.raises(TypeError):
        call_cross(d, n_tokens=None)  # q is an address
    with pytest.raises(ValueError):  # enough elements of the right type, but not on the device (nor with memory)
        call_cross(d, q=torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="meta"))
    with pytest.raises(ValueError):
        call_cross(d, q=torch.zeros((2, 8, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        call_evict(d, weights_in=torch.zeros((2, 2, 128)).transpose(0, 1))
    refused(EINVAL, call_cross, d, q=None, n_tokens=None)
    # counts that pass 64 bits ask for more elements than any tensor has
    huge = desc(B=2**31 - 1, Hkv=2**10, Hq=2**10, maxp=2**26, P=16, N=1)
    with pytest.raises(ValueError):
        call_evict(huge, weights_in=torch.zeros(16))
