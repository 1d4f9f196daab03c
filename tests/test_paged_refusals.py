"""Calls of the paged cache that the host refuses before anything is launched (no GPU)."""
import ctypes

import pytest

import test_abi_paged as T


@pytest.fixture(scope="module")
def A():
    from lvlm_kv_cache_gb300 import build

    build.build()
    from lvlm_kv_cache_gb300 import aircache

    aircache.lib()
    return aircache


@pytest.mark.parametrize("field", ["positions", "cu_tokens", "seen", "status"])
@pytest.mark.parametrize("by", [1, 2])
def test_rotation_refuses_integers_off_their_alignment(A, field, by):
    at = 0x1900000 + by
    p = T.rotate(A, **({} if field == "status" else {field: at}))
    status = ctypes.c_void_p(at) if field == "status" else None
    assert A.lib().aircache_rotate(ctypes.byref(p), status, None) == A.ERR_INVALID_ARG


@pytest.mark.parametrize("field", ["keep", "seen", "lens_out"])
@pytest.mark.parametrize("by", [1, 2])
def test_eviction_refuses_integers_off_their_alignment(A, field, by):
    p = T.evict(A, **{field: 0x1900000 + by})
    assert A.lib().aircache_evict(ctypes.byref(p), T.WS, 1 << 40, None) == A.ERR_INVALID_ARG
    assert A.lib().aircache_evict_workspace_size(ctypes.byref(p)) == 0


# Ten tokens: of 28 query heads and 4 key heads of 128.  The first two lay rows of different tokens and heads onto one
# another (token 1's head 0 on token 0's head 1; token 3's head 0 on token 0's head 2), the third by half a row.
@pytest.mark.parametrize("over", [
    dict(qo_stride_tok=128, qo_stride_head=128), dict(ko_stride_tok=256, ko_stride_head=384),
    dict(qo_stride_tok=192, qo_stride_head=128), dict(ko_stride_tok=192, ko_stride_head=256)])
def test_rotation_refuses_outputs_whose_own_rows_overlap(A, over):
    assert A.lib().aircache_rotate(ctypes.byref(T.rotate(A, **over)), None, None) == A.ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(q_out=0x1100000), dict(q_out=0x1200000), dict(k_out=0x1000000), dict(k_out=0x1200000), dict(q_out=0x1400000)])
def test_rotation_refuses_outputs_on_other_inputs(A, over):
    assert A.lib().aircache_rotate(ctypes.byref(T.rotate(A, **over)), None, None) == A.ERR_INVALID_ARG


def test_rotation_refuses_keys_and_values_in_one_place(A):
    p = T.rotate(A, T.pages(A, v=0x100000))
    assert A.lib().aircache_rotate(ctypes.byref(p), None, None) == A.ERR_INVALID_ARG


# four sequences; lens at 0x400000, mass and order of 50 x 4 x 16 slots at 0x500000 and 0x600000
@pytest.mark.parametrize("over", [
    dict(lens_out=0x400004), dict(lens_out=0x3ffff4), dict(lens_out=0x70000c), dict(lens_out=0x70fff8),
    dict(mass_out=0x500010), dict(mass_out=0x500000 + 50 * 4 * 16 * 4 - 16), dict(mass_out=0x4ffff0),
    dict(order_out=0x600010), dict(mass_out=0x600000), dict(order_out=0x500000), dict(mass_out=0x900000, order_out=0x900100)])
def test_eviction_refuses_outputs_that_overlap_in_part(A, over):
    p = T.evict(A, **over)
    assert A.lib().aircache_evict(ctypes.byref(p), T.WS, 1 << 40, None) == A.ERR_INVALID_ARG
    assert A.lib().aircache_evict_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("mass_out", [0x500010, 0x500000 + 50 * 4 * 16 * 4 - 16, 0x4ffff0])
def test_decode_refuses_a_mass_that_overlaps_in_part(A, mass_out):
    p = T.decode(A, mass_out=mass_out)
    assert A.lib().aircache_paged_decode(ctypes.byref(p), T.WS, 1 << 40, None) == A.ERR_INVALID_ARG
    assert A.lib().aircache_paged_decode_workspace_size(ctypes.byref(p)) == 0


def test_arrays_next_to_one_another_are_taken(A):
    beside = 0x500000 + 50 * 4 * 16 * 4
    p = T.evict(A, lens_out=0x400010, mass_out=beside, order_out=beside + 50 * 4 * 16 * 4)
    assert A.lib().aircache_evict_workspace_size(ctypes.byref(p)) > 0
    assert A.lib().aircache_paged_decode_workspace_size(ctypes.byref(T.decode(A, mass_out=beside))) > 0
