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
