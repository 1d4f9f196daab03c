"""Calls of aircache_paged_attend and aircache_shared_decode that the host refuses before anything is launched, and the
64-bit forms of both on cases worked out by hand (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import test_abi_paged as T
from oracle import paged as O


@pytest.fixture(scope="module")
def A():
    from lvlm_kv_cache_gb300 import build

    build.build()
    from lvlm_kv_cache_gb300 import aircache

    aircache.lib()
    return aircache


def attend(A, pg=None, **over):  # ten tokens of four sequences, 28 to 4 heads of 128; fifty pages at 1 and 2 MB
    p = A.PagedAttendProblemStruct(
        pages=ctypes.pointer(pg if pg is not None else T.pages(A)), num_tokens=10, h_q=28, dtype=A.BF16, causal=1,
        reserved0=0, scale=0.1, reserved1=0.0, cu_tokens=0x1700000, row_begin=None, row_end=None, q=0x1000000,
        q_stride_tok=3584, q_stride_head=128, out=0x1100000, out_stride_tok=3584, out_stride_head=128, lse=None)
    for n, x in over.items():
        setattr(p, n, x)
    return p


def shared(A, own=None, pg=None, **over):
    p = A.SharedDecodeProblemStruct(own=own if own is not None else T.decode(A), cu_seqs=0xa00000,
                                    prefix=ctypes.pointer(pg if pg is not None else T.pages(A, num_seqs=2)))
    for n, x in over.items():
        setattr(p, n, x)
    return p


def attend_status(A, p):
    return A.lib().aircache_paged_attend(ctypes.byref(p), T.WS, 1 << 40, None)


def shared_status(A, p):
    return A.lib().aircache_shared_decode(ctypes.byref(p), T.WS, 1 << 40, None)


@pytest.mark.parametrize("field,value", T.BAD_PAGES)
def test_bad_pages(A, field, value):
    p = attend(A, T.pages(A, **{field: value}))
    assert attend_status(A, p) == A.ERR_INVALID_ARG
    assert A.lib().aircache_paged_attend_workspace_size(ctypes.byref(p)) == 0
    for p in (shared(A, pg=T.pages(A, **{"num_seqs": 2, field: value})), shared(A, own=T.decode(A, T.pages(A, **{field: value})))):
        assert shared_status(A, p) == A.ERR_INVALID_ARG
        assert A.lib().aircache_shared_decode_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("over,code", [
    (dict(h_q=27), -1), (dict(h_q=0), -1), (dict(h_q=68, out_stride_tok=8704), -2), (dict(dtype=0), -1), (dict(dtype=2), -1), (dict(causal=2), -1),
    (dict(causal=-1), -1), (dict(reserved0=1), -1), (dict(reserved1=1.0), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(num_tokens=-1), -1),
    (dict(num_tokens=(1 << 31) - 1), -1), (dict(q=None), -1), (dict(q=0x1000008), -1), (dict(q_stride_tok=4), -1),
    (dict(q_stride_tok=0), -1), (dict(q_stride_tok=-3584), -1), (dict(q_stride_head=0), -1), (dict(q_stride_head=132), -1),
    (dict(out=None), -1), (dict(out=0x1100008), -1), (dict(out_stride_tok=3588), -1), (dict(out_stride_tok=0), -1),
    (dict(out_stride_head=-128), -1), (dict(cu_tokens=None), -1), (dict(cu_tokens=0x1700002), -1),
    (dict(row_begin=0x1700001), -1), (dict(row_end=0x1700002), -1), (dict(lse=0x1800002), -1)])
def test_bad_attend(A, over, code):
    p = attend(A, **over)
    assert attend_status(A, p) == code
    assert A.lib().aircache_paged_attend_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("over", [
    dict(out_stride_head=64), dict(out_stride_tok=128), dict(out_stride_tok=192, out_stride_head=128),
    dict(out_stride_tok=256, out_stride_head=1280),                     # rows of out that meet
    dict(out=0x1000000), dict(out=0x1000100), dict(out=0x1000000 - 256),  # out and q
    dict(out=0x100000), dict(out=0x200010), dict(out=0x100000 + 49 * 16 * 512 * 2 - 16),  # out and the cache
    dict(lse=0x1100000), dict(lse=0x1100000 + 9 * 7168 + 27 * 256), dict(lse=0x1000010),  # lse and out, q
    dict(lse=0x100000), dict(lse=0x200010)])                            # lse and the cache
def test_attend_refuses_outputs_that_lie_on_something(A, over):
    assert attend_status(A, attend(A, **over)) == A.ERR_INVALID_ARG


def test_attend_takes_what_is_apart(A):
    size = A.lib().aircache_paged_attend_workspace_size
    for over in (dict(), dict(out_stride_tok=128, out_stride_head=1280), dict(lse=0x1120000, row_begin=0x1800000, row_end=0x1800028),
                 dict(num_tokens=1, q_stride_tok=0, out_stride_tok=0), dict(out=0x1000000 + 9 * 7168 + 28 * 256)):
        assert size(ctypes.byref(attend(A, **over))) > 0, over
    assert size(ctypes.byref(attend(A, T.pages(A, kv_dtype=A.INT8, k_scale=0x800000, v_scale=0x810000)))) > 0


def test_attend_workspace(A):
    lib = A.lib()
    p = attend(A)
    need = lib.aircache_paged_attend_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert lib.aircache_paged_attend(ctypes.byref(p), T.WS, need - 1, None) == A.ERR_WORKSPACE
    assert lib.aircache_paged_attend(ctypes.byref(p), ctypes.c_void_p(0x900010), need, None) == A.ERR_INVALID_ARG
    assert lib.aircache_paged_attend(ctypes.byref(p), None, need, None) == A.ERR_INVALID_ARG
    assert lib.aircache_paged_attend(None, T.WS, need, None) == A.ERR_INVALID_ARG
    assert lib.aircache_paged_attend_workspace_size(None) == 0
    assert lib.aircache_paged_attend(ctypes.byref(attend(A, T.pages(A, num_seqs=0))), T.WS, need, None) == A.OK
    assert lib.aircache_paged_attend(ctypes.byref(attend(A, num_tokens=0)), T.WS, need, None) == A.OK


@pytest.mark.parametrize("field,value,code", [
    ("h_q", 27, -1), ("h_q", 68, -2), ("dtype", 0, -1), ("reserved0", 1, -1), ("scale", 0.0, -1), ("total_rows", 0, -1),
    ("q", None, -1), ("q_stride_seq", 0, -1), ("q_stride_head", 0, -1), ("out", 0x800004, -1), ("lse", 0x900002, -1),
    ("mass_out", 0x500010, -1)])
def test_bad_own_step(A, field, value, code):
    assert shared_status(A, shared(A, own=T.decode(A, **{field: value}))) == code


@pytest.mark.parametrize("over", [dict(h_kv=2), dict(head_dim=64), dict(num_seqs=-1)])
def test_prefixes_of_another_kind(A, over):
    assert shared_status(A, shared(A, pg=T.pages(A, **dict(dict(num_seqs=2), **over)))) == A.ERR_INVALID_ARG


def test_shared_workspace(A):
    lib = A.lib()
    p = shared(A)
    need = lib.aircache_shared_decode_workspace_size(ctypes.byref(p))
    assert need > lib.aircache_paged_decode_workspace_size(ctypes.byref(T.decode(A))) and need % 256 == 0
    assert lib.aircache_shared_decode(ctypes.byref(p), T.WS, need - 1, None) == A.ERR_WORKSPACE
    assert lib.aircache_shared_decode(ctypes.byref(p), ctypes.c_void_p(0x900010), need, None) == A.ERR_INVALID_ARG
    assert lib.aircache_shared_decode(ctypes.byref(p), None, need, None) == A.ERR_INVALID_ARG
    assert lib.aircache_shared_decode(None, T.WS, need, None) == A.ERR_INVALID_ARG
    for bad in (dict(cu_seqs=None), dict(cu_seqs=0xa00002), dict(prefix=None)):
        assert shared_status(A, shared(A, **bad)) == A.ERR_INVALID_ARG
    none = T.decode(A, T.pages(A, num_seqs=0))
    assert shared_status(A, shared(A, own=none)) == A.OK


def test_tensors_of_the_wrong_kind(A):
    class Cache:  # a PagedCache's side of it; a real one wants a GPU
        d, h_kv, num_seqs, num_pages, page_rows, max_pages, mass = 64, 2, 3, 4, 16, 2, None
        k, c = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16), A.PagesStruct()

    q, cu = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    rows = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        A.PagedAttendProblem(q, Cache, cu)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., ::2]), dict(cu_tokens=cu[:3]), dict(cu_tokens=cu.long()),
                dict(out=q.float()), dict(out=q[:4]), dict(lse=torch.zeros((5, 3))), dict(lse=torch.zeros((5, 4)).double()),
                dict(row_begin=rows[:4]), dict(row_end=rows.long())):
        a = dict(q=q, cache=Cache, cu_tokens=cu)
        a.update(bad)
        with pytest.raises(ValueError) as e:
            A.PagedAttendProblem(**a)
        assert "CUDA" not in str(e.value)


# ---------------------------------------------------------------- the 64-bit forms, by hand

def by_hand():
    k, v = np.zeros((2, 2, 1, 2)), np.zeros((2, 2, 1, 2))
    k[0, :, 0, 0], k[1, :, 0, 0] = [0.0, np.log(3.0)], [np.log(4.0), 7.0]
    v[0, :, 0], v[1, 0, 0], v[1, 1, 0] = np.eye(2), [2.0, 2.0], [np.nan, np.nan]
    return dict(k=k, v=v, k_scale=None, v_scale=None, table=np.array([[0, 1]]), lens=np.array([3]))


def test_oracle_attend_by_hand():
    q = np.tile(np.array([[[1.0, 0.0]]]), (3, 1, 1))
    out, lse, _, _ = O.attend(q, [0, 2], by_hand(), 1.0, causal=True)
    np.testing.assert_allclose(out[:2, 0], [[0.25, 0.75], [9 / 8, 11 / 8]])  # weights 1, 3; then 1, 3, 4
    np.testing.assert_allclose(lse[:2, 0], np.log([4.0, 8.0]))
    assert np.isnan(out[2]).all()
    out, lse, _, _ = O.attend(q, [0, 3], by_hand(), 1.0, begin=[1, 2, 2], end=[2, 99, 2])
    np.testing.assert_allclose(out[:, 0], [[0.0, 1.0], [2.0, 2.0], [0.0, 0.0]])
    np.testing.assert_allclose(lse[:2, 0], np.log([3.0, 4.0]))
    assert np.isneginf(lse[2, 0])


def test_oracle_shared_decode_by_hand():
    c = by_hand()
    own = dict(c, table=np.array([[1, 0], [1, 0]]), lens=np.array([1, 1]))
    pre = dict(c, lens=np.array([2]))
    q = np.tile(np.array([[[1.0, 0.0]]]), (2, 1, 1))
    out, lse, w, _, _, _ = O.shared_decode(q, own, pre, [0, 1], 1.0)
    np.testing.assert_allclose(out[:, 0], [[9 / 8, 11 / 8], [2.0, 2.0]])
    np.testing.assert_allclose(lse[:, 0], np.log([8.0, 4.0]))
    np.testing.assert_allclose([w[0][0, 0], w[1][0, 0]], [0.5, 1.0])
