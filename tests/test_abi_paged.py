"""Host-side checks of the paged-cache entry points (no GPU, nothing launched)
and of their 64-bit forms on cases worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as O


@pytest.fixture(scope="module")
def A():
    from lvlm_kv_cache_gb300 import build

    build.build()
    from lvlm_kv_cache_gb300 import aircache

    aircache.lib()
    return aircache


def pages(A, **over):
    c = A.PagesStruct(num_seqs=4, h_kv=4, head_dim=128, kv_dtype=A.BF16, page_rows=16, max_pages=10, num_pages=50,
                      k=0x100000, v=0x200000, stride_page=16 * 512, stride_row=512, stride_head=128, table=0x300000,
                      table_stride=10, lens=0x400000, k_scale=None, v_scale=None, mass=0x500000, order=0x600000)
    for n, x in over.items():
        setattr(c, n, x)
    return c


def decode(A, pg=None, **over):
    p = A.PagedDecodeProblemStruct(pages=ctypes.pointer(pg if pg is not None else pages(A)), h_q=28, dtype=A.BF16,
                                   scale=0.1, reserved0=0, total_rows=640, q=0x700000, q_stride_seq=28 * 128,
                                   q_stride_head=128, out=0x800000, lse=None, mass_out=None)
    for n, x in over.items():
        setattr(p, n, x)
    return p


def evict(A, pg=None, **over):
    p = A.EvictProblemStruct(pages=ctypes.pointer(pg if pg is not None else pages(A)), keep=0x700000, seen=0x710000,
                             lens_out=0x720000, mass_out=0x500000, order_out=0x600000, sink=1, recent=2, max_rows=160)
    for n, x in over.items():
        setattr(p, n, x)
    return p


def rotate(A, pg=None, **over):
    p = A.RotateProblemStruct(
        num_tokens=10, num_seqs=4, h_q=28, h_kv=4, head_dim=128, dtype=A.BF16, rotary_dim=128, interleaved=0, axes=1,
        section0=0, section1=0, eps=1e-6, reserved0=0, q=0x1000000, k=0x1100000, v=0x1200000, q_stride_tok=4608,
        q_stride_head=128, k_stride_tok=4608, k_stride_head=128, v_stride_tok=4608, v_stride_head=128,
        q_out=0x1300000, k_out=0x1400000, qo_stride_tok=3584, qo_stride_head=128, ko_stride_tok=512,
        ko_stride_head=128, q_weight=0x1500000, k_weight=0x1500100, turns=0x1600000, positions=None,
        cu_tokens=0x1700000, seen=0x1800000, pages=ctypes.pointer(pg if pg is not None else pages(A)))
    for n, x in over.items():
        setattr(p, n, x)
    return p


WS = ctypes.c_void_p(0x900000)

BAD_PAGES = [
    ("num_seqs", -1), ("num_seqs", 65536), ("h_kv", 0), ("head_dim", 96), ("kv_dtype", 0), ("kv_dtype", 2),
    ("page_rows", 8), ("page_rows", 24), ("page_rows", 8192), ("max_pages", 0), ("max_pages", 1 << 28),
    ("num_pages", 0), ("num_pages", 1 << 31), ("k", None), ("v", 0x200008), ("stride_page", 0), ("stride_row", 516),
    ("stride_head", -128), ("table", None), ("table_stride", 9), ("lens", None), ("lens", 0x400002), ("mass", 0x500004),
    ("order", 0x600008)]


@pytest.mark.parametrize("field,value", BAD_PAGES)
def test_bad_pages_rejected_by_every_entry_point(A, field, value):
    lib = A.lib()
    pg = pages(A, **{field: value})
    assert lib.aircache_paged_decode(ctypes.byref(decode(A, pg)), WS, 1 << 40, None) == A.ERR_INVALID_ARG
    assert lib.aircache_paged_decode_workspace_size(ctypes.byref(decode(A, pg))) == 0
    assert lib.aircache_evict(ctypes.byref(evict(A, pg)), WS, 1 << 40, None) == A.ERR_INVALID_ARG
    assert lib.aircache_evict_workspace_size(ctypes.byref(evict(A, pg))) == 0
    assert lib.aircache_rotate(ctypes.byref(rotate(A, pg)), None, None) == A.ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,code", [
    ("h_q", 27, -1), ("h_q", 0, -1), ("h_q", 68, -2), ("dtype", 0, -1), ("reserved0", 1, -1), ("scale", 0.0, -1),
    ("scale", float("nan"), -1), ("scale", float("inf"), -1), ("scale", -1.0, -1), ("total_rows", 0, -1),
    ("total_rows", 1 << 31, -1), ("q", None, -1), ("q", 0x700008, -1), ("q_stride_head", 4, -1),
    ("q_stride_seq", -8, -1), ("out", None, -1), ("out", 0x800004, -1), ("lse", 0x900002, -1)])
def test_bad_decode_rejected(A, field, value, code):
    p = decode(A, **{field: value})
    assert A.lib().aircache_paged_decode(ctypes.byref(p), WS, 1 << 40, None) == code
    assert A.lib().aircache_paged_decode_workspace_size(ctypes.byref(p)) == 0


def test_decode_workspace_and_mass(A):
    lib = A.lib()
    p = decode(A)
    need = lib.aircache_paged_decode_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert lib.aircache_paged_decode(ctypes.byref(p), WS, need - 1, None) == A.ERR_WORKSPACE
    assert lib.aircache_paged_decode(ctypes.byref(p), ctypes.c_void_p(0x900010), need, None) == A.ERR_INVALID_ARG
    assert lib.aircache_paged_decode(ctypes.byref(p), None, need, None) == A.ERR_INVALID_ARG
    assert lib.aircache_paged_decode(None, WS, need, None) == A.ERR_INVALID_ARG
    more = lib.aircache_paged_decode_workspace_size(ctypes.byref(decode(A, mass_out=0x500000)))
    assert more >= need + 640 * 28 * 4  # the logits of the rows
    none = pages(A, mass=None)
    assert lib.aircache_paged_decode(ctypes.byref(decode(A, none, mass_out=0x500000)), WS, 1 << 40, None) == -1
    assert lib.aircache_paged_decode(ctypes.byref(decode(A, pages(A, num_seqs=0))), WS, 1 << 40, None) == A.OK


@pytest.mark.parametrize("over,code", [
    (dict(keep=None), -1), (dict(lens_out=None), -1), (dict(lens_out=0x400000), -1), (dict(lens_out=0x700000), -1), (dict(lens_out=0x710000), -1),
    (dict(mass_out=0x500008), -1), (dict(mass_out=None), -1),
    (dict(order_out=None), -1), (dict(sink=-1), -1), (dict(recent=-1), -1), (dict(seen=None), -1),
    (dict(max_rows=0), -1), (dict(max_rows=393217), -2)])
def test_bad_evict_rejected(A, over, code):
    p = evict(A, **over)
    assert A.lib().aircache_evict(ctypes.byref(p), WS, 1 << 40, None) == code
    assert A.lib().aircache_evict_workspace_size(ctypes.byref(p)) == 0


def test_evict_pages_and_workspace(A):
    lib = A.lib()
    p = evict(A)
    need = lib.aircache_evict_workspace_size(ctypes.byref(p))
    assert need >= 4 * 4 * 160 * 4 and need % 256 == 0
    assert lib.aircache_evict(ctypes.byref(p), WS, need - 1, None) == A.ERR_WORKSPACE
    assert lib.aircache_evict(ctypes.byref(p), None, need, None) == A.ERR_INVALID_ARG
    for over in (dict(mass=None), dict(order=None)):
        assert lib.aircache_evict(ctypes.byref(evict(A, pages(A, **over))), WS, 1 << 40, None) == A.ERR_INVALID_ARG
    assert lib.aircache_evict(ctypes.byref(evict(A, pages(A, num_seqs=0))), WS, 1 << 40, None) == A.OK


@pytest.mark.parametrize("over", [
    dict(dtype=0), dict(head_dim=64), dict(num_tokens=-1), dict(num_tokens=1 << 31), dict(num_seqs=5),
    dict(reserved0=1), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q=None), dict(q_out=None),
    dict(k=None), dict(v=None), dict(h_q=0), dict(h_kv=2), dict(rotary_dim=24), dict(rotary_dim=144),
    dict(rotary_dim=-16), dict(turns=None), dict(axes=2), dict(axes=3), dict(axes=3, positions=0x1900000, section0=65),
    dict(axes=3, positions=0x1900000, section0=-1), dict(seen=None), dict(cu_tokens=None), dict(q=0x1000008),
    dict(k_stride_tok=4604), dict(qo_stride_head=-128), dict(q_out=0x1000000), dict(k_out=0x1100000),
    dict(q_weight=0x1500002), dict(qo_stride_head=64), dict(ko_stride_tok=0), dict(qo_stride_tok=64)])
def test_bad_rotate_rejected(A, over):
    p = rotate(A, **over)
    assert A.lib().aircache_rotate(ctypes.byref(p), None, None) == A.ERR_INVALID_ARG


def test_rotate_without_cache(A):
    lib = A.lib()
    none = ctypes.POINTER(A.PagesStruct)()
    for over in (dict(v=None, k_out=None), dict(), dict(v=None, cu_tokens=None, seen=None)):
        p = rotate(A, **over)
        p.pages = none  # no output for k; a v without a cache; no positions
        assert lib.aircache_rotate(ctypes.byref(p), None, None) == A.ERR_INVALID_ARG
    p = rotate(A, num_tokens=0)
    assert lib.aircache_rotate(ctypes.byref(p), None, None) == A.OK


def test_tensors_of_the_wrong_kind_are_refused(A):
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((1, 2), dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        A.PagedCache(k, k.clone(), t, n)
    for bad in (dict(k=k.float(), v=k.float()), dict(v=k[:2]), dict(table=t.long()), dict(lens=n.long()),
                dict(k_scale=torch.zeros((4, 2, 16))), dict(mass=torch.zeros((4, 16, 2))),
                dict(order=torch.zeros((4, 2, 16), dtype=torch.int64))):
        a = dict(k=k, v=k.clone(), table=t, lens=n)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            A.PagedCache(**a)
    with pytest.raises(ValueError):  # one row of pages for every sequence
        A.PagedCache(k, k.clone(), t.expand(3, 2), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        A.RotateProblem()
    with pytest.raises(ValueError):
        A.RotateProblem(k[0].float())


def test_rotation_table_keeps_the_frequencies(A):
    f = 1e6 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    t = A.rotation_table(f)
    assert t.dtype == torch.float32 and tuple(t.shape) == (64, 2)
    back = t.double().sum(1) * 2 * np.pi
    assert float(((back - f) / f).abs().max()) < 2.0 ** -47
    assert torch.equal(A.rotation_table(f.tolist()), t)


# ---------------------------------------------------------------- the 64-bit forms, by hand

def test_oracle_moves_by_hand():
    mass = np.array([5.0, 1.0, 4.0, 1.0, 3.0, 9.0, 1.0])
    kept, moves = O.evict_moves(mass, None, 4, 0, 0, 0)
    assert kept == [0, 2, 4, 5] and moves == [(4, 1), (5, 3)]
    kept, moves = O.evict_moves(mass, np.arange(7), 3, 7, 0, 2)  # rows 5 and 6 are recent
    assert kept == [0, 5, 6] and moves == [(5, 1), (6, 2)]
    kept, moves = O.evict_moves(np.array([1.0, 1.0, 1.0, 2.0]), None, 2, 0, 0, 0)  # ties to the lower row
    assert kept == [0, 3] and moves == [(3, 1)]
    assert O.evict_moves(mass, None, 7, 0, 0, 0) == (list(range(7)), [])
    kept, _ = O.evict_moves(np.array([np.nan, -np.inf, 0.0]), None, 2, 0, 0, 0)
    assert kept == [0, 2]


def test_oracle_rotation_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    y, _ = O.rotate(x, None, 0.0, np.array([[np.pi / 2, 0.0]]), False)
    np.testing.assert_allclose(y[0, 0], [-3.0, 2.0, 1.0, 4.0], atol=1e-12)
    y, _ = O.rotate(x, None, 0.0, np.array([[np.pi / 2]]), True)
    np.testing.assert_allclose(y[0, 0], [-2.0, 1.0, 3.0, 4.0], atol=1e-12)
    y, _ = O.rotate(x, np.full(4, 2.0), 0.0, np.zeros((1, 0)), False)
    np.testing.assert_allclose(y[0, 0], 2 * x[0, 0] / np.sqrt(7.5))


def test_oracle_decode_by_hand():
    k = np.zeros((2, 1, 1, 2))
    k[1, 0, 0] = [np.log(3.0), 0.0]
    v = np.array([[[[1.0, 0.0]]], [[[0.0, 1.0]]]])
    c = dict(k=k, v=v, k_scale=None, v_scale=None, table=np.array([[0, 1]]), lens=np.array([2]))
    out, lse, w, _, _ = O.decode(np.array([[[1.0, 0.0]]]), c, 1.0)
    np.testing.assert_allclose(out[0, 0], [0.25, 0.75])
    np.testing.assert_allclose(lse, np.log(4.0))
    np.testing.assert_allclose(w[0], [[0.25, 0.75]])
