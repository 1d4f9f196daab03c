"""Outputs of aircache_paged_attend and aircache_shared_decode that lie on what the call reads: refused by the host before
anything is launched (no GPU)."""
import ctypes

import pytest

import test_abi_paged as T
from test_attend_refusals import A, attend, attend_status, shared, shared_status  # noqa: F401

# of test_abi_paged's pages: fifty of 16 rows of 4 heads of 128 (bf16: 16 KB a page), keys at 1 MB, values at 2 MB, the
# table of 4 x 10 at 3 MB, 4 lengths at 4 MB
K, V, PAGE = 0x100000, 0x200000, 16 * 512 * 2
SCALES = dict(kv_dtype=2, k_scale=0x30000, v_scale=0x40000)  # 50 x 4 x 16 floats each: 12,800 bytes


def size(A, p):  # noqa: F811
    return A.lib().aircache_paged_attend_workspace_size(ctypes.byref(p))


@pytest.mark.parametrize("name", ["out", "lse"])
@pytest.mark.parametrize("at", [K + 49 * PAGE, K + 50 * PAGE - 16, V + 49 * PAGE + 512, V + 50 * PAGE - 16, 0x300000, 0x300000 + 144,
                                0x400000, 0x1700000, 0x1700010])
def test_attend_refuses_outputs_on_the_last_page_and_on_integers(A, name, at):  # noqa: F811
    p = attend(A, **{name: at})
    assert attend_status(A, p) == A.ERR_INVALID_ARG and size(A, p) == 0


@pytest.mark.parametrize("name", ["out", "lse"])
def test_attend_refuses_outputs_on_a_cache_of_one_page(A, name):  # noqa: F811
    for at in (K, V, K + PAGE - 16):
        assert attend_status(A, attend(A, T.pages(A, num_pages=1), **{name: at})) == A.ERR_INVALID_ARG
    assert size(A, attend(A, T.pages(A, num_pages=1), **{name: K + PAGE})) > 0


@pytest.mark.parametrize("name", ["out", "lse"])
def test_attend_refuses_outputs_on_scales_and_ranges(A, name):  # noqa: F811
    for at in (0x30000, 0x30000 + 12800 - 16, 0x40000 + 12784):
        assert attend_status(A, attend(A, T.pages(A, **SCALES), **{name: at})) == A.ERR_INVALID_ARG
        assert size(A, attend(A, **{name: at})) > 0  # (without scales nothing lies there)
    for over in (dict(row_begin=0x1800000), dict(row_end=0x1800000)):
        assert attend_status(A, attend(A, **dict(over, **{name: 0x1800020}))) == A.ERR_INVALID_ARG


def test_attend_takes_outputs_right_behind_what_it_reads(A):  # noqa: F811
    for at in (K + 50 * PAGE, V + 50 * PAGE, 0x300000 + 160, 0x400000 + 16, 0x1700000 + 32):
        for over in (dict(out=at), dict(lse=at)):
            assert size(A, attend(A, **over)) > 0, over
    assert size(A, attend(A, T.pages(A, **SCALES), lse=0x30000 + 12800, out=0x40000 + 12800)) > 0


def test_attend_of_strides_past_the_addresses(A):  # noqa: F811
    # spans are counted without passing their own integers: pages that reach over everything behind them
    far = T.pages(A, num_pages=(1 << 31) - 1, stride_page=1 << 61)
    assert attend_status(A, attend(A, far)) == A.ERR_INVALID_ARG
    assert attend_status(A, attend(A, q_stride_tok=1 << 62)) == A.ERR_INVALID_ARG


# the prefixes' pages: another pool at 32 and 33 MB, table of 2 x 10 and 2 lengths behind it; own rows as above, their
# mass (50 x 4 x 16 floats) at 5 MB, q of 4 x 28 x 128 at 7 MB, cu_seqs (3) at 10 MB
PREFIX = dict(num_seqs=2, k=0x2000000, v=0x2100000, table=0x2200000, lens=0x2201000, mass=None, order=None)


def step(A, mass=False, int8=False, **own):  # noqa: F811
    scales = dict(kv_dtype=A.INT8, k_scale=0x2300000, v_scale=0x2310000) if int8 else {}
    if mass:
        own = dict(dict(mass_out=0x500000), **own)
    return shared(A, own=T.decode(A, **own), pg=T.pages(A, **dict(PREFIX, **scales)))


@pytest.mark.parametrize("name", ["out", "lse", "mass_out"])
@pytest.mark.parametrize("at", [0x2000000, 0x2000000 + 50 * PAGE - 16, 0x2100000 + 49 * PAGE, 0x2200000 + 64, 0x2201000, 0xa00000, K,
                                V + 50 * PAGE - 16, 0x300000, 0x400000, 0x700000, 0x700000 + 4 * 7168 - 16])
def test_shared_decode_refuses_outputs_on_what_it_reads(A, name, at):  # noqa: F811
    p = step(A, **{name: at})
    assert shared_status(A, p) == A.ERR_INVALID_ARG
    assert A.lib().aircache_shared_decode_workspace_size(ctypes.byref(p)) == 0


def test_shared_decode_refuses_outputs_on_scales_and_on_one_another(A):  # noqa: F811
    size = lambda p: A.lib().aircache_shared_decode_workspace_size(ctypes.byref(p))  # noqa: E731
    for at in (0x2300000 + 12784, 0x2310000):
        assert shared_status(A, step(A, int8=True, out=at)) == A.ERR_INVALID_ARG
        assert size(step(A, out=at)) > 0
    for over in (dict(lse=0x800000 + 4 * 7168 - 16), dict(out=0x500000), dict(lse=0x500000 + 12784), dict(mass_out=0x800000)):
        assert shared_status(A, step(A, mass=True, **over)) == A.ERR_INVALID_ARG, over
    for over in (dict(), dict(lse=0x800000 + 4 * 7168), dict(lse=0x500000 + 12800), dict(mass_out=0x2400000)):
        assert size(step(A, mass=True, **over)) > 0, over
    one_pool = dict(num_seqs=2)  # own rows and prefixes of one pool, with its mass
    assert size(shared(A, own=T.decode(A, mass_out=0x500000), pg=T.pages(A, **one_pool))) > 0
    assert size(shared(A, own=T.decode(A, out=0x500000), pg=T.pages(A, **one_pool))) > 0  # (without mass_out it is not read)
