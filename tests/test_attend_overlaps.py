"""Outputs of aircache_paged_attend that lie on what the call reads: refused by the host before
anything is launched (no GPU)."""
import ctypes

import pytest

import test_abi_paged as T
from test_attend_refusals import A, attend, attend_status  # noqa: F401

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
