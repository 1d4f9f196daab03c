"""aircache_paged_attend where values that are not finite lie in rows that a token does not see, or weigh nothing: what
sees such a value becomes NaN or infinite, nothing else does.

Tolerances: as in test_gpu_paged_attend.py, and one term more.  The walk that clears such values holds weights 2^-40 as
large as the first one: where the largest of a row is 2^-40, fp32's smallest normal number, 2^-126, is 2^-86 of it, and a
weight below that may be 0.  R rows of values up to |v| then miss at most R 2^-86 |v|."""
import numpy as np
import pytest
import torch

import paged_utils as P
from oracle import paged as O
from test_gpu_paged_attend import A, HALF, i32, queries  # noqa: F401

pytestmark = pytest.mark.gpu


def spoil(cache, rows, value):
    """Makes the values of the first sequence's rows `value` (int8 rows: their scales)."""
    n = cache.page_rows
    for at in rows:
        pg = cache.table[0, at // n].long()
        if cache.k.dtype == torch.int8:
            cache.v_scale[pg, :, at % n] = value
        else:
            cache.v[pg, at % n, :, ::5] = value


def attend(A, cache, q, cu, causal=False, begin=None, end=None):  # noqa: F811
    fit = lambda x: None if x is None else i32(list(x))  # noqa: E731
    prob = A.PagedAttendProblem(q, cache, i32(cu), lse=True, causal=causal, row_begin=fit(begin), row_end=fit(end))
    A.paged_attend(prob)
    return prob.out, prob.lse


def check(out, lse, q, cu, clean, free, causal=False, begin=None, end=None):
    """The tokens `free` are as the definition makes them without the spoilt rows."""
    d = q.shape[2]
    want, want_lse, size, spread = O.attend(q.double().cpu().numpy(), cu, clean, d ** -0.5, causal, begin, end)
    got, gl = out.double().cpu().numpy()[free], lse.double().cpu().numpy()[free]
    want, want_lse, size, spread = want[free], want_lse[free], size[free], spread[free]
    assert np.all(np.isfinite(got)), f"{(~np.isfinite(got)).sum()} outputs of tokens that do not see the row"
    dx = d * 2.0 ** -24 * size
    top = np.abs(clean["v"]).max() * (1.0 if clean["v_scale"] is None else clean["v_scale"].max())
    tol = (HALF + 2 * dx[..., None] + 2.0 ** -18) * spread + HALF * np.abs(want) + clean["lens"].max() * 2.0 ** -86 * top
    ratio = np.abs(got - want) / tol
    assert np.all(ratio <= 1), f"worst {ratio.max():.2f} at {np.unravel_index(ratio.argmax(), ratio.shape)}"
    seen = np.isfinite(want_lse)
    assert np.array_equal(seen, np.isfinite(gl))
    assert np.all(np.abs(gl[seen] - want_lse[seen]) <= (dx + 2.0 ** -20 * (1 + np.abs(want_lse)))[seen])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("h_q,h_kv,d", [(28, 4, 128), (8, 8, 64), (16, 1, 128)])
def test_gaps_between_ranges(A, h_q, h_kv, d, value, int8):  # noqa: F811
    # the tokens of a unit see the ends of a long sequence, and the tiles between them are whole CTAs' runs
    R, begin, end = 20000, [0, 19900, 5, 7], [100, 20000, 70, 7]
    cache = P.build(A, [R], h_kv, d, 32, seed=40, mass=False, order=False, int8=int8)
    q, clean = queries(4, h_q, d, 40), P.host(cache)
    spoil(cache, (10000, 101 + 128, 4000, 15000), value)
    out, lse = attend(A, cache, q, [0, 4], begin=begin, end=end)
    check(out, lse, q, [0, 4], clean, np.arange(4), begin=begin, end=end)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [40, 300])
def test_images_in_a_row_of_which_tokens_see_the_latest(A, n, int8):  # noqa: F811
    # three images, the second one followed by no text: nobody sees it, and every row of it is spoilt
    R, cut = 9000, [0, 2500, 7000, 9000]
    cache = P.build(A, [R, 50], 2, 128, 16, seed=41, mass=False, order=False, int8=int8)
    q, clean = queries(n + 3, 14, 128, 41), P.host(cache)
    begin = [cut[0]] * (n // 2) + [cut[2]] * (n - n // 2) + [0] * 3
    end = [cut[1]] * (n // 2) + [cut[3]] * (n - n // 2) + [50] * 3
    spoil(cache, range(cut[1], cut[2]), float("nan"))
    out, lse = attend(A, cache, q, [0, n, n + 3], begin=begin, end=end)
    check(out, lse, q, [0, n, n + 3], clean, np.arange(n + 3), begin=begin, end=end)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("h_q,h_kv", [(28, 4), (8, 2), (16, 1)])
def test_a_token_at_a_tiles_border_whose_key_and_value_are_not_numbers(A, h_q, h_kv, int8):  # noqa: F811
    # tokens that see it have a sum that is not a number either; for those before it the part that begins there is empty
    for R in (1408, 2000, 2944, 5003, 9991, 20100):
        n = R % 128 + 40 if R % 128 else 168
        at = (R - 1) // 128 * 128
        cache = P.build(A, [R], h_kv, 128, 32, seed=42, mass=False, order=False, int8=int8)
        q, clean = queries(n, h_q, 128, 42), P.host(cache)
        pg = cache.table[0, at // 32].long()
        if int8:
            cache.k_scale[pg, :, at % 32] = float("nan")
        else:
            cache.k[pg, at % 32] = float("nan")
        spoil(cache, [at], float("nan"))
        out, lse = attend(A, cache, q, [0, n], causal=True)
        before = at - (R - n)
        check(out, lse, q, [0, n], clean, np.arange(before), causal=True)
        assert torch.isnan(out[before:, :, ::5]).all()


@pytest.mark.parametrize("R", [20000, 100])
def test_a_value_that_weighs_nothing_is_seen_all_the_same(A, R):  # noqa: F811
    # logits of minus infinity (under fp32's range) weigh 0, and 0 times NaN is NaN, wherever a CTA's run begins
    cache = P.build(A, [R], 2, 128, 16, seed=43, mass=False, order=False)
    q = torch.full((3, 14, 128), 3e38, dtype=torch.bfloat16, device="cuda")
    pg, r = cache.table[0].long(), torch.arange(R, device="cuda")
    cache.k[pg[r // 16], r % 16] = -1.0
    cache.k[pg[0], 3] = 0.0  # one row has the logit 0
    spoil(cache, [R // 2], float("nan"))
    out, lse = attend(A, cache, q, [0, 3])
    v = cache.v[pg[0], 3].repeat_interleave(7, 0).expand(3, -1, -1)
    spoilt = torch.zeros(128, dtype=torch.bool, device="cuda")
    spoilt[::5] = True
    assert torch.isnan(out[..., spoilt]).all()
    assert torch.equal(out[..., ~spoilt], v[..., ~spoilt]) and torch.all(lse == 0)
