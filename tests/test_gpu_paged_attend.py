"""aircache_paged_attend against its definition in 64 bits (oracle/paged.py).

Tolerances.  A dot product in fp32 over D exact products is off by at most
D 2^-24 sum |q_d k_d| scale =: dx (at the row where that is largest), and a
weight by a relative 2 dx + 2^-18 (two exponentials of that error, the base-2
exponential's own 2^-22, products and sums of up to some thousand terms).  lse: dx + 2^-20 (1 + |lse|).
out: each weight is rounded to bf16 before it meets V, int8 rows' with the value's scale
(2^-8 of it), and out is rounded to bf16:
(2^-8 + 2 dx + 2^-18) sum w |v| + 2^-8 |out|."""
import numpy as np
import pytest
import torch

import paged_utils as P
from oracle import paged as O

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lvlm_kv_cache_gb300 import build

    build.build()
    from lvlm_kv_cache_gb300 import aircache

    aircache.lib()
    return aircache


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(T, h_q, d, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((T, h_q, d), generator=g, device="cuda")).to(torch.bfloat16)


def verify(out, lse, q, cu, c, scale=None, causal=False, begin=None, end=None):
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    want, want_lse, size, spread = O.attend(q.double().cpu().numpy(), cu, c, scale, causal, begin, end)
    T = int(cu[-1])
    want, want_lse, size, spread = want[:T], want_lse[:T], size[:T], spread[:T]
    dx = d * 2.0 ** -24 * size
    got = out.double().cpu().numpy()[:T]
    tol = (HALF + 2 * dx[..., None] + 2.0 ** -18) * spread + HALF * np.abs(want) + 1e-30
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= tol), f"out: worst {np.max(err / tol):.2f} at {np.unravel_index(np.argmax(err / tol), err.shape)}"
    if lse is not None:
        gl = lse.double().cpu().numpy()[:T]
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(gl))
        e = np.abs(gl[~empty] - want_lse[~empty])
        t = dx[~empty] + 2.0 ** -20 * (1 + np.abs(want_lse[~empty]))
        assert np.all(e <= t), f"lse: worst {np.max(e / t):.2f}"


def case(A, new, lens, h_q, h_kv, d, page_rows, seed=0, causal=False, begin=None, end=None, q_scale=1.5, q=None,
         scale=None, pad=2, **kw):
    """lens: rows of each cache, the new tokens' own among them (causal)."""
    cache = P.build(A, lens, h_kv, d, page_rows, seed=seed, mass=False, order=False, **kw)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + pad  # tokens behind the last sequence
    q = queries(T, h_q, d, seed, q_scale) if q is None else q
    out = torch.full((T, h_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, h_q), 7.0, device="cuda")
    fit = lambda x: None if x is None else i32(list(x) + [0] * (T - len(x)))  # noqa: E731
    before = P.state(cache)
    prob = A.PagedAttendProblem(q, cache, i32(cu.tolist()), out=out, lse=lse, causal=causal, scale=scale,
                                row_begin=fit(begin), row_end=fit(end))
    A.paged_attend(prob)
    verify(out, lse, q, cu, P.host(cache), scale, causal, begin, end)
    assert torch.all(out[cu[-1]:] == 7.0) and torch.all(lse[cu[-1]:] == 7.0)
    P.assert_same_state(before, P.state(cache))
    return prob, cache, q


NEW = [1, 2, 0, 17, 18, 19, 36, 37, 5, 73]
OLD = [0, 126, 40, 111, 0, 128, 300, 91, 1000, 55]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("page_rows", [16, 48, 64, 256])
def test_ragged(A, page_rows, causal, d, int8):
    lens = [a + b for a, b in zip(NEW, OLD)]
    case(A, NEW, lens, 28, 4, d, page_rows, seed=d + page_rows, causal=causal, int8=int8)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (16, 1), (9, 1), (8, 8), (10, 2), (24, 3)])
def test_heads(A, h_q, h_kv, int8):
    case(A, [130, 1, 0, 14, 3], [140, 5, 9, 300, 257], h_q, h_kv, 128, 32, seed=h_q, causal=True, int8=int8)
    case(A, [5, 129, 1], [200, 0, 128], h_q, h_kv, 64, 32, seed=h_q, int8=int8)


@pytest.mark.parametrize("int8", [False, True])
def test_one_sequence_is_joined_from_many_parts(A, int8):
    case(A, [3], [20011], 28, 4, 128, 64, seed=3, causal=True, int8=int8)
    case(A, [40, 1], [9000, 1], 4, 1, 64, 16, seed=4, int8=int8)
    case(A, [260], [3000], 2, 1, 128, 256, seed=4, causal=True, int8=int8)


def test_many_short_sequences(A):
    g = np.random.default_rng(5)
    new = g.integers(0, 4, 700)
    case(A, new.tolist(), (new + g.integers(0, 40, 700)).tolist(), 4, 2, 64, 16, seed=5, causal=True)


@pytest.mark.parametrize("int8", [False, True])
def test_slots_behind_the_last_row_hold_anything(A, int8):
    # NaN rows (bf16) or NaN scales (int8) behind the end, in a tile's middle and in its own page
    for causal in (True, False):
        case(A, [1, 17, 20, 50], [1, 17, 70, 250], 8, 2, 128, 64, seed=6, int8=int8, fill=float("nan"), causal=causal)
        case(A, [1, 17, 20, 50], [129, 17, 383, 513], 8, 8, 64, 16, seed=6, int8=int8, fill=float("inf"), causal=causal)


def test_many_sequences(A):
    # more than one CTA stages in shared memory, most of them without tokens
    g = np.random.default_rng(30)
    new = np.where(g.random(6000) < 0.1, g.integers(1, 4, 6000), 0)
    case(A, new.tolist(), (new + g.integers(0, 20, 6000)).tolist(), 2, 1, 64, 16, seed=30, causal=True)


def test_pages_of_many_rows(A):
    for page_rows, int8 in ((4096, False), (2048, True), (112, False), (4080, True)):
        case(A, [20, 3], [5000, 4097], 4, 2, 128, page_rows, seed=31, causal=True, int8=int8)


@pytest.mark.parametrize("int8", [False, True])
def test_offsets_past_32_bits(A, int8):
    # pages so far apart that elements (and, int8, bytes) of the last are past 2^32 from the first
    d, h, page_rows, n, R = 128, 2, 64, 30, 300
    small = P.build(A, [R], h, d, page_rows, seed=32, mass=False, order=False, int8=int8)
    apart, pages_n = 1 << 30, small.num_pages
    k = torch.empty(apart * (pages_n - 1) + page_rows * h * d, dtype=small.k.dtype, device="cuda")
    v = torch.empty_like(k)
    far = [x.as_strided(small.k.shape, (apart, h * d, d, 1)) for x in (k, v)]
    far[0].copy_(small.k)
    far[1].copy_(small.v)
    cache = A.PagedCache(far[0], far[1], small.table, small.lens, k_scale=small.k_scale, v_scale=small.v_scale)
    q = queries(n, 8, d, 32)
    prob = A.PagedAttendProblem(q, cache, i32([0, n]), lse=True, causal=True)
    A.paged_attend(prob)
    verify(prob.out, prob.lse, q, [0, n], P.host(small), causal=True)


@pytest.mark.parametrize("int8", [False, True])
def test_rows_past_two_to_the_28(A, int8):
    # a table of more than 2^24 pages (the same 64 of them again and again), of which the tokens see a window
    d, h, page_rows, n, pages_n = 64, 1, 16, 9, 64
    at, R = (1 << 28) + 5, (1 << 28) + 700
    small = P.build(A, [page_rows * pages_n], h, d, page_rows, seed=34, mass=False, order=False, int8=int8)
    table = small.table[0].repeat(R // (page_rows * pages_n) + 1).reshape(1, -1)
    cache = A.PagedCache(small.k, small.v, table, i32([R]), k_scale=small.k_scale, v_scale=small.v_scale)
    q = queries(n, 4, d, 34)
    begin, end = [at + 10 * i for i in range(n)], [at + 10 * i + 300 for i in range(n)]
    prob = A.PagedAttendProblem(q, cache, i32([0, n]), lse=True, row_begin=i32(begin), row_end=i32(end))
    A.paged_attend(prob)
    base = at // (page_rows * pages_n) * page_rows * pages_n  # (the window lies within one round of the pages)
    verify(prob.out, prob.lse, q, [0, n], P.host(small), begin=[x - base for x in begin], end=[x - base for x in end])


@pytest.mark.parametrize("fused,wide", [(True, 0), (False, 3), (True, 1)])
def test_strides(A, fused, wide):
    for d, int8 in ((128, False), (64, True), (64, False)):
        case(A, [33, 7, 64], [33, 100, 64], 6, 2, d, 32, seed=7, fused=fused, wide=wide, int8=int8, causal=True)
    # views of one projection, every second head, a transposed output
    T, h_q, d = 45, 6, 128
    q = queries(T, 2 * h_q + 3, d, 8)[:, 1:1 + 2 * h_q:2]
    cache = P.build(A, [40, 90, 64], 3, d, 16, seed=8)
    out = torch.full((h_q + 1, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    o = out[:h_q].transpose(0, 1)
    prob = A.PagedAttendProblem(q, cache, i32([0, 20, 40, 45]), out=o, causal=True)
    A.paged_attend(prob)
    verify(o, None, q, [0, 20, 40, 45], P.host(cache), causal=True)
    assert torch.all(out[h_q] == 7.0)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_ranges(A, causal, int8):
    g = np.random.default_rng(11)
    new, lens = [60, 1, 130, 0, 20], [700, 40, 1000, 30, 20]
    T = sum(new)
    begin, end = g.integers(-50, 900, T), g.integers(-50, 1100, T)
    begin[:20], end[:20] = 130, 120                      # nothing at all
    begin[61:100], end[61:100] = -2 ** 31, 2 ** 31 - 1   # everything
    begin[150:], end[150:] = 255, 257                    # two rows across tiles
    for b, e in ((begin, end), (begin, None), (None, end)):
        case(A, new, lens, 14, 2, 128, 32, seed=12, causal=causal, int8=int8, begin=b, end=e)
    case(A, new, lens, 4, 4, 64, 16, seed=13, causal=causal, int8=int8, begin=begin, end=end)


def test_a_window_over_the_last_rows(A):
    new, lens = [100, 300], [900, 300]
    hi = np.concatenate([R - n + 1 + np.arange(n) for n, R in zip(new, lens)])
    case(A, new, lens, 28, 4, 128, 64, seed=14, causal=True, begin=hi - 100)


def test_tokens_that_see_nothing(A):
    case(A, [5, 40], [0, 0], 28, 4, 128, 16, seed=15)
    case(A, [5, 40, 3], [70, 300, 0], 28, 4, 128, 16, seed=15, end=[0] * 48)
    # some rows of a tile only, with NaN where nobody looks
    case(A, [30], [300], 28, 4, 128, 16, seed=15, begin=[400] * 10 + [128] * 10 + [0] * 10, fill=float("nan"))


# A later token's key and value are nobody's but its own (and those behind it): bf16 rows of NaN and infinities
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("h_q,h_kv,n,R,d", [(28, 4, 50, 170, 128), (8, 8, 200, 2600, 64), (14, 2, 9, 6000, 128), (2, 2, 140, 140, 128)])
def test_masked_rows_that_are_not_finite(A, value, h_q, h_kv, n, R, d):
    cache = P.build(A, [R, R], h_kv, d, 32, seed=16, mass=False, order=False)
    q = queries(2 * n, h_q, d, 16)
    cu = [0, n, 2 * n]
    at = R - n + n // 2  # the row of token n // 2
    clean = P.host(cache)
    pg = cache.table[0].long()
    for name in ("k", "v"):
        t = getattr(cache, name)
        t[pg[at // 32], at % 32] = value
        t[pg[(R - 1) // 32], (R - 1) % 32, :, ::3] = value
    prob = A.PagedAttendProblem(q, cache, i32(cu), lse=True, causal=True)
    A.paged_attend(prob)
    want, want_lse, size, spread = O.attend(q.double().cpu().numpy(), cu, clean, d ** -0.5, True)
    got = prob.out.double().cpu().numpy()
    tol = (HALF + 2.0 ** -12) * spread + HALF * np.abs(want)
    free = np.r_[0:n // 2, n:2 * n]  # the tokens before it, and the other sequence
    assert np.all(np.isfinite(got[free])) and np.all(np.abs(got - want)[free] <= tol[free])
    assert not np.isfinite(got[n // 2:n]).any()  # its key has given every logit sum a NaN, an infinity or a zero weight
    assert np.all(np.abs(prob.lse.double().cpu().numpy() - want_lse)[free] < 1e-3)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_stay_in_their_column(A, value):
    n, R, d = 40, 300, 128
    cache = P.build(A, [R], 2, d, 32, seed=17, mass=False, order=False)
    q = queries(n, 14, d, 17, 0.2)
    clean = P.host(cache)
    at = R - n + 11
    cache.v[cache.table[0, at // 32].long(), at % 32, 1, 5] = value
    prob = A.PagedAttendProblem(q, cache, i32([0, n]), causal=True)
    A.paged_attend(prob)
    want, _, size, spread = O.attend(q.double().cpu().numpy(), [0, n], clean, d ** -0.5, True)
    got = prob.out.double().cpu().numpy()
    hit = np.zeros(got.shape, bool)
    hit[11:, 7:, 5] = True
    assert np.all(np.isnan(got[hit]) if np.isnan(value) else got[hit] == value)
    tol = (HALF + 2.0 ** -12) * spread + HALF * np.abs(want)
    assert np.all(np.abs(got - want)[~hit] <= tol[~hit])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("where", ["all see it", "the last token sees it", "everywhere"])
@pytest.mark.parametrize("lens", [[6000, 700], [300] * 40])
def test_values_that_are_not_finite_cost_little(A, lens, where, int8):
    # units in many parts and whole ones; what has to be formed again is formed by tiles as before: a few times as long
    new = [200 if len(lens) == 2 else 9] * len(lens)
    cache = P.build(A, lens, 4, 128, 64, seed=36, mass=False, order=False, int8=int8)
    q = queries(sum(new), 28, 128, 36)
    cu = np.concatenate([[0], np.cumsum(new)])
    good = P.host(cache)
    want, _, size, spread = O.attend(q.double().cpu().numpy(), cu, good, 128 ** -0.5, True)
    nan = torch.zeros(sum(new), dtype=torch.bool)
    for s, n in enumerate(lens):
        at = torch.arange(n, device="cuda") if where == "everywhere" else torch.tensor([70 if where == "all see it" else n - 1], device="cuda")
        pg = cache.table[s].long()[at // 64]
        if int8:
            cache.v_scale[pg, 2, at % 64] = float("nan")
        else:
            cache.v[pg, at % 64, 2] = float("nan")
        nan[int(cu[s + 1]) - 1 if where == "the last token sees it" else int(cu[s]):int(cu[s + 1])] = True
    prob = A.PagedAttendProblem(q, cache, i32(cu.tolist()), causal=True)
    ws = prob.new_workspace()
    A.paged_attend(prob, ws)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    A.aircache_paged_attend(prob, ws)
    end.record()
    end.synchronize()
    got = prob.out.double().cpu().numpy()
    hit = nan[:, None].numpy() & (np.arange(28) // 7 == 2)[None]
    assert np.all(np.isnan(got[hit]))
    tol = (HALF + 2 * 128 * 2.0 ** -24 * size[..., None] + 2.0 ** -18) * spread + HALF * np.abs(want) + 1e-30  # (as in verify: the last, a weight
    # under 2^-126, fp32's smallest, may be 0: at most 6,000 of them times values under 2^7 are 2^-106)
    assert np.all(np.abs(got - want)[~hit] <= tol[~hit])
    assert begin.elapsed_time(end) < 20  # ms (row by row it would be hundreds; by tiles it is a fraction of one)


def test_int8_scales_that_are_not_finite(A):
    n, R = 40, 300
    cache = P.build(A, [R, R], 2, 128, 32, seed=18, mass=False, order=False, int8=True)
    q = queries(2 * n, 14, 128, 18)
    clean = P.host(cache)
    at = R - n + 11
    for t in (cache.k_scale, cache.v_scale):
        t[cache.table[0, at // 32].long(), 1, at % 32] = float("nan")
    cache.k[cache.table[0, at // 32].long(), at % 32, 1] = 0
    prob = A.PagedAttendProblem(q, cache, i32([0, n, 2 * n]), causal=True)
    A.paged_attend(prob)
    want, _, _, spread = O.attend(q.double().cpu().numpy(), [0, n, 2 * n], clean, 128 ** -0.5, True)
    got = prob.out.double().cpu().numpy()
    hit = np.zeros(got.shape, bool)
    hit[11:n, 7:] = True
    assert np.all(np.isnan(got[hit]))
    tol = (HALF + 2.0 ** -12) * spread + HALF * np.abs(want)
    assert np.all(np.abs(got - want)[~hit] <= tol[~hit])


@pytest.mark.parametrize("int8", [False, True])
def test_values_near_the_end_of_the_range(A, int8):
    # the unnormalised sum passes fp32's range, the output does not
    cache = P.build(A, [300, 4000], 2, 128, 32, seed=18, mass=False, order=False, int8=int8)
    q = queries(40, 14, 128, 18, 0.3)
    if int8:
        cache.v.fill_(100)
        cache.v_scale.fill_(3e36)
    else:
        cache.v.fill_(3e38)
    prob = A.PagedAttendProblem(q, cache, i32([0, 20, 40]), causal=True)
    A.paged_attend(prob)
    got = prob.out.double()
    want = 3e38 if int8 else float(torch.tensor(3e38, dtype=torch.bfloat16))
    assert float((got / want - 1).abs().max()) <= 3 * HALF  # (weights and their sum, and the output)


def test_far_apart_logits(A):
    # a few rows have all the weight, the reference moves with almost every tile; and the smallest scales
    case(A, [50, 3], [900, 2000], 14, 2, 128, 64, seed=19, q_scale=60.0, causal=True)
    case(A, [50, 3], [900, 2000], 14, 2, 128, 64, seed=19, scale=1e-30)
    cache = P.build(A, [600], 2, 128, 64, seed=20, mass=False, order=False)
    q = queries(30, 14, 128, 20)
    r = torch.arange(600, device="cuda")
    k = cache.k[cache.table[0].long()[r // 64], r % 64]
    cache.k[cache.table[0].long()[r // 64], r % 64] = (k * (1 + r[:, None, None] / 20)).to(torch.bfloat16)
    prob = A.PagedAttendProblem(q, cache, i32([0, 30]), lse=True)
    A.paged_attend(prob)
    verify(prob.out, prob.lse, q, [0, 30], P.host(cache))


def test_logits_under_the_range_weigh_nothing(A):
    cache = P.build(A, [200, 200], 2, 128, 16, seed=21, mass=False, order=False)
    q = torch.full((60, 14, 128), 3e38, dtype=torch.bfloat16, device="cuda")
    pg = cache.table.long()
    r = torch.arange(200, device="cuda")
    cache.k[pg[0][r // 16], r % 16] = -1.0
    cache.k[pg[1][r // 16], r % 16] = -1.0
    cache.k[pg[1, 3], 7] = 0.0  # one row of the second sequence has the logit 0
    prob = A.PagedAttendProblem(q, cache, i32([0, 30, 60]), lse=True)
    A.paged_attend(prob)
    assert torch.all(prob.out[:30] == 0) and torch.all(torch.isneginf(prob.lse[:30]))
    v = cache.v[pg[1, 3], 7].repeat_interleave(7, 0)
    assert torch.equal(prob.out[30:], v.expand(30, -1, -1)) and torch.all(prob.lse[30:] == 0)


# ------------------------------------------------------------------ use

def test_the_same_call_gives_the_same_bits(A):
    lens, new = [5000, 700, 1], [40, 300, 1]
    cache = P.build(A, lens, 4, 128, 64, seed=22, mass=False, order=False)
    q = queries(sum(new), 28, 128, 22)
    cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    prob = A.PagedAttendProblem(q, cache, cu, lse=True, causal=True)
    ws = prob.new_workspace()
    A.paged_attend(prob, ws)
    first = P.bits(prob.out), P.bits(prob.lse)
    for _ in range(5):
        prob.out.zero_()
        A.paged_attend(prob, ws)
        assert np.array_equal(first[0], P.bits(prob.out)) and np.array_equal(first[1], P.bits(prob.lse))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("h_q,h_kv,new,lens", [(28, 4, [40, 300, 1], [5000, 700, 1]), (9, 1, [3, 17], [6000, 130]),
                                               (8, 8, [70, 129], [2000, 3000])])
def test_what_another_call_left_has_no_say(A, h_q, h_kv, new, lens, int8):
    # between two runs of a call another one leaves large queries and keys wherever the first has rows without a query
    # and slots without a row
    d = 128
    cache = P.build(A, lens, h_kv, d, 64, seed=22, mass=False, order=False, int8=int8)
    q = queries(sum(new), h_q, d, 22)
    cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    prob = A.PagedAttendProblem(q, cache, cu, lse=True, causal=True)
    ws = prob.new_workspace()
    other = P.build(A, [20000], h_kv, d, 64, seed=23, mass=False, order=False, int8=int8)
    loud = [A.PagedAttendProblem(queries(300, h_q, d, 24 + i, scale), other, i32([0, 300]))
            for i, scale in enumerate((1e-3, 1e2, 1e4))]
    A.paged_attend(prob, ws)
    first = P.bits(prob.out), P.bits(prob.lse)
    for turn in range(6):
        A.paged_attend(loud[turn % 3])
        prob.out.zero_()
        A.paged_attend(prob, ws)
        assert np.array_equal(first[0], P.bits(prob.out)) and np.array_equal(first[1], P.bits(prob.lse))


@pytest.mark.parametrize("int8", [False, True])
def test_captured_calls_follow_their_inputs(A, int8):
    # one workspace, lengths and queries that change between replays, on another stream than the default
    S, h_q, h_kv, d, page_rows = 4, 14, 2, 128, 16
    cache = P.build(A, [400, 300, 200, 100], h_kv, d, page_rows, seed=23, int8=int8, mass=False, order=False)
    q = queries(100, h_q, d, 23)
    cu = i32([0, 10, 10, 60, 90])
    prob = A.PagedAttendProblem(q, cache, cu, lse=True, causal=True)
    ws = prob.new_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        A.aircache_paged_attend(prob, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            A.aircache_paged_attend(prob, ws)
            A.aircache_paged_attend(prob, ws)
    torch.cuda.synchronize()
    for turn, (lens, c) in enumerate([((400, 300, 200, 100), (0, 10, 10, 60, 90)), ((17, 0, 50, 99), (0, 0, 0, 50, 100)),
                                      ((399, 1, 128, 16), (0, 99, 100, 100, 100))]):
        cache.lens.copy_(i32(list(lens)))
        cu.copy_(i32(list(c)))
        q.copy_(queries(100, h_q, d, 30 + turn))
        graph.replay()
        torch.cuda.synchronize()
        verify(prob.out, prob.lse, q, c, P.host(cache), causal=True)
        assert A.aircache_get_error(ws) == A.OK


def test_two_calls_at_once(A):
    probs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        cache = P.build(A, [3000, 50], 4, 128, 64, seed=24 + i, mass=False, order=False)
        q = queries(120, 28, 128, 24 + i)
        probs.append((A.PagedAttendProblem(q, cache, i32([0, 100, 120]), lse=True), cache, q))
    torch.cuda.synchronize()
    works = [p.new_workspace() for p, _, _ in probs]
    torch.cuda.synchronize()
    for _ in range(10):
        for (p, _, _), ws, s in zip(probs, works, streams):
            A.aircache_paged_attend(p, ws, s)
    torch.cuda.synchronize()
    for p, cache, q in probs:
        verify(p.out, p.lse, q, [0, 100, 120], P.host(cache))


def test_sequences_may_share_pages(A):
    cache = P.build(A, [200, 200], 2, 128, 16, seed=26, mass=False, order=False)
    cache.table[1].copy_(cache.table[0])
    q = queries(40, 14, 128, 26)
    prob = A.PagedAttendProblem(q, cache, i32([0, 15, 40]))
    A.paged_attend(prob)
    verify(prob.out, None, q, [0, 15, 40], P.host(cache))


# ------------------------------------------------------------------ what the device refuses

@pytest.mark.parametrize("int8", [False, True])
def test_bad_pages_and_lengths(A, int8):
    for change in ("page", "negative page", "long", "negative", "short"):
        cache = P.build(A, [200, 100, 50], 2, 128, 16, seed=27, int8=int8, mass=False, order=False)
        good = P.host(cache)
        q = queries(60, 14, 128, 27)
        if change == "page":
            cache.table[1, 3] = cache.num_pages
        elif change == "negative page":
            cache.table[1, 3] = -1
        else:
            cache.lens[1] = {"long": 4000, "negative": -5, "short": 7}[change]
        out = torch.full((60, 14, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        prob = A.PagedAttendProblem(q, cache, i32([0, 20, 40, 60]), out=out, causal=True)
        ws = prob.new_workspace()
        with pytest.raises(A.AirCacheError) as e:
            A.paged_attend(prob, ws)
        assert e.value.status == A.ERR_DEVICE_BOUNDS
        want = O.attend(q.double().cpu().numpy(), [0, 20, 40, 60], good, 128 ** -0.5, True)
        got = out.double().cpu().numpy()
        rest = np.r_[0:20, 40:60]
        assert np.all(np.abs(got - want[0])[rest] <= ((HALF + 2.0 ** -12) * want[3] + HALF * np.abs(want[0]))[rest])
        if change in ("long", "negative"):
            assert torch.all(out[20:40] == 0)
        ws.zero_()
        cache.table.copy_(torch.from_numpy(good["table"]).cuda())
        cache.lens.copy_(i32([200, 100, 50]))
        A.paged_attend(prob, ws)  # (the workspace is as good as new)
        verify(out, None, q, [0, 20, 40, 60], good, causal=True)


@pytest.mark.parametrize("cu", [[0, 30, 20, 60], [0, 20, 40, 61], [-1, 20, 40, 60], [0, 20, 2 ** 31 - 1, 60], [0, -2 ** 31, 40, 60],
                                [60, 60, 0, 60]])
def test_bad_token_offsets(A, cu):
    cache = P.build(A, [200, 100, 50], 2, 128, 16, seed=28, mass=False, order=False)
    q = queries(60, 14, 128, 28)
    big = torch.full((80, 14, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    prob = A.PagedAttendProblem(q, cache, i32(cu), out=big[10:70])
    with pytest.raises(A.AirCacheError) as e:
        A.paged_attend(prob)
    assert e.value.status == A.ERR_DEVICE_BOUNDS
    assert torch.all(big[:10] == 7.0) and torch.all(big[70:] == 7.0)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("few", [True, False])
def test_offsets_out_of_order_over_many_rows(A, few, int8):
    # the units that CTAs find then differ from CTA to CTA: all of them are cut, none has parts behind the last CTA
    S, T = (4, 60) if few else (40, 2000)
    cache = P.build(A, [9000, 20, 9000, 9000] + [3000] * (S - 4), 2, 128, 64, seed=35, mass=False, order=False, int8=int8)
    q = queries(T, 32, 128, 35)
    for cu in ([0, T, 0] + [T] * (S - 2), [0, T // 2, T // 4, T] + [0] * (S - 4) + [T], [T, 0] * (S // 2) + [T]):
        big = torch.full((T + 20, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        prob = A.PagedAttendProblem(q, cache, i32(cu), out=big[10:T + 10])
        with pytest.raises(A.AirCacheError) as e:
            A.paged_attend(prob)
        assert e.value.status == A.ERR_DEVICE_BOUNDS
        assert torch.all(big[:10] == 7.0) and torch.all(big[T + 10:] == 7.0)


def test_no_tokens_and_no_sequences(A):
    cache = P.build(A, [20, 10], 2, 128, 16, seed=29, mass=False, order=False)
    prob = A.PagedAttendProblem(torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda"), cache, i32([0, 0, 0]))
    assert A.paged_attend(prob).shape == (0, 4, 128)
    out = torch.full((3, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    prob = A.PagedAttendProblem(queries(3, 4, 128), cache, i32([0, 0, 0]), out=out)
    A.paged_attend(prob)
    assert torch.all(out == 7.0)
