"""aircache_paged_decode against its definition in 64 bits (oracle/paged.py).

Tolerances.  A dot product in fp32 over D exact products is off by at most
D 2^-24 sum |q_d k_d| scale =: dx (at the row where that is largest), and a
weight by a relative 2 dx + 2^-20 (two exponentials of that error, the base-2
exponential's own 2^-22, products).  lse: dx + 2^-20 (1 + |lse|).  out: each
weight also becomes a sum of two bf16 before it meets V (2^-8 of 2^-8), or one f16
(2^-11), and out is rounded to bf16: (2^-16 or 2^-11, + 2 dx + 2^-18) sum w |v| + 2^-8 |out|.  int8 rows: the
weight times the value's scale is held in f16, 2^14 to the largest of them, so a
small one is also off by half of f16's least step, 2^-25 / 2^14 of the largest,
which its code (at most 127) multiplies: n 127 2^-39 max w s on top.  mass: the
weights' error and fp32 sums."""
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


def queries(S, h_q, d, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((S, h_q, d), generator=g, device="cuda")).to(torch.bfloat16)


def verify(prob, cache_before, q, scale=None, skip_mass=False):
    c = cache_before
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, lse, w, size, spread = O.decode(q.double().cpu().numpy(), c, scale)
    dx = d * 2.0 ** -24 * size
    got = prob.out.double().cpu().numpy()
    weight = 2.0 ** -16 if c["v_scale"] is None else 2.0 ** -11
    tol = (weight + 2 * dx[..., None] + 2.0 ** -18) * spread + HALF * np.abs(out) + 1e-30
    if c["v_scale"] is not None:
        top = O.largest_weighted_scale(q.double().cpu().numpy(), c, scale)
        tol += (c["lens"][:, None] * 127 * 2.0 ** -39 * top)[..., None]
    assert np.all(np.isfinite(got))
    err = np.abs(got - out)
    assert np.all(err <= tol), f"out: worst {np.max(err / tol):.2f}"
    if prob.lse is not None:
        gl = prob.lse.double().cpu().numpy()
        empty = np.isneginf(lse)
        assert np.array_equal(empty, np.isneginf(gl))
        e = np.abs(gl[~empty] - lse[~empty])
        t = dx[~empty] + 2.0 ** -20 * (1 + np.abs(lse[~empty]))
        assert np.all(e <= t), f"lse: worst {np.max(e / t):.2f}"
    if prob.mass_out is not None and not skip_mass:
        gm = prob.mass_out.double().cpu().numpy()
        h = c["k"].shape[2]
        g = q.shape[1] // h
        for s in range(len(w)):
            pg, r = O.slots(c, s)
            for j in range(h):
                want = c["mass"][pg, j, r].astype(np.float64) + w[s][j]
                rel = 2 * dx[s, j * g:(j + 1) * g].max() + 2.0 ** -20 if len(pg) else 0
                e = np.abs(gm[pg, j, r] - want)
                assert np.all(e <= rel * w[s][j] + 2.0 ** -23 * (np.abs(want) + g)), f"mass of {s}, {j}"


def case(A, lens, h_q, h_kv, d, page_rows, seed=0, q_scale=1.5, fill=None, **kw):
    cache = P.build(A, lens, h_kv, d, page_rows, seed=seed, fill=fill, **kw)
    q = queries(len(lens), h_q, d, seed, q_scale)
    before = P.host(cache)
    prob = A.PagedDecodeProblem(q, cache, lse=True, accumulate=cache.mass is not None)
    A.paged_decode(prob)
    verify(prob, before, q)
    after = P.host(cache)  # nothing but the mass of the attended rows has changed
    used = np.zeros(after["k"].shape[:2], bool)
    for s in range(len(lens)):
        used[O.slots(before, s)] = True
    for n in before:
        if before[n] is None:
            continue
        a, b = before[n], after[n]
        if n == "mass":
            a, b = a.transpose(0, 2, 1)[~used], b.transpose(0, 2, 1)[~used]
        assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), n
    return prob, cache, q


LENS = [1, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 300, 1000, 0]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page_rows", [16, 48, 64, 256])
def test_ragged(A, page_rows, d, int8):
    case(A, LENS, 28, 4, d, page_rows, seed=d + page_rows, int8=int8)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (16, 1), (9, 1), (32, 32), (10, 2), (24, 3)])
def test_heads(A, h_q, h_kv, int8):
    case(A, [77, 5, 200, 0, 64], h_q, h_kv, 128, 32, seed=h_q, int8=int8)


@pytest.mark.parametrize("int8", [False, True])
def test_one_long_sequence_is_joined_from_many_parts(A, int8):
    case(A, [20011], 28, 4, 128, 64, seed=3, int8=int8)
    case(A, [9000, 1], 4, 1, 64, 16, seed=4, int8=int8)


def test_many_short_sequences(A):
    g = np.random.default_rng(5)
    case(A, g.integers(0, 40, 700).tolist(), 4, 2, 64, 16, seed=5)


@pytest.mark.parametrize("int8", [False, True])
def test_slots_behind_the_last_row_hold_anything(A, int8):
    # NaN rows (bf16) or NaN scales (int8) behind the end, in a tile's middle and in its own page
    case(A, [1, 17, 70, 250], 8, 2, 128, 64, seed=6, int8=int8, fill=float("nan"))


@pytest.mark.parametrize("fused,wide", [(True, 0), (False, 3), (True, 1)])
def test_strides(A, fused, wide):
    case(A, [33, 100, 64], 6, 2, 128, 32, seed=7, fused=fused, wide=wide)
    case(A, [33, 100, 64], 6, 2, 64, 32, seed=7, fused=fused, wide=wide, int8=True)
    q = queries(3, 12, 128, 8)[:, ::2]  # strided query heads
    cache = P.build(A, [5, 90, 64], 3, 128, 16, seed=8)
    prob = A.PagedDecodeProblem(q, cache, lse=True)
    A.paged_decode(prob)
    verify(prob, P.host(cache), q)


def test_large_and_small_logits(A):
    for qs in (1e-3, 30.0):
        case(A, [500, 40], 7, 1, 128, 32, seed=9, q_scale=qs)
        case(A, [500, 40], 7, 1, 128, 32, seed=9, q_scale=qs, int8=True)


def test_scale_and_another_mass_array(A):
    cache = P.build(A, [100, 0, 37], 2, 64, 16, seed=10)
    q = queries(3, 8, 64, 10)
    before = P.host(cache)
    out = torch.full_like(cache.mass, -5.0)
    prob = A.PagedDecodeProblem(q, cache, scale=0.31, lse=True, mass_out=out)
    A.paged_decode(prob)
    verify(prob, before, q, scale=0.31)
    assert np.array_equal(before["mass"], cache.mass.cpu().numpy())
    touched = np.zeros(out.shape, bool)
    for s in range(3):
        pg, r = O.slots(before, s)
        touched[pg, :, r] = True
    assert np.all(out.cpu().numpy()[~touched] == -5.0)


def test_int8_scales_of_zero_and_of_any_size(A):
    cache = P.build(A, [90, 64], 2, 128, 32, seed=11, int8=True)
    cache.v_scale.mul_(torch.exp(8 * torch.randn_like(cache.v_scale)))
    cache.v_scale[::2, :, ::3] = 0.0
    cache.k_scale[:, :, ::5] = 0.0
    q = queries(2, 6, 128, 11)
    before = P.host(cache)
    prob = A.PagedDecodeProblem(q, cache, lse=True, accumulate=True)
    A.paged_decode(prob)
    verify(prob, before, q)
    cache.v_scale.zero_()
    A.paged_decode(prob)
    assert not prob.out.any()


def test_repeated_calls_and_workspace_reuse(A):
    cache = P.build(A, [3000, 5, 0, 700], 4, 128, 16, seed=12)
    q = queries(4, 28, 128, 12)
    prob = A.PagedDecodeProblem(q, cache, lse=True)
    ws = prob.new_workspace()
    first = A.paged_decode(prob, ws).clone()
    lse = prob.lse.clone()
    for _ in range(5):
        prob.out.fill_(9.0)
        A.aircache_paged_decode(prob, ws)
    assert torch.equal(first, prob.out) and torch.equal(lse, prob.lse)
    # lengths change on the device between calls; the same problem serves
    cache.lens.copy_(torch.tensor([10, 0, 0, 650], dtype=torch.int32))
    A.paged_decode(prob, ws)
    verify(prob, P.host(cache), q)
    assert A.aircache_get_error(ws) == A.OK


def test_captured_and_replayed_on_another_stream(A):
    cache = P.build(A, [2000, 64, 0, 129], 4, 128, 16, seed=13)
    q = queries(4, 28, 128, 13)
    prob = A.PagedDecodeProblem(q, cache, lse=True, accumulate=True)
    ws = prob.new_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    before = P.host(cache)
    with torch.cuda.stream(s):
        A.aircache_paged_decode(prob, ws)
    s.synchronize()
    verify(prob, before, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        A.aircache_paged_decode(prob, ws)
    for seed in (14, 15):
        q.copy_(queries(4, 28, 128, seed))
        torch.cuda.synchronize()
        before = P.host(cache)
        graph.replay()
        torch.cuda.synchronize()
        verify(prob, before, q)
    assert A.aircache_get_error(ws) == A.OK


def test_shared_pages(A):
    # two sequences with the same prefix pages; the bound of the rows is given, since the rows count twice
    cache = P.build(A, [128, 128, 40], 2, 128, 16, seed=16, mass=False)
    cache.table[1, :4] = cache.table[0, :4]
    q = queries(3, 8, 128, 16)
    prob = A.PagedDecodeProblem(q, cache, lse=True, total_rows=296)
    A.paged_decode(prob)
    verify(prob, P.host(cache), q)
    for s in (0, 1):
        cache.table[s] = cache.table[2, 0]  # the same page again and again
    A.paged_decode(prob)
    verify(prob, P.host(cache), q)


def test_more_rows_than_the_bound(A):
    cache = P.build(A, [100, 60], 2, 64, 16, seed=17)
    q = queries(2, 4, 64, 17)
    prob = A.PagedDecodeProblem(q, cache, accumulate=True, total_rows=150)
    prob.out.fill_(3.0)
    before = P.state(cache)
    ws = prob.new_workspace()
    A.aircache_paged_decode(prob, ws)
    assert A.aircache_get_error(ws) == A.ERR_CAPACITY
    assert bool((prob.out == 3.0).all())
    P.assert_same_state(before, P.state(cache))


def test_bad_lengths_and_pages(A):
    cache = P.build(A, [100, 60, 33, 90], 2, 64, 16, seed=18)
    q = queries(4, 4, 64, 18)
    cache.lens[1] = -4
    cache.lens[2] = 10 ** 6
    prob = A.PagedDecodeProblem(q, cache, lse=True, accumulate=True)
    ws = prob.new_workspace()
    before = P.host(cache)
    A.aircache_paged_decode(prob, ws)
    assert A.aircache_get_error(ws) == A.ERR_DEVICE_BOUNDS
    before["lens"][1:3] = 0
    verify(prob, before, q)
    # a page that does not exist: its rows count as not there
    ws.zero_()
    cache.lens.copy_(torch.tensor([100, 0, 0, 0], dtype=torch.int32))
    good = int(cache.table[0, 2])
    for bad in (-1, cache.num_pages, 2 ** 31 - 1):
        cache.table[0, 2] = bad
        c = P.host(cache)
        A.aircache_paged_decode(prob, ws)
        assert A.aircache_get_error(ws) == A.ERR_DEVICE_BOUNDS
        ws.zero_()
        # the definition over the 84 rows of the other pages
        c["table"][0] = np.concatenate([np.delete(c["table"][0], 2), [0]])
        at = np.concatenate([np.arange(32), np.arange(48, 100)])
        full = P.host(cache)
        out, lse, w, size, spread = O.decode(q[:1].double().cpu().numpy(), sub_rows(full, at), 64 ** -0.5)
        assert np.all(np.abs(prob.out[:1].double().cpu().numpy() - out) <= 2 * HALF * spread + HALF * np.abs(out))
        assert np.allclose(prob.lse[:1].double().cpu().numpy(), lse, rtol=1e-5, atol=1e-5)
    cache.table[0, 2] = good


def sub_rows(c, at):
    """Sequence 0's rows `at` as a cache of their own, one row to a page."""
    pr = c["k"].shape[1]
    pg, r = c["table"][0][at // pr], at % pr
    return dict(k=c["k"][pg, r][:, None], v=c["v"][pg, r][:, None], k_scale=None, v_scale=None, mass=None, order=None,
                table=np.arange(len(at))[None], lens=np.array([len(at)]))


def test_agrees_with_contiguous_decode(A):
    # the same rows through aircache_decode: both are the same attention
    lens = [700, 64, 1]
    cache = P.build(A, lens, 4, 128, 64, seed=19)
    q = queries(3, 28, 128, 19)
    out = A.paged_decode(A.PagedDecodeProblem(q, cache))
    c = P.host(cache)
    ks, vs = [], []
    for s in range(3):
        pg, r = (torch.as_tensor(x, device="cuda") for x in O.slots(c, s))
        ks.append(cache.k[pg.long(), r])
        vs.append(cache.v[pg.long(), r])
    offs = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64, device="cuda")
    ref = A.decode(A.DecodeProblem(q, torch.cat(ks), torch.cat(vs), offsets=offs, max_rows=700))
    spread = torch.as_tensor(O.decode(q.double().cpu().numpy(), c, 128 ** -0.5)[4], device="cuda")
    assert bool(((out.double() - ref.double()).abs() <= 3 * HALF * spread + HALF * ref.double().abs()).all())


def test_elements_past_32_bits(A):
    # pages whose element offsets pass 2^31 (a view of one large buffer: only the few pages in use are written)
    page_rows, h, d = 64, 8, 128
    P_ = 2 ** 31 // (page_rows * h * d) + 40
    k = torch.empty((P_, page_rows, h, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = P.build(A, [64 * 6 + 5], h, d, page_rows, seed=20, mass=False, order=False)
    use = [P_ - 1, 3, P_ - 17, P_ - 2, 11, P_ - 30, P_ - 5]
    for i, pg in enumerate(use):
        k[pg], v[pg] = small.k[small.table[0, i]], small.v[small.table[0, i]]
    table = torch.tensor([use], dtype=torch.int32, device="cuda")
    q = queries(1, 16, d, 20)
    big = A.PagedCache(k, v, table, small.lens)
    assert torch.equal(A.paged_decode(A.PagedDecodeProblem(q, big, total_rows=389)),
                       A.paged_decode(A.PagedDecodeProblem(q, small, total_rows=389)))


@pytest.mark.parametrize("int8", [False, True])
def test_nan_in_a_row_that_counts_is_not_hidden(A, int8):
    # one sequence's keys (or their scales) are all NaN, another's one value; the third is clean
    cache = P.build(A, [40, 300, 70], 2, 128, 16, seed=21, int8=int8)
    q = queries(3, 6, 128, 21)
    if int8:
        cache.k_scale[cache.table[0, :3].long()] = float("nan")
        cache.v_scale[cache.table[1, 9].long(), 0, 5] = float("nan")
    else:
        cache.k[cache.table[0, :3].long()] = float("nan")
        cache.v[cache.table[1, 9].long(), 5, 0, 17] = float("nan")
    prob = A.PagedDecodeProblem(q, cache, lse=True)
    A.paged_decode(prob)
    assert bool(torch.isnan(prob.out[0]).all()) and bool(torch.isnan(prob.lse[0]).all())
    hit = torch.isnan(prob.out[1])
    assert bool(hit[:3, 17].all()) and not bool(hit[3:].any())
    assert bool(torch.isfinite(prob.out[2]).all()) and bool(torch.isfinite(prob.lse[1:]).all())
    one = P.build(A, [70], 2, 128, 16, seed=21, int8=int8)  # the query itself
    q1 = queries(1, 6, 128, 21)
    q1[0, 2] = float("nan")
    p1 = A.PagedDecodeProblem(q1, one, lse=True)
    A.paged_decode(p1)
    assert bool(torch.isnan(p1.out[0, 2]).all())


@pytest.mark.parametrize("int8", [False, True])
def test_logits_below_fp32_weigh_nothing(A, int8):
    # finite keys whose product with one of the queries is under fp32's range, in all of a warp's first rows, in the
    # last ones, and in every row of the second sequence; the group's other queries do not see that element
    cache = P.build(A, [600, 20], 1, 128, 16, seed=22, int8=int8)
    q = queries(2, 6, 128, 22)
    q[:, :, 7] = 0.0
    q[:, 2] = 0.0
    q[:, 2, 7] = 100.0
    lowest = torch.cat([torch.arange(16), torch.arange(64, 97), torch.arange(560, 600)])
    for s, rows in ((0, lowest), (1, torch.arange(20))):
        pg, r = cache.table[s, (rows // 16).cuda()].long(), (rows % 16).cuda()
        cache.k[pg, r] = 0
        cache.k[pg, r, 0, 7] = -127 if int8 else -3e38
        if int8:
            cache.k_scale[pg, 0, r] = 1e36
    before = P.host(cache)
    prob = A.PagedDecodeProblem(q, cache, lse=True, accumulate=True)
    A.paged_decode(prob)
    # (the oracle's weights of those rows are 0: exp of less than -1e38)
    out, lse, w, _, spread = O.decode(q.double().cpu().numpy(), before, 128 ** -0.5)
    seen = np.setdiff1d(np.arange(600), lowest.numpy())
    pg, r = (x[seen] for x in O.slots(before, 0))
    k = before["k"][pg, r, 0].astype(np.float64) * (before["k_scale"][pg, 0, r][:, None] if int8 else 1)
    size = np.abs(k) @ np.abs(q[0].double().cpu().numpy()).T * 128 ** -0.5
    dx = 128 * 2.0 ** -24 * size.max(0)
    tol = ((2.0 ** -11 if int8 else 2.0 ** -16) + 2 * dx[:, None] + 2.0 ** -18) * spread[0] + HALF * np.abs(out[0])
    if int8:
        tol += 600 * 127 * 2.0 ** -39 * before["v_scale"].max()
    assert np.all(np.abs(prob.out[0].double().cpu().numpy() - out[0]) <= tol)
    assert np.all(np.abs(prob.lse[0].double().cpu().numpy() - lse[0]) <= dx + 2.0 ** -20 * (1 + np.abs(lse[0])))
    # no row of the second sequence has a logit in range: none weighs anything for that query
    assert bool((prob.out[1, 2] == 0).all()) and bool(torch.isneginf(prob.lse[1, 2]))
    assert bool(torch.isfinite(prob.out[1]).all()) and bool(torch.isfinite(prob.lse[1, [0, 1, 3, 4, 5]]).all())
    for s, weight in ((0, w[0][0]), (1, None)):
        pg, r = O.slots(before, s)
        got = prob.mass_out.double().cpu().numpy()[pg, 0, r] - before["mass"][pg, 0, r]
        if weight is None:  # (five queries that see equal keys)
            weight = np.full(20, 5 / 20)
            rel = 2.0 ** -20
        else:
            rel = 2 * dx.max() + 2.0 ** -20
        assert np.all(np.abs(got - weight) <= rel * weight + 2.0 ** -23 * (1 + weight + 6))


# The calls above are short by the table and the bound: a cluster to a (sequence, KV head), one kernel.  These
# run the same rows so (tight) and as a list of tiles with a second kernel (wide: a table and a bound for far more).
def both_ways(A, lens, h_q, h_kv, d, page_rows, seed, **kw):
    for wide in (False, True):
        cache = P.build(A, lens, h_kv, d, page_rows, seed=seed, max_pages=80000 // page_rows if wide else None, **kw)
        yield wide, cache, lambda q, **k: A.PagedDecodeProblem(q, cache, total_rows=80000 if wide else max(1, sum(lens)), **k)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,h_q,h_kv,d,page_rows", [
    ([300], 7, 1, 128, 16), ([2048, 0], 28, 4, 128, 64), ([2048], 16, 1, 64, 32), ([1000], 9, 1, 128, 48),
    ([130] * 16, 28, 4, 128, 16), ([64] * 40, 8, 4, 64, 64), ([1] * 30, 10, 2, 128, 16),
    ([700, 3, 0, 64, 65], 32, 32, 64, 16), ([15, 0, 640, 321, 1], 12, 6, 128, 256), (LENS, 28, 4, 128, 48),
    (LENS, 16, 16, 64, 16)])
def test_short_and_long_forms(A, lens, h_q, h_kv, d, page_rows, int8):
    q = queries(len(lens), h_q, d, 41)
    for wide, cache, make in both_ways(A, lens, h_q, h_kv, d, page_rows, 41, int8=int8, fill=float("nan")):
        before = P.host(cache)
        for mass in (True, False):
            prob = make(q, lse=True, accumulate=mass)
            A.paged_decode(prob)
            verify(prob, before, q)


def test_bounds_in_both_forms(A):
    lens, q = [100, 200, 70], queries(3, 8, 128, 42)
    for wide, cache, make in both_ways(A, lens, 8, 2, 128, 16, 42):
        before = P.host(cache)
        prob = make(q, lse=True, accumulate=True)
        # a page out of range: its 16 rows count as not there, and what is reported is that
        cache.table[1, 3] = cache.num_pages
        ws = prob.new_workspace()
        A.aircache_paged_decode(prob, ws)
        with pytest.raises(A.AirCacheError) as e:
            A.paged_decode(prob, ws)
        assert e.value.status == A.ERR_DEVICE_BOUNDS
        cache.mass.copy_(torch.as_tensor(before["mass"]))
        A.aircache_paged_decode(prob, ws)
        rest = np.setdiff1d(np.arange(200), np.arange(48, 64))
        c = {n: before[n] for n in before}
        pg, r = O.slots(before, 1)
        sub = dict(k=c["k"][pg, r][rest][:, None], v=c["v"][pg, r][rest][:, None], k_scale=None, v_scale=None,
                   mass=None, order=None, table=np.arange(len(rest))[None], lens=np.array([len(rest)]))
        out, lse, w, size, spread = O.decode(q[1:2].double().cpu().numpy(), sub, 128 ** -0.5)
        dx = 128 * 2.0 ** -24 * size
        tol = (2.0 ** -16 + 2 * dx[..., None] + 2.0 ** -18) * spread + HALF * np.abs(out)
        assert np.all(np.abs(prob.out[1:2].double().cpu().numpy() - out) <= tol)
        gm = prob.mass_out.double().cpu().numpy()[pg, :, r] - before["mass"][pg, :, r]
        assert np.all(gm[48:64] == 0)
        assert np.all(np.abs(gm[rest] - w[0].T) <= (2 * dx.max() + 2.0 ** -20) * w[0].T + 2.0 ** -23 * 6)
        cache.table[1, 3] = torch.as_tensor(before["table"][1, 3])
        # a bad length counts as 0
        cache.lens[1] = -5
        ws = prob.new_workspace()
        A.aircache_paged_decode(prob, ws)
        with pytest.raises(A.AirCacheError):
            A.paged_decode(prob, ws)
        assert not prob.out[1].any() and bool(torch.isneginf(prob.lse[1]).all())
        cache.lens[1] = 200
        # more rows than the bound: nothing is computed
        small = A.PagedDecodeProblem(q, cache, lse=True, total_rows=369 if not wide else 80000)
        if wide:
            cache.lens[2] = cache.max_pages * 16
        small.out.fill_(7.0)
        with pytest.raises(A.AirCacheError) as e:
            A.paged_decode(small)
        assert e.value.status == A.ERR_CAPACITY
        assert bool((small.out == 7.0).all())


def test_nan_is_not_hidden_by_the_list(A):
    lens, q = [40, 300, 70], queries(3, 6, 128, 43)
    for wide, cache, make in both_ways(A, lens, 6, 2, 128, 16, 43):
        cache.k[cache.table[0, :3].long()] = float("nan")
        cache.v[cache.table[1, 9].long(), 5, 0, 17] = float("nan")
        prob = make(q, lse=True)
        A.paged_decode(prob)
        assert bool(torch.isnan(prob.out[0]).all()) and bool(torch.isnan(prob.lse[0]).all())
        hit = torch.isnan(prob.out[1])
        assert bool(hit[:3, 17].all()) and not bool(hit[3:].any())
        assert bool(torch.isfinite(prob.out[2]).all()) and bool(torch.isfinite(prob.lse[1:]).all())
