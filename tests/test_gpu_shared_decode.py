"""aircache_shared_decode against its definition in 64 bits (oracle/paged.py): a softmax over the prefix's rows and the
sequence's own.

Tolerances: those of aircache_paged_decode for the own rows (test_gpu_paged_decode.py) and of aircache_paged_attend for
the prefix's, whose weights are rounded to bf16 (2^-8 of each, of the prefix's part of sum w |v| alone).  Joining the two
log-sum-exps, whose own rounding is 2^-24 of up to some hundred, adds 2^-16 to every weight's relative error."""
import numpy as np
import pytest
import torch

import paged_utils as P
from oracle import paged as O
from test_gpu_paged_attend import A, HALF, i32, queries  # noqa: F401

pytestmark = pytest.mark.gpu


def verify(prob, q, c, prefix, cu, mass_before=None):
    d = q.shape[2]
    qd = q.double().cpu().numpy()
    out, lse, w, size, spread, far = O.shared_decode(qd, c, prefix, cu, d ** -0.5)
    dx = d * 2.0 ** -24 * size
    got = prob.out.double().cpu().numpy()
    weight = 2.0 ** -16 if c["v_scale"] is None else 2.0 ** -11
    tol = (weight + 2 * dx[..., None] + 2.0 ** -16) * spread + HALF * far + HALF * np.abs(out) + 1e-30
    if c["v_scale"] is not None:
        tol += (c["lens"][:, None] * 127 * 2.0 ** -39 * O.largest_weighted_scale(qd, c, d ** -0.5))[..., None]
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
    if prob.mass_out is not None:
        gm = prob.mass_out.double().cpu().numpy()
        h = c["k"].shape[2]
        g = q.shape[1] // h
        for s in range(len(w)):
            pg, r = O.slots(c, s)
            for j in range(h if len(pg) else 0):
                want = c["mass"][pg, j, r].astype(np.float64) + w[s][j]
                rel = 2 * dx[s, j * g:(j + 1) * g].max() + 2.0 ** -16
                e = np.abs(gm[pg, j, r] - want)
                assert np.all(e <= rel * w[s][j] + 2.0 ** -23 * (np.abs(want) + g)), f"mass of {s}, {j}"


def case(A, groups, prefix, lens, h_q, h_kv, d, page_rows=16, p_page=32, seed=0, int8=False, p_int8=None, mass=False,  # noqa: F811
         q_scale=1.5, fill=None, first=0, **kw):
    """groups: members of each prefix, from sequence `first` on; those before and behind them have none."""
    S = len(lens)
    cache = P.build(A, lens, h_kv, d, page_rows, seed=seed, int8=int8, mass=mass, order=False, fill=fill)
    pre = P.build(A, prefix, h_kv, d, p_page, seed=seed + 100, int8=int8 if p_int8 is None else p_int8, mass=False,
                  order=False, fill=fill)
    cu = first + np.concatenate([[0], np.cumsum(groups)])
    q = queries(S, h_q, d, seed, q_scale)
    before, p_before, p_state = P.host(cache), P.host(pre), P.state(pre)
    prob = A.SharedDecodeProblem(q, cache, pre, i32(cu.tolist()), lse=True, accumulate=mass, **kw)
    A.shared_decode(prob)
    verify(prob, q, before, p_before, cu)
    P.assert_same_state(p_state, P.state(pre))
    return prob, cache, pre, q, cu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("d", [128, 64])
def test_groups(A, d, mass, int8):  # noqa: F811
    # prefixes of every kind, one of them empty, one without members; sequences without own rows and without a prefix
    lens = [0, 5, 64, 700, 1, 33, 0, 128, 90, 300, 0, 17]
    case(A, [3, 0, 1, 5], [300, 50, 0, 129], lens, 28, 4, d, seed=d, int8=int8, mass=mass)
    case(A, [3, 0, 1, 8], [128, 1, 17, 2000], lens, 8, 8, d, seed=d, int8=int8, mass=mass)


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("last", [700, 9000])
def test_sequences_before_the_first_group(A, last, mass):  # noqa: F811
    # (twice: the second call's workspace holds what other sequences got in the first)
    lens = [40, 0, 300, 5, 90, 64, last]
    for first in (0, 3):
        case(A, [2, 1], [200, 130], lens, 14, 2, 128, seed=8, mass=mass, first=first)


@pytest.mark.parametrize("int8,p_int8", [(False, True), (True, False)])
def test_rows_of_two_kinds(A, int8, p_int8):  # noqa: F811
    case(A, [4, 2], [400, 33], [5, 90, 200, 1, 64, 65], 14, 2, 128, seed=1, int8=int8, p_int8=p_int8, mass=True)


@pytest.mark.parametrize("mass", [False, True])
def test_long_own_rows(A, mass):  # noqa: F811
    # the list form of the decode: parts joined by its second kernel
    case(A, [2, 1], [1000, 77], [5000, 9000, 70, 8000], 28, 4, 128, 64, 64, seed=2, mass=mass)
    case(A, [1], [5000], [20000], 16, 1, 128, 64, 64, seed=3, mass=mass, int8=True)


def test_many_members_of_a_long_prefix(A):  # noqa: F811
    g = np.random.default_rng(4)
    case(A, [70], [9001], g.integers(0, 100, 75).tolist(), 14, 2, 128, 16, 256, seed=4)
    case(A, [150], [500], g.integers(0, 100, 150).tolist(), 1, 1, 128, 16, 16, seed=5)
    case(A, [1] * 40, g.integers(0, 300, 40).tolist(), g.integers(0, 100, 40).tolist(), 16, 1, 64, 16, 16, seed=6)


def test_without_prefixes_it_is_the_paged_decode(A):  # noqa: F811
    lens = [0, 5, 640, 70]
    for prefix, cu in (([], [0]), ([300, 40], [0, 0, 0]), ([0, 0], [0, 2, 4])):
        prob, cache, _, q, _ = case(A, np.diff(cu).tolist(), prefix, lens, 14, 2, 128, seed=7)
        other = A.PagedDecodeProblem(q, cache, lse=True)
        A.paged_decode(other)
        assert np.array_equal(P.bits(prob.out), P.bits(other.out)) and np.array_equal(P.bits(prob.lse), P.bits(other.lse))


def test_far_apart_halves(A):  # noqa: F811
    # either half may have all of the weight
    case(A, [3], [500], [300, 300, 300, 5], 14, 2, 128, seed=8, q_scale=40.0, mass=True)
    case(A, [3], [130], [300, 300, 300, 5], 14, 2, 128, seed=9, fill=float("nan"))


def test_not_a_number_in_a_prefix_or_a_sequence(A):  # noqa: F811
    cache = P.build(A, [100, 100, 100, 100], 2, 128, 16, seed=10, mass=False, order=False)
    pre = P.build(A, [200, 200], 2, 128, 16, seed=11, mass=False, order=False)
    q = queries(4, 14, 128, 10)
    clean, p_clean = P.host(cache), P.host(pre)
    pre.k[pre.table[1, 3].long(), 3] = float("nan")
    cache.v[cache.table[0, 2].long(), 5] = float("nan")
    prob = A.SharedDecodeProblem(q, cache, pre, i32([0, 2, 3]), lse=True)
    A.shared_decode(prob)
    out, lse, _, _, spread, _ = O.shared_decode(q.double().cpu().numpy(), clean, p_clean, [0, 2, 3], 128 ** -0.5)
    got = prob.out.double().cpu().numpy()
    assert np.all(np.isnan(got[[0, 2]]))
    assert np.all(np.abs(got - out)[[1, 3]] <= (2 * HALF * spread + HALF * np.abs(out))[[1, 3]])


def test_shared_pages_of_one_pool(A):  # noqa: F811
    # own rows and prefix in the same pool, two prefixes that are one
    cache = P.build(A, [100, 30, 60, 200, 250], 2, 128, 16, seed=12, mass=False, order=False)
    own = A.PagedCache(cache.k, cache.v, cache.table[:3].contiguous(), cache.lens[:3].contiguous())
    pre = A.PagedCache(cache.k, cache.v, cache.table[3:4].expand(2, -1).contiguous(), i32([200, 200]))
    q = queries(3, 14, 128, 12)
    prob = A.SharedDecodeProblem(q, own, pre, i32([0, 1, 3]), lse=True)
    A.shared_decode(prob)
    verify(prob, q, P.host(own), P.host(pre), [0, 1, 3])


def test_captured_steps_follow_their_inputs(A):  # noqa: F811
    cache = P.build(A, [600, 40, 200, 100], 2, 128, 16, seed=13, order=False)
    pre = P.build(A, [500, 90], 2, 128, 32, seed=14, mass=False, order=False)
    q = queries(4, 14, 128, 13)
    cu = i32([0, 2, 4])
    out_mass = torch.zeros_like(cache.mass)
    prob = A.SharedDecodeProblem(q, cache, pre, cu, lse=True, mass_out=out_mass)
    ws = prob.new_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        A.aircache_shared_decode(prob, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            A.aircache_shared_decode(prob, ws)
            A.aircache_shared_decode(prob, ws)
    torch.cuda.synchronize()
    for turn, (lens, p_lens, c) in enumerate([((600, 40, 200, 100), (500, 90), (0, 2, 4)), ((0, 3, 4, 5), (17, 0), (0, 4, 4)),
                                              ((300, 0, 16, 64), (0, 64), (0, 1, 3))]):
        cache.lens.copy_(i32(list(lens)))
        pre.lens.copy_(i32(list(p_lens)))
        cu.copy_(i32(list(c)))
        q.copy_(queries(4, 14, 128, 40 + turn))
        graph.replay()
        torch.cuda.synchronize()
        verify(prob, q, P.host(cache), P.host(pre), list(c))
        assert A.aircache_get_error(ws) == A.OK


def test_bad_prefixes(A):  # noqa: F811
    for change in ("page", "long", "offsets", "past the end"):
        cache = P.build(A, [100, 30, 60, 20], 2, 128, 16, seed=15, mass=False, order=False)
        pre = P.build(A, [200, 90], 2, 128, 16, seed=16, mass=False, order=False)
        q = queries(4, 14, 128, 15)
        cu = i32([0, 2, 4])
        good, p_good = P.host(cache), P.host(pre)
        if change == "page":
            pre.table[1, 2] = -3
        elif change == "long":
            pre.lens[1] = 10 ** 6
        else:
            cu.copy_(i32([0, 2, 1] if change == "offsets" else [0, 2, 5]))
        prob = A.SharedDecodeProblem(q, cache, pre, cu, lse=True)
        ws = prob.new_workspace()
        with pytest.raises(A.AirCacheError) as e:
            A.shared_decode(prob, ws)
        assert e.value.status == A.ERR_DEVICE_BOUNDS
        got = prob.out.double().cpu().numpy()
        if change in ("page", "long"):
            want = O.shared_decode(q.double().cpu().numpy(), good, p_good, [0, 2, 4], 128 ** -0.5)
            assert np.all(np.abs(got - want[0])[:2] <= (2 * HALF * want[4] + HALF * np.abs(want[0]))[:2])
        ws.zero_()
        pre.table.copy_(torch.from_numpy(p_good["table"]).cuda())
        pre.lens.copy_(i32([200, 90]))
        cu.copy_(i32([0, 2, 4]))
        A.shared_decode(prob, ws)
        verify(prob, q, good, p_good, [0, 2, 4])
