"""aircache_evict against its definition (oracle/paged.py): which rows stay,
where the moved ones go, and that every byte of them arrives and no other
changes.  Everything is exact: rows are copied, selections are comparisons."""
import numpy as np
import pytest
import torch

import paged_utils as P
from oracle import paged as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lvlm_kv_cache_gb300 import build

    build.build()
    from lvlm_kv_cache_gb300 import aircache

    aircache.lib()
    return aircache


def expect(st, cache, keep, seen, sink, recent, in_place=True, outs=None):
    """The raw arrays after the eviction, from those before it."""
    pr = cache.page_rows
    table, lens = cache.table.cpu().numpy(), cache.lens.cpu().numpy()
    want = {n: x.copy() for n, x in st.items()}
    if not in_place:
        want["mass"], want["order"] = outs
    mass = cache.mass.cpu().numpy()
    order = None if cache.order is None else cache.order.cpu().numpy()
    new = []
    for s in range(len(lens)):
        n = int(lens[s])
        i = np.arange(n)
        pg, r = table[s][i // pr], i % pr
        new.append(min(n, int(keep[s])))
        for h in range(cache.h_kv):
            kept, moves = O.evict_moves(mass[pg, h, r], None if order is None else order[pg, h, r], int(keep[s]),
                                        int(seen[s]) if seen is not None else 0, sink, recent)
            here = dict((t, f) for f, t in moves)
            for t in (range(new[-1]) if not in_place else here):
                f = here.get(t, t)
                for name in ("mass", "order"):
                    if name in want:
                        want[name][pg[t], h, r[t]] = st[name][pg[f], h, r[f]]
            for f, t in moves:
                for name in ("k", "v"):
                    want[name][pg[t], r[t], h] = st[name][pg[f], r[f], h]
                for name in ("k_scale", "v_scale"):
                    if name in want:
                        want[name][pg[t], h, r[t]] = st[name][pg[f], h, r[f]]
    return want, new


def check(A, cache, keep, seen=None, sink=0, recent=0, in_place=True, max_rows=0, ws=None):
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st = P.state(cache)
    outs = None
    kw = {}
    if not in_place:
        kw["mass_out"] = torch.full_like(cache.mass, -3.0)
        outs = [P.bits(kw["mass_out"]).copy()]
        if cache.order is not None:
            kw["order_out"] = torch.full_like(cache.order, -9)
            outs.append(P.bits(kw["order_out"]).copy())
    want, new = expect(st, cache, keep, seen, sink, recent, in_place, outs)
    lens_out = torch.full_like(cache.lens, -1)
    prob = A.EvictProblem(cache, dev(keep), lens_out, seen=dev(seen), sink=sink, recent=recent, max_rows=max_rows, **kw)
    A.evict(prob, ws)
    assert lens_out.tolist() == new
    got = P.state(cache)
    if not in_place:
        assert np.array_equal(got["mass"], st["mass"])
        got["mass"], got["order"] = P.bits(prob.mass_out), P.bits(prob.order_out)
    P.assert_same_state(want, got)
    return prob


LENS = [0, 1, 5, 16, 17, 64, 100, 300, 1500]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,page_rows", [(128, 16), (64, 48), (64, 256)])
@pytest.mark.parametrize("in_place", [True, False])
def test_ragged(A, d, page_rows, int8, in_place):
    cache = P.build(A, LENS, 3, d, page_rows, seed=d, int8=int8)
    keep = [4, 0, 5, 3, 16, 40, 99, 150, 200]
    check(A, cache, keep, in_place=in_place)


@pytest.mark.parametrize("in_place", [True, False])
def test_protected_rows(A, in_place):
    lens = [40, 200, 1000, 65]
    cache = P.build(A, lens, 2, 128, 16, seed=1)
    # an order with gaps: what is left of a longer stream
    seen = [n + 77 for n in lens]
    cache.order.mul_(1).add_(torch.where(cache.order > 20, 77, 0).to(torch.int32))
    check(A, cache, [30, 60, 300, 64], seen=seen, sink=4, recent=24, in_place=in_place)


def test_keep_equals_the_protected_rows(A):
    lens = [100, 50]
    cache = P.build(A, lens, 2, 64, 16, seed=2)
    check(A, cache, [20, 20], seen=lens, sink=8, recent=12)


def test_sink_only_and_recent_only(A):
    cache = P.build(A, [90], 2, 64, 16, seed=3)
    check(A, cache, [30], sink=10)
    cache = P.build(A, [90], 2, 64, 16, seed=3)
    check(A, cache, [30], seen=[90], recent=25)


@pytest.mark.parametrize("values", ["equal", "few", "zero_signs", "special", "negative"])
def test_ties_and_special_masses(A, values):
    cache = P.build(A, [700, 33, 2100], 2, 64, 16, seed=4, order=False)
    m = cache.mass
    g = torch.Generator(device="cuda").manual_seed(4)
    pick = torch.randint(0, 5, m.shape, generator=g, device="cuda")
    if values == "equal":
        m.fill_(0.25)
    elif values == "few":
        m.copy_(pick.float())
    elif values == "zero_signs":
        m.copy_(torch.where(pick < 2, -0.0, torch.where(pick < 4, 0.0, 1e-42)))
    elif values == "special":
        table = torch.tensor([float("nan"), float("-inf"), float("inf"), 3.4e38, -1.0], device="cuda")
        m.copy_(table[pick])
    else:
        m.mul_(-1.0)
    check(A, cache, [300, 7, 1111])


def test_nothing_to_evict_and_everything(A):
    cache = P.build(A, [10, 64, 0, 500], 2, 128, 16, seed=5)
    check(A, cache, [10, 100, 0, 2 ** 31 - 1])
    check(A, cache, [10, 100, 0, 2 ** 31 - 1], in_place=False)
    check(A, cache, [0, 0, 0, 0])


def test_long_sequences_over_whole_clusters(A):
    # one (sequence, KV head) over eight CTAs, odd lengths; and one that only just fits the selection
    cache = P.build(A, [20011], 1, 64, 64, seed=6)
    check(A, cache, [12345], seen=[20011], sink=3, recent=100)
    cache = P.build(A, [9001, 20], 2, 64, 16, seed=7, int8=True)
    check(A, cache, [1000, 19])


def test_largest_slices(A):
    # 100,000 rows with many units: few CTAs to each, so a slice fills most of a CTA's shared memory
    S, n = 40, [100_000] + [3] * 39
    cache = P.build(A, n, 4, 64, 256, seed=8, order=False)
    check(A, cache, [60_000] + [2] * 39)


def test_the_longest_sequence(A):
    n = A.MAX_EVICT_ROWS - 5
    cache = P.build(A, [n], 1, 64, 256, seed=12, order=False)
    check(A, cache, [150_001], max_rows=A.MAX_EVICT_ROWS)


def test_more_protected_rows_than_places(A):
    # an order that no append makes: every row is "first"; the lowest rows stay
    cache = P.build(A, [500, 40], 2, 64, 16, seed=13)
    cache.order.zero_()
    check(A, cache, [100, 10], sink=1)


def test_again_after_appending(A):
    # an eviction leaves a cache that the next one can cut
    cache = P.build(A, [400, 90], 2, 64, 16, seed=9)
    check(A, cache, [200, 50], seen=[400, 90], recent=16)
    cache.lens.copy_(torch.tensor([200, 50], dtype=torch.int32))
    prob = check(A, cache, [77, 20], seen=[400, 90], recent=16)
    # the same problem and workspace, replayed from a graph on another stream: the lengths are the device's
    ws = prob.new_workspace()
    s = torch.cuda.Stream()
    cache.lens.copy_(torch.tensor([77, 20], dtype=torch.int32))
    prob.keep_alive[1].copy_(torch.tensor([30, 18], dtype=torch.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        A.aircache_evict(prob, ws)
    st = P.state(cache)
    want, new = expect(st, cache, [30, 18], [400, 90], 0, 16)
    graph.replay()
    torch.cuda.synchronize()
    assert prob.lens_out.tolist() == new
    P.assert_same_state(want, P.state(cache))


@pytest.mark.parametrize("what", ["length", "negative", "keep", "protected", "page"])
def test_bad_sequences_are_left_alone(A, what):
    cache = P.build(A, [100, 60], 2, 64, 16, seed=10)
    keep, sink, recent = [50, 30], 2, 3
    if what == "length":
        cache.lens[0] = 10 ** 6
    elif what == "negative":
        cache.lens[0] = -1
    elif what == "keep":
        keep[0] = -1
    elif what == "protected":
        keep[0] = 4
    else:
        cache.table[0, 6] = cache.num_pages
    st = P.state(cache)
    lens = cache.lens.tolist()
    good = A.PagedCache(cache.k, cache.v, cache.table[1:], cache.lens[1:], mass=cache.mass, order=cache.order)
    want, new = expect(st, good, keep[1:], [60], sink, recent)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    prob = A.EvictProblem(cache, t(keep), t([0, 0]), seen=t([100, 60]), sink=sink, recent=recent)
    ws = prob.new_workspace()
    A.aircache_evict(prob, ws)
    assert A.aircache_get_error(ws) == A.ERR_DEVICE_BOUNDS
    assert prob.lens_out.tolist() == [lens[0]] + new
    P.assert_same_state(want, P.state(cache))


def test_lengths_past_max_rows(A):
    cache = P.build(A, [100, 60], 2, 64, 16, seed=11)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    prob = A.EvictProblem(cache, t([50, 30]), t([0, 0]), max_rows=64)
    with pytest.raises(A.AirCacheError):
        A.evict(prob)
    assert prob.lens_out.tolist() == [100, 30]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_rows", [0, 60_000])
@pytest.mark.parametrize("lens,keep,h_kv,d", [
    (LENS, [4, 10, 8, 12, 16, 40, 99, 150, 200], 3, 128), ([3001, 700], [1500, 650], 2, 64),
    ([5003, 8000], [5002, 300], 2, 128), ([16003], [9000], 3, 64), ([400] * 50, [200] * 50, 4, 64)])
def test_moves_by_the_selecting_ctas_and_by_others(A, lens, keep, h_kv, d, max_rows, in_place, int8):
    # a close bound: one kernel, of one to eight CTAs to a (sequence, KV head); a far one: two kernels
    cache = P.build(A, lens, h_kv, d, 16, seed=33, int8=int8)
    check(A, cache, keep, seen=lens, sink=2, recent=2, max_rows=max_rows, in_place=in_place)
