"""aircache_shared_decode where one half of the softmax has all of the weight, and in a workspace that other calls used.

Tolerances: as in test_gpu_shared_decode.py."""
import numpy as np
import pytest
import torch

import paged_utils as P
from test_gpu_paged_attend import A, i32, queries  # noqa: F401
from test_gpu_shared_decode import verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("own", [60, 9000])
@pytest.mark.parametrize("spoilt", ["prefix", "own"])
def test_a_half_that_weighs_nothing_is_seen_all_the_same(A, spoilt, own, mass, value):  # noqa: F811
    # the joint softmax gives the spoilt half's rows weights of 0 (2^-1000 and less), and 0 times NaN is NaN: as in one
    # decode step over the same rows in one table
    page, p_rows = 16, 320
    cache = P.build(A, [p_rows, own, own], 2, 128, page, seed=50, order=False)
    q = queries(2, 14, 128, 50, 0.0) + 30.0
    pg = cache.table.long()
    for s, n in enumerate([p_rows, own, own]):
        r = torch.arange(n, device="cuda")
        cache.k[pg[s, r // page], r % page] = (0.0 if s == 0 else 1.0) * (1 if spoilt == "prefix" else -1)
    cache.v[pg[0 if spoilt == "prefix" else 1, 2], 5, 1, ::7] = value
    one = torch.cat([cache.table[:1, :p_rows // page].expand(2, -1), cache.table[1:]], 1).contiguous()
    both = A.PagedDecodeProblem(q, A.PagedCache(cache.k, cache.v, one, i32([p_rows + own] * 2)), lse=True,
                                total_rows=2 * (p_rows + own))
    A.paged_decode(both)
    mine = A.PagedCache(cache.k, cache.v, cache.table[1:].contiguous(), i32([own, own]), mass=cache.mass if mass else None)
    prefix = A.PagedCache(cache.k, cache.v, cache.table[:1].contiguous(), i32([p_rows]))
    prob = A.SharedDecodeProblem(q, mine, prefix, i32([0, 2]), lse=True, accumulate=mass)
    A.shared_decode(prob)
    hit = torch.zeros((2, 14, 128), dtype=torch.bool, device="cuda")
    hit[:2 if spoilt == "prefix" else 1, 7:, ::7] = True
    assert torch.isnan(both.out[hit]).all() and torch.isfinite(both.out[~hit]).all()
    assert torch.isnan(prob.out[hit]).all() and torch.isfinite(prob.out[~hit]).all()
    assert torch.isfinite(prob.lse).all()


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("last", [700, 9000])
def test_what_other_groups_left_in_the_workspace_has_no_say(A, last, mass):  # noqa: F811
    # one workspace: a call whose prefixes give every sequence NaN, then calls in which sequences before, between and
    # behind the groups have only their own rows
    lens = [40, 0, 300, 5, 90, 64, last]
    cache = P.build(A, lens, 2, 128, 16, seed=51, mass=mass, order=False)
    good = P.build(A, [200, 130], 2, 128, 32, seed=52, mass=False, order=False)
    spoilt = P.build(A, [200, 130], 2, 128, 32, seed=52, mass=False, order=False)
    spoilt.v.fill_(float("nan"))
    spoilt.k.fill_(float("nan"))
    q, before, p_host = queries(7, 14, 128, 51), P.host(cache), P.host(good)
    out_mass = torch.zeros_like(cache.mass) if mass else None
    make = lambda prefix, cu: A.SharedDecodeProblem(q, cache, prefix, i32(cu), lse=True, mass_out=out_mass)  # noqa: E731
    loud = make(spoilt, [0, 4, 7])
    ws = loud.new_workspace()
    for cu in ([3, 5, 6], [0, 2, 3], [6, 6, 7], [7, 7, 7], [2, 2, 2]):
        A.shared_decode(loud, ws)
        assert torch.isnan(loud.out).all()
        prob = make(good, cu)
        A.shared_decode(prob, ws)
        verify(prob, q, before, p_host, cu)
        alone = make(good, cu)
        A.shared_decode(alone)
        assert np.array_equal(P.bits(prob.out), P.bits(alone.out)) and np.array_equal(P.bits(prob.lse), P.bits(alone.lse))
