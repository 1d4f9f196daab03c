"""aircache_shared_decode where one half of the softmax has all of the weight, in a workspace that other calls used, and
the bits that its weights hold.

Tolerances: as in test_gpu_shared_decode.py, and in the last test without what that one allows for weights of the
prefixes' rows in bf16: they are a sum of two bf16, the second of what the first leaves, 2^-8 of 2^-8 of each weight."""
import numpy as np
import pytest
import torch

import paged_utils as P
from oracle import paged as O
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


@pytest.mark.parametrize("int8,p_int8", [(False, False), (True, True), (False, True), (True, False)])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("q_scale", [0.2, 1.5])
def test_weights_of_a_prefix_hold_the_bits_of_a_decode_step(A, q_scale, d, int8, p_int8):  # noqa: F811
    # many rows of like weight and values of either sign: the output is small beside sum w |v|, and so is its own rounding
    lens, prefix, cu = [0, 5, 70, 0, 300, 0], [3000, 140, 0], [0, 3, 5, 6]
    cache = P.build(A, lens, 2, d, 16, seed=53, mass=False, order=False, int8=int8)
    pre = P.build(A, prefix, 2, d, 64, seed=54, mass=False, order=False, int8=p_int8)
    q = queries(6, 14, d, 53, q_scale / (10 if p_int8 else 1))
    prob = A.SharedDecodeProblem(q, cache, pre, i32(cu), lse=True)
    A.shared_decode(prob)
    qd, c = q.double().cpu().numpy(), P.host(cache)
    out, _, _, size, spread, far = O.shared_decode(qd, c, P.host(pre), cu, d ** -0.5)
    dx = d * 2.0 ** -24 * size
    own = 2.0 ** -11 if int8 else 2.0 ** -16
    tol = (2 * dx[..., None] + 2.0 ** -16) * spread + 2.0 ** -16 * far + own * (spread - far) + 2.0 ** -8 * np.abs(out) + 1e-30
    if int8:  # (f16 under a power of two: as in test_gpu_shared_decode.py)
        tol += (c["lens"][:, None] * 127 * 2.0 ** -39 * O.largest_weighted_scale(qd, c, d ** -0.5))[..., None]
    ratio = np.abs(prob.out.double().cpu().numpy() - out) / tol
    assert np.all(ratio <= 1), f"worst {ratio.max():.2f}"
