"""aircache_rotate against its definition in 64 bits (oracle/paged.py).

Tolerance: fp32 work, rounded once.  The pair (a, b) is right to a few fp32
steps after the norm (sum of D squares, rsqrt, two products: under 2^-20
relative), and the angle to 2^-24 turns = 3.8e-7 for positions up to 2^24 plus
sincospif's step, so before the last rounding |error| <= 2e-6 (|a| + |b|); the
rounding to bf16 adds 2^-8 |y|."""
import numpy as np
import pytest
import torch

import paged_utils as P
from oracle import paged as O

pytestmark = pytest.mark.gpu
PRE, HALF = 2e-6, 2.0 ** -8


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lvlm_kv_cache_gb300 import build

    build.build()
    from lvlm_kv_cache_gb300 import aircache

    aircache.lib()
    return aircache


def freqs(rot, base=1e4):
    return base ** (-np.arange(0, rot, 2) / rot) if rot else np.zeros(0)


def check(got, x, w, eps, angle, inter, pre=PRE):
    y, size = O.rotate(x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), eps, angle, inter)
    err = np.abs(got.double().cpu().numpy() - y)
    tol = HALF * np.abs(y) * (1 + 2.0 ** -7) + pre * size + 1e-30
    assert np.all(err <= tol), f"worst {np.max(err / tol):.2f}"


@pytest.mark.parametrize("d,rot,h_q,h_kv,inter,norm", [
    (128, 128, 28, 4, False, True), (128, 64, 7, 7, False, False), (64, 64, 5, 1, False, True),
    (64, 16, 32, 32, True, False), (128, 128, 1, 1, True, True), (64, 0, 3, 2, False, True),
    (128, 16, 16, 1, False, True), (128, 112, 9, 3, False, False), (64, 48, 9, 3, False, True),
    (64, 48, 4, 4, True, True)])
def test_dense_matches_definition(A, d, rot, h_q, h_kv, inter, norm):
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    for T in (1, 3, 77):
        qkv = torch.randn((T, (h_q + h_kv) * d), generator=g, device="cuda").to(torch.bfloat16)
        q, k = qkv[:, :h_q * d].view(T, h_q, d), qkv[:, h_q * d:].view(T, h_kv, d)
        pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
        w = (1 + 0.3 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16) if norm else [None, None]
        f = freqs(rot)
        turns = A.rotation_table(torch.tensor(f)).cuda() if rot else None
        prob = A.RotateProblem(q, k, positions=pos, turns=turns, q_weight=w[0], k_weight=w[1], eps=1e-5,
                               interleaved=inter)
        qo, ko = A.rotate(prob)
        angle = pos.double().cpu().numpy()[:, None] * f
        check(qo, q, w[0], 1e-5, angle, inter)
        check(ko, k, w[1], 1e-5, angle, inter)


@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 64, True), (64, 64, False), (64, 64, True)])
def test_many_tokens(A, d, rot, inter):
    # more tokens than warps stay on the GPU at once: the kernel's form for long prompts
    g = torch.Generator(device="cuda").manual_seed(6)
    T = 5003
    q = torch.randn((T, 3, d), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((T, 2, d), generator=g, device="cuda").to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = freqs(rot)
    prob = A.RotateProblem(q, k, positions=pos, turns=A.rotation_table(torch.tensor(f)).cuda(), q_weight=w[0],
                           k_weight=w[1], interleaved=inter)
    A.rotate(prob)
    angle = pos.double().cpu().numpy()[:, None] * f
    check(prob.q_out, q, w[0], 1e-6, angle, inter)
    check(prob.k_out, k, w[1], 1e-6, angle, inter)


def test_three_axes(A):
    T, d = 300, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((T, 4, d), generator=g, device="cuda").to(torch.bfloat16)
    f = freqs(d, 1e6)
    for sections in ((16, 24, 24), (64, 0, 0), (0, 0, 64), (1, 62, 1)):
        pos = torch.randint(0, 30000, (3, T), generator=g, device="cuda", dtype=torch.int32)
        prob = A.RotateProblem(q, positions=pos, sections=sections, turns=A.rotation_table(torch.tensor(f)).cuda())
        qo, ko = A.rotate(prob)
        assert ko is None
        axis = np.repeat(np.arange(3), sections)
        check(qo, q, None, 0.0, pos.cpu().numpy().astype(np.float64)[axis].T * f, False)


@pytest.mark.parametrize("top,pre", [(1 << 24, PRE), ((1 << 31) - 1, 3e-5)])
def test_far_positions(A, top, pre):
    # up to 2^24 the table's second float is exact enough; at 2^31 its own rounding, 2^-49 of a frequency of up to
    # 2^-2.6 turns, and the sum with the products' errors (up to 2^5 turns, rounded at 2^-19) make 2^-18 turns = 2.4e-5
    T, d = 500, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((T, 2, d), generator=g, device="cuda").to(torch.bfloat16)
    pos = top - 1 - torch.randint(0, top // 2, (T,), generator=g, device="cuda", dtype=torch.int64)
    pos[0] = top - 1 if top < (1 << 31) else (1 << 31) - 1
    f = freqs(d, 1e4)
    prob = A.RotateProblem(q, positions=pos.to(torch.int32), turns=A.rotation_table(torch.tensor(f)).cuda())
    A.rotate(prob)
    check(prob.q_out, q, None, 0.0, np.fmod(pos.cpu().numpy()[:, None] * f, 2 * np.pi), False, pre)


def test_in_place_and_zero_rows(A):
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((50, 6, 128), generator=g, device="cuda").to(torch.bfloat16)
    q[3] = 0.0  # a row of zeros: eps keeps it finite
    k = torch.randn((50, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    turns = A.rotation_table(torch.tensor(freqs(128))).cuda()
    a = A.RotateProblem(q, k, positions=pos, turns=turns, q_weight=w, k_weight=w)
    A.rotate(a)
    q2, k2 = q.clone(), k.clone()
    A.rotate(A.RotateProblem(q2, k2, q_out=q2, k_out=k2, positions=pos, turns=turns, q_weight=w, k_weight=w))
    assert torch.equal(a.q_out, q2) and torch.equal(a.k_out, k2)
    assert not a.q_out[3].any() and torch.isfinite(a.q_out.float()).all()


def append_case(A, lens_new, lens_old, int8, page_rows, d=128, h_q=7, h_kv=3, pad=0, seed=5, dropped=0, fused=False):
    """Appends lens_new tokens to sequences of lens_old rows; returns everything a check needs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    after = [a + b for a, b in zip(lens_old, lens_new)]
    cache = P.build(A, after, h_kv, d, page_rows, seed=seed, int8=int8, fused=fused)
    T = sum(lens_new) + pad
    qkv = torch.randn((T, (h_q + 2 * h_kv) * d), generator=g, device="cuda").to(torch.bfloat16)
    q = qkv[:, :h_q * d].view(T, h_q, d)
    k = qkv[:, h_q * d:(h_q + h_kv) * d].view(T, h_kv, d)
    v = qkv[:, (h_q + h_kv) * d:].view(T, h_kv, d)
    if sum(lens_new):
        v[0] = 0.0  # a row of zeros: scale 0, codes 0
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens_new)]), dtype=torch.int32, device="cuda")
    seen = torch.tensor([n + dropped for n in after], dtype=torch.int32, device="cuda")
    w = (1 + 0.3 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
    f = freqs(d)
    q_out = torch.full((T, h_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((T, h_kv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    prob = A.RotateProblem(q, k, v, q_out=q_out, k_out=k_out, cache=cache, cu_tokens=cu, seen=seen,
                           turns=A.rotation_table(torch.tensor(f)).cuda(), q_weight=w[0], k_weight=w[1])
    return cache, prob, (q, k, v, w, f, cu, seen)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("page_rows,d,new,old", [
    (16, 128, [1] * 9, [0, 1, 15, 16, 17, 40, 300, 31, 32]),
    (64, 64, [0, 70, 1, 0, 129, 3, 0], [5, 0, 63, 0, 1, 64, 9]),
    (64, 128, [2200, 1, 1800], [0, 50, 7]), (48, 128, [50], [0]), (256, 64, [1, 1], [255, 256]), (16, 128, [1] * 70, list(range(70)))])
def test_append(A, int8, page_rows, d, new, old):
    pad, dropped = 5, 1000
    cache, prob, (q, k, v, w, f, cu, seen) = append_case(A, new, old, int8, page_rows, d, pad=pad, dropped=dropped)
    before = P.host(cache)
    A.rotate(prob)
    after = P.host(cache)
    T = sum(new)
    pos = np.concatenate([np.arange(o + dropped, o + n + dropped) for o, n in zip(old, new)])
    angle = pos[:, None] * f
    check(prob.q_out[:T], q[:T], w[0], 1e-6, angle, False)
    check(prob.k_out[:T], k[:T], w[1], 1e-6, angle, False)
    assert bool((prob.q_out[T:] == 7.0).all()) and bool((prob.k_out[T:] == 7.0).all())  # padding
    want = {n: x for n, x in before.items()}
    yk, size = O.rotate(k[:T].double().cpu().numpy(), w[1].double().cpu().numpy(), 1e-6, angle, False)
    yv = v[:T].double().cpu().numpy()
    t = 0
    for s, (n, o) in enumerate(zip(new, old)):
        for i in range(o, o + n):
            pg, r = after["table"][s][i // page_rows], i % page_rows
            want["mass"][pg, :, r] = 0.0
            want["order"][pg, :, r] = pos[t]
            if not int8:
                assert np.array_equal(after["k"][pg, r], prob.k_out[t].double().cpu().numpy())
                assert np.array_equal(after["v"][pg, r], yv[t])
            for name, y, sz in (("k", yk[t], size[t]), ("v", yv[t], 0 * size[t])):
                if int8:
                    code, sc = after[name][pg, r].astype(np.float64), after[name + "_scale"][pg, :, r].astype(np.float64)
                    top = np.abs(y).max(-1)
                    off = PRE * sz.max(-1)  # the values' own error before the code
                    assert np.all(np.abs(sc * 127 - top) <= off + 2.0 ** -22 * top)
                    # half a step, the error of the values, and the scale's over a code of at most 127
                    assert np.all(np.abs(code * sc[:, None] - y) <= (0.5 + 1e-4) * sc[:, None] + 2 * off[:, None])
                    want[name + "_scale"][pg, :, r] = after[name + "_scale"][pg, :, r]
                want[name][pg, r] = after[name][pg, r]
            t += 1
    for name in want:
        if want[name] is not None:
            assert np.array_equal(want[name], after[name]), name  # nothing else was written


@pytest.mark.parametrize("size", [1.0, 1e30, 1e-36, 1e-38, 3e-40])
def test_int8_values_are_coded_exactly(A, size):
    # values pass unrotated: scale and code are exact functions of the bf16 input, as aircache_quantize_int8's
    # (down to scales that are subnormal, where 1/scale overflows and max/127 is a coarse rounding)
    cache, prob, (q, k, v, *_rest) = append_case(A, [200], [0], True, 32, seed=8)
    v.copy_((v.double() * size).to(torch.bfloat16))
    A.rotate(prob)
    c = P.host(cache)
    x = v.float().cpu().numpy()
    pg, r = O.slots(c, 0)
    s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    assert np.array_equal(c["v_scale"][pg, :, r], s)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(s[..., None] > 0, x / s[..., None], np.float32(0))
    want = np.clip(np.copysign(np.floor(np.abs(t).astype(np.float64) + 0.5), t), -127, 127)
    assert np.array_equal(c["v"][pg, r].astype(np.float64), want)


def test_out_of_bounds_is_reported_and_not_written(A):
    cache, prob, (q, k, v, w, f, cu, seen) = append_case(A, [2, 2, 2], [3, 3, 3], False, 16)
    cache.table[1, 0] = cache.num_pages  # sequence 1: a page that does not exist
    cache.lens[2] = 1                    # sequence 2: two tokens, one row
    before = P.state(cache)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    A.aircache_rotate(prob, st)
    assert A.aircache_get_error(st) == A.ERR_DEVICE_BOUNDS
    after = P.state(cache)
    pg = int(cache.table[0, 0])
    keep = [i for i in range(cache.num_pages) if i != pg and i != int(cache.table[2, 0])]
    for n in before:
        assert np.array_equal(before[n][keep], after[n][keep]), n
    assert not bool((prob.q_out == 7.0).any())  # the queries are written all the same
    cache.lens[2] = 100  # past the table
    A.aircache_rotate(prob, st)
    with pytest.raises(A.AirCacheError):
        A.rotate(prob)


def test_tokens_that_the_batch_does_not_have(A):
    cache, prob, (q, k, v, w, f, cu, seen) = append_case(A, [3, 4], [0, 5], False, 16)
    cu[2] = 9  # seven tokens are there
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    A.aircache_rotate(prob, st)
    assert A.aircache_get_error(st) == A.ERR_DEVICE_BOUNDS


def test_status_of_another_kind_is_refused(A):
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    prob = A.RotateProblem(q)
    for bad in (torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            A.aircache_rotate(prob, bad)


def test_plain_rows_into_pages(A):
    # no norm, no rotation, no queries: what a compacted cache goes through on its way into pages
    cache = P.build(A, [40, 0, 7], 2, 64, 16)
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn((47, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((47, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 40, 40, 47], dtype=torch.int32, device="cuda")
    A.rotate(A.RotateProblem(None, k, v, cache=cache, cu_tokens=cu, seen=cache.lens))
    c = P.host(cache)
    for s, (a, b) in enumerate(((0, 40), (40, 40), (40, 47))):
        pg, r = O.slots(c, s)
        assert np.array_equal(c["k"][pg, r], k[a:b].double().cpu().numpy())
        assert np.array_equal(c["v"][pg, r], v[a:b].double().cpu().numpy())
        assert np.array_equal(c["order"][pg, :, r], np.repeat(np.arange(b - a)[:, None], 2, 1))


def test_nothing_to_do(A):
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert A.rotate(A.RotateProblem(q))[0].shape == (0, 4, 64)
    cache = P.build(A, [0, 0], 2, 64, 16)
    before = P.state(cache)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    A.rotate(A.RotateProblem(None, k, k.clone(), cache=cache, cu_tokens=cu, seen=cache.lens))  # padding only
    P.assert_same_state(before, P.state(cache))


def test_batches_without_sequences(A):
    e = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    pages = e(2, 16, 2, 64, dt=torch.bfloat16)
    cache = A.PagedCache(pages, pages.clone(), e(0, 3), e(0), mass=e(2, 2, 16, dt=torch.float32))
    assert A.paged_decode(A.PagedDecodeProblem(e(0, 4, 64, dt=torch.bfloat16), cache)).shape == (0, 4, 64)
    assert A.evict(A.EvictProblem(cache, e(0), e(0))).shape == (0,)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,d,h_q,h_kv", [((2, 1, 3), 128, 33, 2), ((9, 300, 91), 64, 40, 3), ((700, 1, 1200), 128, 28, 4),
                                            ((2600, 7, 900), 64, 32, 32), ((3000, 60, 2500), 128, 6, 1),
                                            ((39000, 5, 1), 64, 2, 1)])
def test_the_split_of_the_work_changes_nothing(A, new, d, h_q, h_kv, int8):
    # one batch against its sequences one by one: other numbers of warps to a token, the same bits
    T, lens = sum(new), [n + 5 for n in new]
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn((T, h_q + 2 * h_kv, d), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x.split([h_q, h_kv, h_kv], dim=1)
    w = (1 + 0.3 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
    turns = A.rotation_table(torch.tensor(freqs(d))).cuda()
    i32 = lambda *xs: torch.tensor(xs, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    whole, parts = (P.build(A, lens, h_kv, d, 32, seed=32, int8=int8) for _ in range(2))
    kw = dict(turns=turns, q_weight=w[0], k_weight=w[1])
    qo, _ = A.rotate(A.RotateProblem(q, k, v, cache=whole, cu_tokens=i32(*cu), seen=i32(*lens), **kw))
    for s, n in enumerate(new):
        at = slice(cu[s], cu[s + 1])
        one = A.PagedCache(parts.k, parts.v, parts.table[s:s + 1], parts.lens[s:s + 1].clone(), k_scale=parts.k_scale,
                           v_scale=parts.v_scale, mass=parts.mass, order=parts.order)
        qs, _ = A.rotate(A.RotateProblem(q[at], k[at], v[at], cache=one, cu_tokens=i32(0, n), seen=i32(lens[s]), **kw))
        assert np.array_equal(P.bits(qs), P.bits(qo[at]))
    P.assert_same_state(P.state(whole), P.state(parts))
