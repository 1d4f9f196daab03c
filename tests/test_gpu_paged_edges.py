"""The paged cache's operators, and the int8 storage they share their codes with, at the
ends of their ranges: infinities and NaN, sizes far apart, orders and lengths at int32's
ends, first calls from several threads, bounds that are left to their defaults.

Results are exact or go by the tolerances that test_gpu_paged_decode.py derives."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_utils as P
import test_gpu_paged_decode as D
from conftest import ROOT
from oracle import paged as O

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lvlm_kv_cache_gb300 import build

    build.build()
    from lvlm_kv_cache_gb300 import aircache

    aircache.lib()
    return aircache


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("length", [-1, -2, -5, -(2 ** 31), -(2 ** 31) + 1, -(2 ** 31) + 4, 2 ** 31 - 1])
def test_rotation_reads_nothing_through_a_length_out_of_bounds(A, length):
    n = [3, 5]
    cache = P.build(A, [20, 5], 2, 64, 16, seed=51)
    cache.lens[0] = length
    k = normal(8, 2, 64, seed=52)
    before = P.state(cache)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    A.aircache_rotate(A.RotateProblem(None, k, k.clone(), cache=cache, cu_tokens=i32(0, 3, 8), seen=i32(3, 5)), st)
    assert A.aircache_get_error(st) == A.ERR_DEVICE_BOUNDS
    after = P.state(cache)
    own = int(cache.table[1, 0])
    for name in before:  # sequence 1's five rows are its page's; nothing else is written
        rest = [i for i in range(cache.num_pages) if i != own]
        assert np.array_equal(before[name][rest], after[name][rest]), name
    assert np.array_equal(after["k"][own][:5], P.bits(k[3:]))


@pytest.mark.parametrize("dense", [False, True])
def test_the_first_cuda_call_of_a_thread(A, dense):
    # a thread that has no CUDA context yet: the call binds its device's
    import threading

    q, k, v = normal(2, 4, 128, seed=53), normal(100, 2, 128, seed=54), normal(100, 2, 128, seed=55)
    if dense:
        prob = A.DecodeProblem(q, k, v, offsets=torch.tensor([0, 60, 100], device="cuda"))
        call = A.aircache_decode
    else:
        prob = A.PagedDecodeProblem(q, P.build(A, [70, 33], 2, 128, 16, seed=56))
        call = A.aircache_paged_decode
    ws = prob.new_workspace()
    call(prob, ws)
    want = prob.out.clone()
    prob.out.zero_()
    torch.cuda.synchronize()
    wrong = []

    def run():
        try:
            call(prob, ws)
        except A.AirCacheError as e:
            wrong.append(str(e))

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not wrong and torch.equal(prob.out, want)


def test_first_calls_from_several_threads(A):
    # a fresh process whose threads make their first call at once: each gets the answer of a call alone
    code = """
import sys, threading
sys.path[:0] = [%r, %r + "/tests"]
import torch
import paged_utils as P
from lvlm_kv_cache_gb300 import aircache as A
lens, n = [70, 33], 16
jobs = []
for i in range(n):
    cache = P.build(A, lens, 2, 128, 16, seed=45)
    q = torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(46)).to(torch.bfloat16).cuda()
    prob = A.PagedDecodeProblem(q, cache)
    jobs.append((prob, prob.new_workspace(), torch.cuda.Stream()))
torch.cuda.synchronize()
gate, wrong = threading.Barrier(n), []
def call(prob, ws, stream):
    try:
        gate.wait()
        A.aircache_paged_decode(prob, ws, stream)
    except Exception as e:
        wrong.append(str(e))
threads = [threading.Thread(target=call, args=j) for j in jobs]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not wrong, wrong
assert all(torch.equal(j[0].out, jobs[0][0].out) for j in jobs)
print("same")
""" % (ROOT, ROOT)
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
        assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


@pytest.mark.parametrize("d", [64, 128])
def test_quantized_infinities_are_not_numbers(A, oracle, d):
    # a head with an infinity has the scale inf and codes of 0, which stand for NaN: no infinity changes its sign
    k, v = normal(600, 3, d, seed=1), normal(600, 3, d, seed=2)
    clean = A.quantize_int8(k, v, torch.tensor([0, 100, 350, 600], device="cuda"))
    k[5, 0, 7], k[5, 0, 8], k[120, 1, 0], v[599, 2, d - 1] = INF, -INF, INF, -INF
    k8, v8, ks, vs = A.quantize_int8(k, v, torch.tensor([0, 100, 350, 600], device="cuda"))
    hit = [(k8, ks, 0, slice(0, 100), 0), (k8, ks, 1, slice(100, 350), 1), (v8, vs, 2, slice(350, 600), 2)]
    for codes, scale, u, rows, h in hit:
        assert float(scale[u, h]) == INF and not bool(codes[rows, h].any())
    for codes, scale, was, was_scale, at in ((k8, ks, clean[0], clean[2], hit[:2]), (v8, vs, clean[1], clean[3], hit[2:])):
        same, same_scale = torch.ones_like(codes, dtype=torch.bool), torch.ones_like(scale, dtype=torch.bool)
        for _, _, u, rows, h in at:
            same[rows, h] = False
            same_scale[u, h] = False
        assert torch.equal(codes[same], was[same]) and torch.equal(scale[same_scale], was_scale[same_scale])


def test_quantized_nan_has_the_code_0(A):
    k = normal(64, 2, 64, seed=3)
    k[4, 0, 5] = NAN
    k8, _, _, _ = A.quantize_int8(k, k.clone(), torch.tensor([0, 64], device="cuda"))
    assert int(k8[4, 0, 5]) == 0


@pytest.mark.parametrize("size", [1e-36, 1e-38, 3e-40])
def test_quantized_subnormal_scales(A, size):
    k = (normal(200, 2, 128, seed=4).double() * size).to(torch.bfloat16)
    k8, _, ks, _ = A.quantize_int8(k, k.clone(), torch.tensor([0, 200], device="cuda"))
    x = k.float().cpu().numpy()
    s = (np.abs(x).max((0, 2)) / np.float32(127)).astype(np.float32)
    assert np.array_equal(ks[0].cpu().numpy(), s)
    t = (x / s[None, :, None]).astype(np.float64)
    want = np.clip(np.copysign(np.floor(np.abs(t) + 0.5), t), -127, 127)
    assert np.array_equal(k8.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("d,inter", [(128, False), (64, True)])
@pytest.mark.parametrize("norm", [True, False])
def test_rows_with_nan_or_infinity_are_appended_as_such(A, d, inter, norm):
    # an int8 row that holds a NaN or an infinity reads as NaN throughout: its scale is NaN or infinite and its codes
    # are 0.  All other rows are as if there were none
    n, h_q, h_kv = 40, 4, 2
    q, k, v = normal(n, h_q, d, seed=5), normal(n, h_kv, d, seed=6), normal(n, h_kv, d, seed=7)
    f = 1e4 ** (-np.arange(0, d // 2, 2) / (d // 2))
    turns = A.rotation_table(torch.tensor(f)).cuda()
    w = (1 + 0.3 * normal(d, seed=8).float()).to(torch.bfloat16) if norm else None

    def append(k, v):
        cache = P.build(A, [n], h_kv, d, 16, seed=9, int8=True)
        A.rotate(A.RotateProblem(q, k, v, cache=cache, cu_tokens=i32(0, n), seen=i32(n), turns=turns, k_weight=w,
                                 interleaved=inter))
        return cache

    clean = P.host(append(k, v))
    bad = {0: [(3, 0, 1, NAN), (3, 1, d - 1, NAN), (9, 0, 0, INF), (10, 0, d - 2, -INF), (17, 1, 5, INF), (17, 1, 6, -INF),
               (39, 1, d // 4, NAN), (39, 1, 2, INF)],
           1: [(0, 0, 0, NAN), (3, 1, d - 1, INF), (8, 0, 63, -INF), (9, 1, 4, INF), (9, 1, 5, -INF), (38, 0, 2, NAN),
               (38, 0, 9, -INF)]}
    for x, at in ((k, bad[0]), (v, bad[1])):
        for t, h, e, y in at:
            x[t, h, e] = y
    cache = append(k, v)
    got = P.host(cache)
    pg, r = O.slots(got, 0)
    for name, x, at in (("k", k, bad[0]), ("v", v, bad[1])):
        hit = np.zeros((n, h_kv), bool)
        hit[[t for t, *_ in at], [h for _, h, *_ in at]] = True
        codes, scale = got[name][pg, r], got[name + "_scale"][pg, :, r]
        assert not np.isfinite(scale[hit]).any() and not codes[hit].any()
        nan_in = np.isnan(x.float().cpu().numpy()).any(-1)
        assert np.isnan(scale[nan_in]).all()
        assert np.array_equal(codes[~hit], clean[name][pg, r][~hit])
        assert np.array_equal(scale[~hit], clean[name + "_scale"][pg, :, r][~hit])
    # and the attention over them does not hide them: keys' heads first (all of a head's queries), then values'
    out = A.paged_decode(A.PagedDecodeProblem(q[:1], cache))
    assert bool(torch.isnan(out).all())


@pytest.mark.parametrize("h_q,h_kv", [(7, 1), (16, 1)])
@pytest.mark.parametrize("big", [2.0 ** 40, 2.0 ** 70, INF])
def test_a_large_query_leaves_its_groups_others_alone(A, h_q, h_kv, big):
    # int8 rows: queries enter the product in 16 bits, each head under a power of two of its own
    for wide, cache, prob in D.both_ways(A, [70, 901], h_q, h_kv, 128, 16, 41, int8=True):
        q = D.queries(2, h_q, 128, 42)
        q[:, 1] *= 1e-3
        small, before = q.clone(), P.host(cache)
        q[:, 0] = INF if big == INF else q[:, 0] * big
        small[:, 0] = 0.0
        p = prob(q, lse=True, accumulate=big != INF)
        A.paged_decode(p)
        if big == INF:  # head 0 is NaN; the others' results by the definition
            assert bool(torch.isnan(p.out[:, 0]).all())
            p.out[:, 0] = torch.stack([x.mean(0) for x in (torch.tensor(O.rows(before, "v", s, 0)) for s in range(2))])
            p.lse[:, 0] = torch.log(cache.lens.float())
            D.verify(p, before, small)
        else:
            D.verify(p, before, q)


def test_protected_orders_at_the_ends_of_int32(A):
    import test_gpu_evict as E

    # without recent rows no order is too new, the largest among them
    cache = P.build(A, [300, 40], 2, 64, 16, seed=43)
    cache.order[cache.order % 3 == 1] = 2 ** 31 - 1
    E.check(A, cache, [100, 20], sink=2)
    # seen - recent below int32: every order is at or behind it
    cache = P.build(A, [300, 40], 2, 64, 16, seed=44)
    E.check(A, cache, [100, 20], seen=[-(2 ** 31) + 3, 40], recent=7)


@pytest.mark.parametrize("T,h,tok,head", [(9, 5, 64, 9 * 64), (9, 5, 7 * 64, 64), (2, 2, 128, 192), (3, 2, 128, 5 * 64)])
def test_outputs_of_any_layout_without_overlap(A, T, h, tok, head):
    q = normal(T, h, 64, seed=57)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    turns = A.rotation_table([1e4 ** (-i / 64) for i in range(0, 64, 2)]).cuda()
    want, _ = A.rotate(A.RotateProblem(q, positions=pos, turns=turns))
    buf = torch.zeros(T * tok + h * head, dtype=torch.bfloat16, device="cuda")
    out = buf.as_strided((T, h, 64), (tok, head, 1))
    A.rotate(A.RotateProblem(q, q_out=out, positions=pos, turns=turns))
    assert torch.equal(out, want)


def test_eviction_without_a_bound_takes_tables_of_any_width(A):
    # 30,000 pages of 16 rows to a sequence: more than the longest eviction, though none is that long
    lens = [100, 60]
    tight, wide = (P.build(A, lens, 2, 64, 16, seed=47, max_pages=m) for m in (7, 30000))
    outs = []
    for cache in (tight, wide):
        prob = A.EvictProblem(cache, i32(50, 30), i32(0, 0), seen=i32(*lens), sink=1, recent=4)
        outs.append(A.evict(prob).tolist())
    assert outs == [[50, 30]] * 2
    P.assert_same_state(P.state(tight), P.state(wide))


def test_sizes_of_refused_problems_name_the_reason(A):
    cache = P.build(A, [100], 2, 64, 16, seed=48)
    with pytest.raises(A.AirCacheError) as e:
        A.EvictProblem(cache, i32(50), i32(0), max_rows=A.MAX_EVICT_ROWS + 1).workspace_size()
    assert e.value.status == A.ERR_UNSUPPORTED
    with pytest.raises(A.AirCacheError) as e:
        A.PagedDecodeProblem(normal(1, 2 * 17, 64), cache).workspace_size()
    assert e.value.status == A.ERR_UNSUPPORTED
    with pytest.raises(A.AirCacheError) as e:
        A.EvictProblem(cache, i32(50), i32(0), sink=-1).workspace_size()
    assert e.value.status == A.ERR_INVALID_ARG


def test_a_negative_bound_of_the_rows_is_refused(A):
    cache = P.build(A, [100], 2, 64, 16, seed=49)
    q = normal(1, 4, 64, seed=50)
    with pytest.raises(A.AirCacheError) as e:
        A.paged_decode(A.PagedDecodeProblem(q, cache, total_rows=-5), check=False)
    assert e.value.status == A.ERR_INVALID_ARG


@pytest.mark.parametrize("what", ["mass", "moves"])
def test_smoke_sees_a_wrong_mass_and_wrong_moves(A, monkeypatch, what):
    import __graft_entry__ as g

    if what == "mass":
        right = O.decode

        def decode(q, c, scale):
            out, lse, w, size, spread = right(q, c, scale)
            w[1][0, 3] += 1e-3  # one row of one KV head
            return out, lse, w, size, spread

        monkeypatch.setattr(O, "decode", decode)
    else:
        rule = O.evict_moves

        def moves(*a):  # the last move is not made (the newest rows lie behind keep: there is one)
            kept, to = rule(*a)
            return kept, to[:-1]

        monkeypatch.setattr(O, "evict_moves", moves)
    with pytest.raises(AssertionError):
        g.smoke()


def test_early_decode_behind_a_kernel_that_does_not_write_its_rows(A):
    # two layers' rows are rotated into dense arenas; the kernel just before each early decode writes neither its
    # ranges nor its rows: a rotation of queries, and the decode of the layer before
    n, h, d = 20000, 4, 128
    ks, vs = (normal(2, n, h, d, seed=60 + i) for i in range(2))
    q = normal(2, 28, d, seed=62)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    turns = A.rotation_table([1e4 ** (-i / d) for i in range(0, d, 2)]).cuda()
    arena, q_rot = torch.zeros_like(ks), torch.zeros_like(q)
    offs = torch.tensor([0, 500, n], device="cuda")
    write = [A.RotateProblem(None, ks[i], k_out=arena[i], positions=pos, turns=turns) for i in range(2)]
    turn_q = A.RotateProblem(q, q_out=q_rot, positions=i32(499, n - 1), turns=turns)
    steps = [A.DecodeProblem(q_rot, arena[i], vs[i], offsets=offs, early_cache=True) for i in range(2)]
    ws = [p.new_workspace() for p in steps]

    def run(apart):
        arena.zero_()
        q_rot.zero_()
        torch.cuda.synchronize()
        for call in (lambda: A.aircache_rotate(write[0]), lambda: A.aircache_rotate(write[1]),
                     lambda: A.aircache_rotate(turn_q), lambda: A.aircache_decode(steps[0], ws[0]),
                     lambda: A.aircache_decode(steps[1], ws[1])):
            call()
            if apart:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [p.out.clone() for p in steps]

    want = run(True)
    for _ in range(20):
        got = run(False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the rows of layer 1 are written while layer 0 is decoded
    A.aircache_rotate(turn_q)
    for _ in range(20):
        arena[1].zero_()
        torch.cuda.synchronize()
        A.aircache_rotate(write[1])
        A.aircache_decode(steps[0], ws[0])
        A.aircache_decode(steps[1], ws[1])
        torch.cuda.synchronize()
        assert torch.equal(steps[1].out, want[1])
