"""The paged-cache operators as they are used together: prompts are normed,
rotated and appended; steps append one token each, attend and accumulate mass;
when a sequence outgrows its budget it is evicted; and a compressed cache goes
into pages and is decoded on.  Each call's result is checked against the plain
64-bit form on the cache as it stood before that call."""
import numpy as np
import pytest
import torch

import paged_utils as P
from lvlm_kv_cache_gb300 import workloads as W
from oracle import paged as O
from test_gpu_paged_decode import verify
from test_gpu_evict import expect
from test_gpu_rotate import check as check_rotated

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


@pytest.mark.parametrize("int8", [False, True])
def test_prompts_steps_and_evictions(A, int8):
    S, h_q, h_kv, d, page_rows = 4, 14, 2, 128, 16
    prompts, budget, slack = [150, 3, 64, 90], 96, 16
    cap = [max(p, budget + slack) for p in prompts]
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = P.build(A, cap, h_kv, d, page_rows, seed=1, int8=int8)
    f = 1e4 ** (-np.arange(0, d, 2) / d)
    turns = A.rotation_table(torch.tensor(f)).cuda()
    w = (1 + 0.3 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
    seen = torch.zeros(S, dtype=torch.int32, device="cuda")
    keep = torch.full((S,), budget, dtype=torch.int32, device="cuda")
    lens_out = torch.zeros_like(seen)
    cache.lens.zero_()

    def append(counts):
        T = sum(counts)
        qkv = torch.randn((T, (h_q + 2 * h_kv) * d), generator=g, device="cuda").to(torch.bfloat16)
        q = qkv[:, :h_q * d].view(T, h_q, d)
        k = qkv[:, h_q * d:(h_q + h_kv) * d].view(T, h_kv, d)
        v = qkv[:, (h_q + h_kv) * d:].view(T, h_kv, d)
        n = torch.tensor(counts, dtype=torch.int32, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        seen.add_(n)
        cache.lens.add_(n)
        prob = A.RotateProblem(q, k, v, cache=cache, cu_tokens=cu, seen=seen, turns=turns, q_weight=w[0], k_weight=w[1])
        A.rotate(prob)
        pos = np.concatenate([np.arange(e - c, e) for e, c in zip(seen.tolist(), counts)])
        check_rotated(prob.q_out, q, w[0], 1e-6, pos[:, None] * f, False)
        return prob.q_out

    append(prompts)
    ev = A.EvictProblem(cache, keep, lens_out, seen=seen, sink=2, recent=12)
    ws_e = ev.new_workspace()
    ws_d = None
    evictions = 0
    for step in range(40):
        q = append([1] * S)
        before = P.host(cache)
        prob = A.PagedDecodeProblem(q, cache, lse=True, accumulate=True)
        ws_d = prob.new_workspace() if ws_d is None else ws_d
        A.paged_decode(prob, ws_d)
        verify(prob, before, q)
        if int(cache.lens.max()) >= budget + slack or step == 0:
            st = P.state(cache)
            want, new = expect(st, cache, keep.tolist(), seen.tolist(), 2, 12)
            A.evict(ev, ws_e)
            assert lens_out.tolist() == new
            P.assert_same_state(want, P.state(cache))
            cache.lens.copy_(lens_out)
            evictions += 1
            # the protected tokens are still there, under every head
            c = P.host(cache)
            for s in range(S):
                pg, r = O.slots(c, s)
                for h in range(h_kv):
                    have = set(c["order"][pg, h, r].tolist())
                    e = int(seen[s])
                    assert have >= set(range(min(2, e))) | set(range(max(0, e - 12), e))
    assert evictions >= 3


def test_compressed_cache_goes_on_in_pages(A):
    # prefill compression -> pages -> decode: the compacted rows' attention, then grown by new tokens
    wl = W.make("ragged", seed=31, device="cuda", layers=2, requests=3)
    s = wl.spec
    prob = A.Problem(wl.q, wl.k, wl.v, wl.cu_seqlens, wl.cu_visual, max(s.n_visual), max(s.n_text), alpha=s.alpha,
                     r=s.r, total_tokens=wl.total_tokens, total_visual=wl.total_visual)
    res = A.compress(prob)
    offs = res["out_offsets"].tolist()
    B, layer, page_rows = prob.B, 1, 32
    lens = [offs[layer * B + b + 1] - offs[layer * B + b] for b in range(B)]
    lo, hi = offs[layer * B], offs[(layer + 1) * B]
    cache = P.build(A, [n + 8 for n in lens], s.H_kv, s.D, page_rows, seed=32)
    cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    seen = torch.tensor([a + b for a, b in zip(s.n_visual, s.n_text)], dtype=torch.int32, device="cuda")
    cu = torch.tensor([o - lo for o in offs[layer * B:(layer + 1) * B + 1]], dtype=torch.int32, device="cuda")
    A.rotate(A.RotateProblem(None, res["out_k"][lo:hi], res["out_v"][lo:hi], cache=cache, cu_tokens=cu, seen=seen))
    g = torch.Generator(device="cuda").manual_seed(33)
    q = torch.randn((B, s.H_q, s.D), generator=g, device="cuda").to(torch.bfloat16)
    dec = A.PagedDecodeProblem(q, cache, lse=True, accumulate=True)
    before = P.host(cache)
    A.paged_decode(dec)
    verify(dec, before, q)
    offs_t = res["out_offsets"][layer * B:(layer + 1) * B + 1]
    ref = A.decode(A.DecodeProblem(q, res["out_k"], res["out_v"], offsets=offs_t, max_rows=max(lens)))
    spread = torch.as_tensor(O.decode(q.double().cpu().numpy(), before, s.D ** -0.5)[4], device="cuda")
    half = 2.0 ** -8
    assert bool(((dec.out.double() - ref.double()).abs() <= 3 * half * spread + half * ref.double().abs()).all())


def test_two_layers_on_two_streams_with_their_own_workspaces(A):
    caches = [P.build(A, [3000, 20, 600], 4, 128, 16, seed=40 + i) for i in range(2)]
    g = torch.Generator(device="cuda").manual_seed(41)
    qs = [torch.randn((3, 28, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    probs = [A.PagedDecodeProblem(q, c, lse=True, accumulate=True) for q, c in zip(qs, caches)]
    wss = [p.new_workspace() for p in probs]
    before = [P.host(c) for c in caches]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for p, ws, st in zip(probs, wss, streams):
        with torch.cuda.stream(st):
            A.aircache_paged_decode(p, ws)
    torch.cuda.synchronize()
    for p, b, q, ws in zip(probs, before, qs, wss):
        verify(p, b, q)
        assert A.aircache_get_error(ws) == A.OK


def test_calls_on_a_side_stream_without_a_workspace(A):
    # the conveniences allocate and zero their workspace on the stream that the call uses
    s = torch.cuda.Stream()
    cache = P.build(A, [500, 33], 2, 64, 16, seed=50)
    g = torch.Generator(device="cuda").manual_seed(51)
    q = torch.randn((2, 6, 64), generator=g, device="cuda").to(torch.bfloat16)
    before = P.host(cache)
    busy = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3  # keeps the current stream behind
    prob = A.PagedDecodeProblem(q, cache, lse=True, accumulate=True)
    A.paged_decode(prob, stream=s)
    verify(prob, before, q)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    keep, out = t([100, 20]), t([0, 0])
    torch.cuda.synchronize()
    st = P.state(cache)
    want, new = expect(st, cache, [100, 20], None, 0, 0)
    assert A.evict(A.EvictProblem(cache, keep, out), stream=s).tolist() == new
    P.assert_same_state(want, P.state(cache))


@pytest.mark.parametrize("int8", [False, True])
def test_a_captured_step_equals_the_eager_one(A, int8):
    # append, attend with mass and evict as one graph on a side stream, replayed with new projections and lengths,
    # against the same calls made one by one on a copy of the cache: the same bits
    S, h_q, h_kv, d, page_rows = 5, 10, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(60)
    qkv = torch.randn((S, (h_q + 2 * h_kv) * d), generator=g, device="cuda").to(torch.bfloat16)
    f = 1e4 ** (-np.arange(0, d, 2) / d)
    turns = A.rotation_table(torch.tensor(f)).cuda()
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")

    def world():
        cache = P.build(A, [300, 41, 17, 90, 64], h_kv, d, page_rows, seed=61, int8=int8)
        w = dict(cache=cache, qkv=qkv.clone(), seen=t([400, 41, 20, 95, 64]), keep=t([250, 50, 16, 88, 63]),
                 out=t([0] * S))
        q = w["qkv"][:, :h_q * d].view(S, h_q, d)
        k = w["qkv"][:, h_q * d:(h_q + h_kv) * d].view(S, h_kv, d)
        v = w["qkv"][:, (h_q + h_kv) * d:].view(S, h_kv, d)
        w["rot"] = A.RotateProblem(q, k, v, cache=cache, cu_tokens=cu, seen=w["seen"], turns=turns)
        w["dec"] = A.PagedDecodeProblem(w["rot"].q_out, cache, lse=True, accumulate=True)
        w["ev"] = A.EvictProblem(cache, w["keep"], w["out"], seen=w["seen"], sink=1, recent=4)
        w["ws_d"], w["ws_e"], w["st"] = w["dec"].new_workspace(), w["ev"].new_workspace(), t([0])
        return w

    def step(w):
        A.aircache_rotate(w["rot"], w["st"])
        A.aircache_paged_decode(w["dec"], w["ws_d"])
        A.aircache_evict(w["ev"], w["ws_e"])

    a, b = world(), world()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(b)
    for i in range(3):
        lens = [300 - 9 * i, 41 + i, 17, 90 - 30 * i, 64]
        new = torch.randn(qkv.shape, generator=g, device="cuda").to(torch.bfloat16)
        for w in (a, b):
            w["qkv"].copy_(new)
            w["cache"].lens.copy_(t(lens))
        torch.cuda.synchronize()
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        P.assert_same_state(P.state(a["cache"]), P.state(b["cache"]))
        for x, y in ((a["dec"].out, b["dec"].out), (a["dec"].lse, b["dec"].lse), (a["out"], b["out"]),
                     (a["rot"].q_out, b["rot"].q_out)):
            assert np.array_equal(P.bits(x), P.bits(y))
        for w in (a, b):
            assert [A.aircache_get_error(w[n]) for n in ("st", "ws_d", "ws_e")] == [A.OK] * 3
