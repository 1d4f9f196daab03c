"""Attention of several tokens and shared prefixes as they are used: an image prompt is appended once and attended chunk
by chunk; chats continue it with questions of their own, decode over the shared rows and their own, and evict their own;
an evicted cache is continued; and an encoder's states are cross-attended by prompts and by single tokens.  Each call's
result is checked against the plain 64-bit form on the caches as they stood before it."""
import numpy as np
import pytest
import torch

import paged_utils as P
from oracle import paged as O
from test_gpu_evict import expect
from test_gpu_paged_attend import A, HALF, i32, verify as verify_attend  # noqa: F401
from test_gpu_paged_decode import verify as verify_decode
from test_gpu_shared_decode import verify as verify_shared

pytestmark = pytest.mark.gpu


class Layer:
    """A layer's projections and their append."""

    def __init__(self, A, h_q, h_kv, d, seed):  # noqa: F811
        self.A, self.h_q, self.h_kv, self.d = A, h_q, h_kv, d
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.turns = A.rotation_table(1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()

    def append(self, cache, counts, seen, rotate=True):
        """New rows of each sequence behind the others; returns the queries and cu_tokens."""
        A, T = self.A, sum(counts)  # noqa: F811
        qkv = torch.randn((T, (self.h_q + 2 * self.h_kv) * self.d), generator=self.g, device="cuda").to(torch.bfloat16)
        a, b = self.h_q * self.d, (self.h_q + self.h_kv) * self.d
        q, k, v = qkv[:, :a].view(T, self.h_q, self.d), qkv[:, a:b].view(T, self.h_kv, self.d), qkv[:, b:].view(T, self.h_kv, self.d)
        cu = i32(np.concatenate([[0], np.cumsum(counts)]).tolist())
        seen.add_(i32(counts))
        cache.lens.add_(i32(counts))
        prob = A.RotateProblem(q, k, v, cache=cache, cu_tokens=cu, seen=seen, turns=self.turns if rotate else None)
        return A.rotate(prob)[0], cu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("h_q,h_kv,d", [(14, 2, 128), (4, 4, 64)])
def test_chats_about_one_prompt(A, h_q, h_kv, d, int8):  # noqa: F811
    layer = Layer(A, h_q, h_kv, d, 1)
    # the prompts, chunk by chunk: the attention over the rows so far equals that of one pass
    pre = P.build(A, [410, 90], h_kv, d, 32, seed=1, int8=int8)
    pre.lens.zero_()
    seen = i32([0, 0])
    for counts in ([200, 64], [150, 0], [60, 26]):
        q, cu = layer.append(pre, counts, seen)
        prob = A.PagedAttendProblem(q, pre, cu, lse=True, causal=True)
        A.paged_attend(prob)
        verify_attend(prob.out, prob.lse, q, cu.tolist(), P.host(pre), causal=True)
    # five chats: three of the first prompt, one of the second, one of its own
    cu_seqs, owner = i32([0, 3, 4]), [0, 0, 0, 1, 2]
    cap = [80] * 5
    own = P.build(A, cap, h_kv, d, 16, seed=2, int8=int8)
    own.lens.zero_()
    seen = i32([0] * 5)
    # their questions see the prompt, whose rows are not theirs, and their own: two attentions joined by log-sum-exp
    counts = [30, 17, 1, 44, 25]
    q, cu = layer.append(own, counts, seen)
    mine = A.PagedAttendProblem(q, own, cu, lse=True, causal=True)
    A.paged_attend(mine)
    verify_attend(mine.out, mine.lse, q, cu.tolist(), P.host(own), causal=True)
    T = [sum(counts[:3]), counts[3]]
    far = A.PagedAttendProblem(q[:sum(T)], pre, i32([0, T[0], sum(T)]), lse=True)
    A.paged_attend(far)
    verify_attend(far.out, far.lse, q[:sum(T)], [0, T[0], sum(T)], P.host(pre))
    # steps: append one token, attend over both, accumulate the own rows' mass, evict the own rows once
    lens_out = i32([0] * 5)
    ws_s = ws_e = None
    for step in range(36):
        q, cu = layer.append(own, [1] * 5, seen)
        before, p_before = P.host(own), P.host(pre)
        prob = A.SharedDecodeProblem(q, own, pre, cu_seqs, lse=True, accumulate=True)
        ws_s = prob.new_workspace() if ws_s is None else ws_s
        A.shared_decode(prob, ws_s)
        verify_shared(prob, q, before, p_before, [0, 3, 4])
        if step == 20:
            ev = A.EvictProblem(own, i32([40] * 5), lens_out, seen=seen, sink=1, recent=8)
            ws_e = ev.new_workspace()
            want, new = expect(P.state(own), own, [40] * 5, seen.tolist(), 1, 8)
            A.evict(ev, ws_e)
            assert lens_out.tolist() == new
            P.assert_same_state(want, P.state(own))
            own.lens.copy_(lens_out)
    # an evicted cache goes on with several tokens at a time (drafts, a further question)
    for counts in ([4] * 5, [3, 9, 0, 1, 2]):
        q, cu = layer.append(own, counts, seen)
        prob = A.PagedAttendProblem(q, own, cu, lse=True, causal=True)
        A.paged_attend(prob)
        verify_attend(prob.out, prob.lse, q, cu.tolist(), P.host(own), causal=True)
    assert len(owner) == 5


@pytest.mark.parametrize("int8", [False, True])
def test_cross_attention_to_images(A, int8):  # noqa: F811
    # an encoder's states (no rotation) of three requests with images of different size, appended image by image; text
    # that sees the images before it; then single tokens, which see all of them
    h_q, h_kv, d = 10, 2, 128
    layer = Layer(A, h_q, h_kv, d, 3)
    images = [[100, 257], [64, 1], [0, 0]]
    cache = P.build(A, [357, 65, 0], h_kv, d, 16, seed=3, int8=int8)
    cache.lens.zero_()
    seen = i32([0, 0, 0])
    for i in range(2):
        layer.append(cache, [x[i] for x in images], seen, rotate=False)
    text = [[5, 30, 7], [0, 2, 40], [3, 4, 0]]  # words before the first image, between the two, behind
    end = np.concatenate([np.repeat([0, im[0], sum(im)], t) for im, t in zip(images, text)])
    T = [sum(t) for t in text]
    q = torch.randn((sum(T), h_q, d), generator=layer.g, device="cuda").to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(T)])
    prob = A.PagedAttendProblem(q, cache, i32(cu.tolist()), lse=True, row_end=i32(end.tolist()))
    A.paged_attend(prob)
    verify_attend(prob.out, prob.lse, q, cu, P.host(cache), end=end)
    assert torch.all(prob.out[:5] == 0) and torch.all(torch.isneginf(prob.lse[:5]))
    # a token each: the same rows by the call for single tokens
    q = torch.randn((3, h_q, d), generator=layer.g, device="cuda").to(torch.bfloat16)
    one = A.PagedAttendProblem(q, cache, i32([0, 1, 2, 3]), lse=True)
    A.paged_attend(one)
    verify_attend(one.out, one.lse, q, [0, 1, 2, 3], P.host(cache))
    dec = A.PagedDecodeProblem(q, cache, lse=True)
    A.paged_decode(dec)
    verify_decode(dec, P.host(cache), q)
    assert float((dec.lse - one.lse)[:2].abs().max()) < 1e-4


def test_a_step_in_a_graph_equals_the_eager_one(A):  # noqa: F811
    # append, attention of the appended tokens and a shared step as one graph, replayed with other projections and lengths
    h_q, h_kv, d, S = 10, 2, 64, 4
    qkv = torch.randn((S, (h_q + 2 * h_kv) * d), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(torch.bfloat16)
    turns = A.rotation_table(1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()

    def world():
        w = dict(own=P.build(A, [300, 41, 17, 90], h_kv, d, 16, seed=6), pre=P.build(A, [700, 60], h_kv, d, 32, seed=7),
                 qkv=qkv.clone(), seen=i32([300, 41, 17, 90]))
        a, b = h_q * d, (h_q + h_kv) * d
        w["rot"] = A.RotateProblem(w["qkv"][:, :a].view(S, h_q, d), w["qkv"][:, a:b].view(S, h_kv, d), w["qkv"][:, b:].view(S, h_kv, d),
                                   cache=w["own"], cu_tokens=i32([0, 1, 2, 3, 4]), seen=w["seen"], turns=turns)
        w["att"] = A.PagedAttendProblem(w["rot"].q_out, w["own"], i32([0, 1, 2, 3, 4]), lse=True, causal=True)
        w["sh"] = A.SharedDecodeProblem(w["rot"].q_out, w["own"], w["pre"], i32([0, 3, 4]), lse=True, accumulate=True)
        w["ws_a"], w["ws_s"], w["st"] = w["att"].new_workspace(), w["sh"].new_workspace(), i32([0])
        return w

    def step(w):
        A.aircache_rotate(w["rot"], w["st"])
        A.aircache_paged_attend(w["att"], w["ws_a"])
        A.aircache_shared_decode(w["sh"], w["ws_s"])

    a, b = world(), world()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(b)
    for i in range(3):
        new = torch.randn(qkv.shape, generator=torch.Generator(device="cuda").manual_seed(8 + i), device="cuda").to(torch.bfloat16)
        for w in (a, b):
            w["qkv"].copy_(new)
            w["own"].lens.copy_(i32([300 - 9 * i, 41, 17 - i, 90 - 30 * i]))
            w["pre"].lens.copy_(i32([700 - 200 * i, 60]))
        torch.cuda.synchronize()
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        P.assert_same_state(P.state(a["own"]), P.state(b["own"]))
        for n in ("att", "sh"):
            assert np.array_equal(P.bits(a[n].out), P.bits(b[n].out)) and np.array_equal(P.bits(a[n].lse), P.bits(b[n].lse))
        for w in (a, b):
            assert [A.aircache_get_error(w[n]) for n in ("st", "ws_a", "ws_s")] == [A.OK] * 3


def test_many_calls_one_behind_the_other(A):  # noqa: F811
    # layers of a step on one stream with nothing between the calls: each kernel starts while the one before ends
    layers = []
    for i in range(6):
        own = P.build(A, [900 - 100 * i, 40, 3], 4, 128, 16, seed=20 + i, order=False)
        pre = P.build(A, [1500], 4, 128, 64, seed=30 + i, mass=False, order=False)
        g = torch.Generator(device="cuda").manual_seed(40 + i)
        q = (1.5 * torch.randn((3, 28, 128), generator=g, device="cuda")).to(torch.bfloat16)
        layers.append((own, pre, q, A.SharedDecodeProblem(q, own, pre, i32([0, 2]), lse=True, mass_out=torch.zeros_like(own.mass)),
                       A.PagedAttendProblem(q, pre, i32([0, 3]), lse=True)))
    works = [(s.new_workspace(), a.new_workspace()) for _, _, _, s, a in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for (_, _, _, s, a), (ws, wa) in zip(layers, works):
            A.aircache_shared_decode(s, ws)
            A.aircache_paged_attend(a, wa)
    torch.cuda.synchronize()
    for own, pre, q, s, a in layers:
        verify_shared(s, q, P.host(own), P.host(pre), [0, 2])
        verify_attend(a.out, a.lse, q, [0, 3], P.host(pre))
