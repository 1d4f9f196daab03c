"""One workspace for every call of a step: attention of several tokens, the decode step, the shared decode step and the
eviction leave it ready for one another, eagerly and in two graphs replayed in turn; results are those of workspaces of
their own, bit for bit."""
import numpy as np
import pytest
import torch

import paged_utils as P
from test_gpu_paged_attend import A, i32, queries  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
def test_one_workspace_for_every_call(A, int8):  # noqa: F811
    lens, new = [5000, 40, 700, 0, 129], [30, 1, 200, 0, 129]
    cache = P.build(A, lens, 2, 128, 16, seed=60, int8=int8)
    pre = P.build(A, [3000, 90], 2, 128, 64, seed=61, int8=int8, mass=False, order=False)
    q, q1 = queries(sum(new), 14, 128, 60), queries(5, 14, 128, 61)
    cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    begin = (torch.arange(sum(new), device="cuda", dtype=torch.int32) * 7) % 50
    mass, joint = torch.zeros_like(cache.mass), torch.zeros_like(cache.mass)
    kept = P.build(A, lens, 2, 128, 16, seed=60, int8=int8)  # (the eviction's: it moves rows)
    start = {n: getattr(kept, n).clone() for n in ("k", "v", "mass", "order", "k_scale", "v_scale") if getattr(kept, n) is not None}
    calls = [
        (A.aircache_paged_attend, A.PagedAttendProblem(q, cache, cu, lse=True, causal=True, row_begin=begin)),
        (A.aircache_paged_decode, A.PagedDecodeProblem(q1, cache, lse=True, mass_out=mass)),
        (A.aircache_shared_decode, A.SharedDecodeProblem(q1, cache, pre, i32([0, 2, 4]), lse=True, mass_out=joint)),
        (A.aircache_evict, A.EvictProblem(kept, i32([600, 40, 100, 0, 128]), lens_out=torch.zeros_like(kept.lens))),
        (A.aircache_paged_attend, A.PagedAttendProblem(q1, cache, i32([0, 1, 2, 3, 4, 5]), lse=True)),
    ]

    def reset():
        for n, t in start.items():
            getattr(kept, n).copy_(t)
        for _, p in calls:
            for n in ("out", "lse"):
                if getattr(p, n, None) is not None:
                    getattr(p, n).zero_()
        mass.zero_()
        joint.zero_()

    def results():
        torch.cuda.synchronize()
        got = [P.bits(t) for _, p in calls for t in (getattr(p, "out", None), getattr(p, "lse", None)) if t is not None]
        return got + [P.bits(mass), P.bits(joint), P.bits(calls[3][1].lens_out)] + list(P.state(kept).values())

    reset()
    for call, p in calls:
        call(p, p.new_workspace())
    want = results()
    ws = torch.zeros(max(p.workspace_size() for _, p in calls), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for order in ((0, 1, 2, 3, 4), (4, 3, 2, 1, 0)):
        with torch.cuda.stream(s):
            reset()
            for i in order:
                calls[i][0](calls[i][1], ws)
        assert all(np.array_equal(a, b) for a, b in zip(want, results()))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(s), torch.cuda.graph(graphs[-1], stream=s):
            for i in order:
                calls[i][0](calls[i][1], ws)
    for g in graphs + graphs[::-1]:
        reset()
        torch.cuda.synchronize()
        g.replay()
        assert all(np.array_equal(a, b) for a, b in zip(want, results()))
    assert A.aircache_get_error(ws) == A.OK
