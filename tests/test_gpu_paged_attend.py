"""aircache_paged_attend against its definition in 64 bits (oracle/paged.py).

Tolerances.  A dot product in fp32 over D exact products is off by at most
D 2^-24 sum |q_d k_d| scale =: dx (at the row where that is largest), and a
weight by a relative 2 dx + 2^-18 (two exponentials of that error, the base-2
exponential's own 2^-22, products and sums of up to some thousand terms).  lse: dx + 2^-20 (1 + |lse|).
out: each weight is rounded to bf16 before it meets V, int8 rows' with the value's scale
(2^-8 of it), and out is rounded to bf16:
(2^-8 + 2 dx + 2^-18) sum w |v| + 2^-8 |out|."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(T, h_q, d, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((T, h_q, d), generator=g, device="cuda")).to(torch.bfloat16)


def verify(out, lse, q, cu, c, scale=None, causal=False, begin=None, end=None):
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    want, want_lse, size, spread = O.attend(q.double().cpu().numpy(), cu, c, scale, causal, begin, end)
    T = int(cu[-1])
    want, want_lse, size, spread = want[:T], want_lse[:T], size[:T], spread[:T]
    dx = d * 2.0 ** -24 * size
    got = out.double().cpu().numpy()[:T]
    tol = (HALF + 2 * dx[..., None] + 2.0 ** -18) * spread + HALF * np.abs(want) + 1e-30
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= tol), f"out: worst {np.max(err / tol):.2f} at {np.unravel_index(np.argmax(err / tol), err.shape)}"
    if lse is not None:
        gl = lse.double().cpu().numpy()[:T]
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(gl))
        e = np.abs(gl[~empty] - want_lse[~empty])
        t = dx[~empty] + 2.0 ** -20 * (1 + np.abs(want_lse[~empty]))
        assert np.all(e <= t), f"lse: worst {np.max(e / t):.2f}"


def case(A, new, lens, h_q, h_kv, d, page_rows, seed=0, causal=False, begin=None, end=None, q_scale=1.5, q=None,
         scale=None, pad=2, **kw):
    """lens: rows of each cache, the new tokens' own among them (causal)."""
    cache = P.build(A, lens, h_kv, d, page_rows, seed=seed, mass=False, order=False, **kw)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + pad  # tokens behind the last sequence
    q = queries(T, h_q, d, seed, q_scale) if q is None else q
    out = torch.full((T, h_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, h_q), 7.0, device="cuda")
    fit = lambda x: None if x is None else i32(list(x) + [0] * (T - len(x)))  # noqa: E731
    before = P.state(cache)
    prob = A.PagedAttendProblem(q, cache, i32(cu.tolist()), out=out, lse=lse, causal=causal, scale=scale,
                                row_begin=fit(begin), row_end=fit(end))
    A.paged_attend(prob)
    verify(out, lse, q, cu, P.host(cache), scale, causal, begin, end)
    assert torch.all(out[cu[-1]:] == 7.0) and torch.all(lse[cu[-1]:] == 7.0)
    P.assert_same_state(before, P.state(cache))
    return prob, cache, q


NEW = [1, 2, 0, 17, 18, 19, 36, 37, 5, 73]
OLD = [0, 126, 40, 111, 0, 128, 300, 91, 1000, 55]


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("page_rows", [16, 48, 64, 256])
def test_ragged(A, page_rows, causal, d):
    lens = [a + b for a, b in zip(NEW, OLD)]
    case(A, NEW, lens, 28, 4, d, page_rows, seed=d + page_rows, causal=causal)
