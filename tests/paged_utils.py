"""Seeded paged caches for the tests, on any device, and their host copies."""
import numpy as np
import torch


def build(A, lens, h_kv, d, page_rows, seed=0, int8=False, mass=True, order=True, device="cuda", spare=3, wide=0,
          fused=False, fill=None, max_pages=None):
    """A PagedCache with shuffled pages.  wide: extra unused heads in each row (strides); fused: K and V in one
    buffer; fill: the value of every slot that holds no row."""
    g = torch.Generator().manual_seed(seed)
    S = len(lens)
    need = [-(-n // page_rows) for n in lens]
    P = sum(need) + spare
    width = max(need + [1]) if max_pages is None else max_pages
    perm = torch.randperm(P, generator=g).tolist()
    table = torch.full((S, width), -7, dtype=torch.int32)  # entries that no row needs are never read
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = torch.tensor(perm[at:at + m], dtype=torch.int32)
        at += m
    kv = torch.randn((P, 2, page_rows, h_kv + wide, d), generator=g)
    used = torch.zeros((P, page_rows), dtype=torch.bool)
    for s, n in enumerate(lens):
        for i in range(0, n, page_rows):
            used[table[s, i // page_rows], :min(page_rows, n - i)] = True
    ks = vs = None
    if int8:
        kv = torch.randint(-127, 128, kv.shape, generator=g).to(torch.int8)
        sc = torch.exp(torch.randn((P, 2, h_kv, page_rows), generator=g)) / 100
        if fill is not None:
            sc = torch.where(used[:, None, None], sc, torch.full_like(sc, fill))
        ks, vs = sc[:, 0].contiguous().to(device), sc[:, 1].contiguous().to(device)
    else:
        kv = kv.to(torch.bfloat16)
        if fill is not None:
            kv[~used[:, None].expand(-1, 2, -1)] = fill
    kv = kv.to(device)
    k, v = kv[:, 0, :, :h_kv], kv[:, 1, :, :h_kv]
    if not fused:
        kk, vv = kv[:, 0].contiguous(), kv[:, 1].contiguous()
        k, v = kk[:, :, :h_kv], vv[:, :, :h_kv]
    m = torch.rand((P, h_kv, page_rows), generator=g).to(device) if mass else None
    o = None
    if order:
        o = torch.zeros((P, h_kv, page_rows), dtype=torch.int32)
        for s, n in enumerate(lens):
            for h in range(h_kv):
                r = torch.randperm(n, generator=g).to(torch.int32)
                i = torch.arange(n)
                o[table[s, i // page_rows].long(), h, i % page_rows] = r
        o = o.to(device)
    return A.PagedCache(k, v, table.to(device), torch.tensor(lens, dtype=torch.int32, device=device), k_scale=ks,
                        v_scale=vs, mass=m, order=o)


def host(cache):
    """The cache as oracle.paged takes it (copies)."""
    n = lambda t: None if t is None else t.detach().cpu().numpy().copy()  # noqa: E731
    f = (lambda t: n(t)) if cache.k.dtype == torch.int8 else (lambda t: n(t.double()))
    return dict(k=f(cache.k), v=f(cache.v), k_scale=n(cache.k_scale), v_scale=n(cache.v_scale), mass=n(cache.mass),
                order=n(cache.order), table=n(cache.table), lens=n(cache.lens))


def bits(t):
    """A tensor's raw bits on the host, for exact comparisons (NaN equal to itself)."""
    t = t.detach().cpu().contiguous()
    return t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()]).numpy()


def state(cache):
    return {n: bits(getattr(cache, n)) for n in ("k", "v", "k_scale", "v_scale", "mass", "order")
            if getattr(cache, n) is not None}


def assert_same_state(a, b, but=()):
    for n in a:
        if n not in but:
            assert np.array_equal(a[n], b[n]), n
