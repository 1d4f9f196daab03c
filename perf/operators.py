"""Workloads of the paged-cache operators: the per-head norm, rotation and
append (``rotate``), one decode step over paged rows with the rows' accumulated
attention mass (``decode``), and the eviction by that mass (``evict``).

``run`` computes a pass in elementary torch operations where ``own`` is false
and through the framework's entry points where it is true.  Sequence lengths
come from the case itself (``lens_seed``), values from the seed of
``prepare``.  Page 0 of every cache is spare: padding entries of the block
table point there, as a serving engine's do.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # eight sequences decoding: one new token each, the smallest call
        dict(name="rotate_step", op="rotate", S=8, lo=1, hi=1, lens_seed=1, h_q=28, h_kv=4, d=128, rot=128,
             page=16, norm=True, inter=False, axes=1, k_out=False, past=2048, fused=False, base=1e6),
        # ragged image prompts (a batch of the ragged compression workload's lengths), three position axes,
        # the rotated keys also dense for the compression
        dict(name="rotate_prompts", op="rotate", S=5, lo=608, hi=10024, lens_seed=2, h_q=28, h_kv=4, d=128, rot=128,
             page=64, norm=True, inter=False, axes=3, k_out=True, past=0, fused=False, base=1e6),
        # far positions, partly rotated interleaved heads without a norm, as many KV heads as query heads
        dict(name="rotate_far_mha64", op="rotate", S=3, lo=211, hi=1501, lens_seed=3, h_q=32, h_kv=32, d=64, rot=32,
             page=32, norm=False, inter=True, axes=1, k_out=False, past=130000, fused=True, base=1e4),
        # one short chat
        dict(name="decode_short", op="decode", S=1, lo=701, hi=701, lens_seed=4, h_q=28, h_kv=4, d=128, page=16,
             int8=False, mass=False, fused=False),
        # a full batch of 16k prompts, mass accumulated for a later eviction
        dict(name="decode_16x16k_mass", op="decode", S=16, lo=16384, hi=16384, lens_seed=5, h_q=28, h_kv=4, d=128,
             page=64, int8=False, mass=True, fused=False),
        # many conversations of very different length, one still empty
        dict(name="decode_ragged_mass", op="decode", S=48, lo=0, hi=9000, lens_seed=6, h_q=28, h_kv=4, d=128,
             page=16, int8=False, mass=True, fused=True),
        # int8 rows of 32k prompts
        dict(name="decode_8x32k_int8", op="decode", S=8, lo=32700, hi=32768, lens_seed=7, h_q=28, h_kv=4, d=128,
             page=32, int8=True, mass=False, fused=False),
        # as many KV heads as query heads, 64-wide heads
        dict(name="decode_mha64", op="decode", S=32, lo=901, hi=2880, lens_seed=8, h_q=32, h_kv=32, d=64, page=32,
             int8=False, mass=False, fused=False),
        # one sequence a page over its budget
        dict(name="evict_step", op="evict", S=1, lo=1088, hi=1088, lens_seed=9, h_kv=4, d=128, page=64, int8=False,
             ratio=0.94, sink=4, recent=64, fused=False),
        # a batch of 16k prompts cut to half
        dict(name="evict_16x16k", op="evict", S=16, lo=16384, hi=16384, lens_seed=10, h_kv=4, d=128, page=64,
             int8=False, ratio=0.5, sink=4, recent=128, fused=False),
        # ragged int8 sequences cut to a quarter, some of them short
        dict(name="evict_ragged_int8", op="evict", S=24, lo=17, hi=9000, lens_seed=11, h_kv=8, d=128, page=16,
             int8=True, ratio=0.25, sink=0, recent=16, fused=False),
        # two long video caches cut to an eighth
        dict(name="evict_2x128k", op="evict", S=2, lo=130500, hi=131072, lens_seed=12, h_kv=4, d=128, page=256,
             int8=False, ratio=0.125, sink=4, recent=1024, fused=False),
    ]


HEADS = [(28, 4), (32, 32), (8, 2), (16, 1), (40, 8), (12, 4), (10, 2)]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["rotate", "decode", "decode", "evict"])
    h_q, h_kv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    S = _log(rng, 1, 48)
    c = dict(op=op, S=S, lens_seed=rng.randrange(1 << 30), h_kv=h_kv, d=d, page=page, fused=rng.random() < 0.3)
    if op == "rotate":
        if rng.random() < 0.5:
            c.update(lo=1, hi=1, past=_log(rng, 1, 30000))
        else:
            hi = _log(rng, 3, max(4, min(9000, 28000 * 36 * 128 // (S * (h_q + 2 * h_kv) * d))))
            c.update(lo=1, hi=hi, past=rng.choice([0, 0, _log(rng, 1, 1000), 200000]))
        rot = rng.choice([d, d, d // 2])
        c.update(h_q=h_q, rot=rot, norm=rng.random() < 0.6, inter=rng.random() < 0.4,
                 axes=rng.choice([1, 3]), k_out=rng.random() < 0.5, base=rng.choice([1e4, 1e6]))
        return c
    most = 16 * 16384 * 4 * 128 // (S * h_kv * d)
    if op == "decode":
        hi = _log(rng, 2, max(3, min(131072, most)))
        c.update(h_q=h_q, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, int8=rng.random() < 0.35,
                 mass=rng.random() < 0.5)
        return c
    hi = _log(rng, 20, max(21, min(131072, most // 2)))
    c.update(lo=rng.choice([1, hi // 2, hi]), hi=hi, int8=rng.random() < 0.35,
             ratio=rng.choice([0.02, 0.25, 0.5, 0.9]), sink=rng.choice([0, 4]), recent=rng.choice([0, 1, 16, 64]))
    return c


def _lens(c):
    r = random.Random(c["lens_seed"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["S"])]


def _keeps(c):
    """Rows to keep of each sequence: a share of it, and what is protected at least."""
    return [max(int(n * c["ratio"]), c["sink"] + c["recent"], 1) for n in _lens(c)]


# ------------------------------------------------------------------ inputs

def _cache(c, lens, gen, rows_of=None):
    """The pages of sequences of up to `lens` rows, shuffled as a long-running engine's are."""
    S, page, h, d = c["S"], c["page"], c["h_kv"], c["d"]
    need = [max(1, -(-n // page)) for n in lens]
    total, width = sum(need) + 1, max(need)
    perm = (torch.randperm(total - 1, generator=gen, device=DEV) + 1).to(torch.int32)
    table = torch.zeros((S, width), dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    kv = torch.randn((total, 2, page, h, d), generator=gen, device=DEV, dtype=torch.float32 if c.get("int8") else torch.bfloat16)
    st = dict(table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), k_scale=None, v_scale=None)
    if c.get("int8"):
        top = kv.abs().amax(-1, keepdim=True)
        codes = torch.round(kv * (127.0 / top)).to(torch.int8)
        sc = (top[..., 0] / 127.0 * torch.exp(0.3 * torch.randn(top.shape[:-1], generator=gen, device=DEV)))
        sc = sc.transpose(2, 3).contiguous()  # [P, 2, H, page]
        st["k_scale"], st["v_scale"] = sc[:, 0].contiguous(), sc[:, 1].contiguous()
        kv = codes
    if c["fused"]:
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
    else:
        st["k"], st["v"] = kv[:, 0].contiguous(), kv[:, 1].contiguous()
    return st


def _spread(st, dense):
    """dense [S, H, R] by row -> paged [P, H, page]; slots without a row hold 0."""
    S, h, R = dense.shape
    P, page = st["k"].shape[0], st["k"].shape[1]
    valid = torch.arange(R, device=DEV)[None] < st["lens"][:, None]
    slot = st["table"].long().repeat_interleave(page, 1)[:, :R], (torch.arange(R, device=DEV) % page).expand(S, R)
    out = torch.zeros((P, page, h), dtype=dense.dtype, device=DEV)
    out[slot[0][valid], slot[1][valid]] = dense.transpose(1, 2)[valid]
    return out.transpose(1, 2).contiguous()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    lens = _lens(c)
    d, h = c["d"], c["h_kv"]
    if c["op"] == "rotate":
        T, h_q = sum(lens), c["h_q"]
        cache = [c["past"] if c["past"] <= 4096 else 64] * c["S"]  # rows before the call (far positions: most were evicted)
        rows = [a + n for a, n in zip(cache, lens)]
        st = _cache(c, rows, gen)
        qkv = torch.randn((T, (h_q + 2 * h) * d), generator=gen, device=DEV, dtype=torch.bfloat16)
        st["q"] = qkv[:, :h_q * d].view(T, h_q, d)
        st["kx"] = qkv[:, h_q * d:(h_q + h) * d].view(T, h, d)
        st["vx"] = qkv[:, (h_q + h) * d:].view(T, h, d)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        st["seen"] = torch.tensor([c["past"] + n for n in lens], dtype=torch.int32, device=DEV)
        st["inv_freq"] = c["base"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
        n_f = c["rot"] // 2
        st["sections"], st["positions"] = None, None
        if c["axes"] == 3:  # time, row and column of an image's tokens
            a = n_f // 4
            st["sections"] = (a, (n_f - a) // 2, n_f - a - (n_f - a) // 2)
            st["positions"] = torch.randint(0, c["past"] + max(lens), (3, T), generator=gen, device=DEV, dtype=torch.int32)
        st["q_w"] = st["k_w"] = None
        if c["norm"]:
            st["q_w"], st["k_w"] = (1 + 0.2 * torch.randn((2, d), generator=gen, device=DEV)).to(torch.bfloat16).unbind(0)
        st["q_out"] = torch.zeros((T, h_q, d), dtype=torch.bfloat16, device=DEV)
        st["k_out"] = torch.zeros((T, h, d), dtype=torch.bfloat16, device=DEV) if c["k_out"] else None
        st["mass"] = torch.rand((st["k"].shape[0], h, c["page"]), generator=gen, device=DEV)
        st["order"] = torch.zeros((st["k"].shape[0], h, c["page"]), dtype=torch.int32, device=DEV)
        st["case"] = c
        return st
    st = _cache(c, lens, gen)
    R = st["table"].shape[1] * c["page"]
    if c["op"] == "decode":
        # queries of about the norm that makes a few hundred rows carry most of the weight
        st["q"] = (1.5 * torch.randn((c["S"], c["h_q"], d), generator=gen, device=DEV)).to(torch.bfloat16)
        st["mass"] = st["mass_out"] = None
        if c["mass"]:
            st["mass"] = _spread(st, torch.rand((c["S"], h, R), generator=gen, device=DEV))
            st["mass_out"] = torch.zeros_like(st["mass"])
        st["out"] = torch.zeros((c["S"], c["h_q"], d), dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.zeros((c["S"], c["h_q"]), dtype=torch.float32, device=DEV)
    else:
        keep = _keeps(c)
        st["keep"] = torch.tensor(keep, dtype=torch.int32, device=DEV)
        seen = [n + n // 2 for n in lens]  # a third of what was appended is gone already
        st["seen"] = torch.tensor(seen, dtype=torch.int32, device=DEV)
        r = torch.arange(R, device=DEV)
        valid = r[None] < st["lens"][:, None]
        asc = (r[None] * st["seen"][:, None] // st["lens"][:, None].clamp(min=1)).to(torch.int32)
        # earlier evictions moved rows into each other's places: all but the newest half are out of order
        key = torch.rand((c["S"], h, R), generator=gen, device=DEV) + (r[None, None] >= st["lens"][:, None, None] // 2) * 2.0
        key = torch.where(valid[:, None], torch.where(key >= 2.0, 2.0 + r / (2.0 * R), key), 4.0)
        order = asc[:, None].expand(-1, h, -1).gather(2, key.argsort(dim=2, stable=True))
        st["order"] = _spread(st, order.contiguous())
        st["mass"] = _spread(st, torch.exp(1.5 * torch.randn((c["S"], h, R), generator=gen, device=DEV)) * 1e-2)
        st["mass_out"] = torch.zeros_like(st["mass"])
        st["order_out"] = torch.zeros_like(st["order"])
        st["lens_out"] = torch.zeros_like(st["lens"])
    st["case"] = c
    return st


# ------------------------------------------------------------------ plain forms

def _rows(st):
    """Page and row of every (sequence, row) of the table's capacity, and which of them hold a row."""
    page = st["k"].shape[1]
    R = st["table"].shape[1] * page
    r = torch.arange(R, device=DEV)
    pg = st["table"].long()[:, r // page]
    return pg, (r % page).expand_as(pg), r[None] < st["lens"][:, None]


def _turned(x, w, cos, sin, c):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    R = c["rot"]
    if c["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., R:]), -1).to(torch.bfloat16)


def _plain_rotate(st):
    c = st["case"]
    T, page = st["q"].shape[0], c["page"]
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    s = torch.searchsorted(st["cu"], t, right=True) - 1
    back = st["cu"][s + 1] - t  # the token's place from its sequence's end
    order = st["seen"][s] - back
    if st["positions"] is None:
        pos = order[:, None].double()
    else:
        axis = torch.repeat_interleave(torch.arange(3, device=DEV), torch.tensor(st["sections"], device=DEV), output_size=c["rot"] // 2)
        pos = st["positions"].double()[axis].T
    ang = pos * st["inv_freq"]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    st["q_out"].copy_(_turned(st["q"], st["q_w"], cos, sin, c))
    k = _turned(st["kx"], st["k_w"], cos, sin, c)
    if st["k_out"] is not None:
        st["k_out"].copy_(k)
    row = (st["lens"][s] - back).long()
    pg = st["table"].long()[s, row // page]
    row = row % page
    st["k"][pg, row] = k
    st["v"][pg, row] = st["vx"]
    st["mass"][pg, :, row] = 0.0
    st["order"][pg, :, row] = order[:, None]


def _plain_decode(st):
    c = st["case"]
    S, h_q, d = st["q"].shape
    h = c["h_kv"]
    pg, row, valid = _rows(st)
    k, v = st["k"][pg, row].float(), st["v"][pg, row].float()  # [S, R, H, D]
    if c["int8"]:
        k = k * st["k_scale"][pg, :, row][..., None]
        v = v * st["v_scale"][pg, :, row][..., None]
    x = torch.matmul(st["q"].float().view(S, h, h_q // h, d), k.permute(0, 2, 3, 1)) * d ** -0.5
    x = x.masked_fill(~valid[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)  # a sequence without rows keeps weights of 0
    w = (x - top).exp()
    total = w.sum(-1, keepdim=True)
    st["lse"].copy_((top + total.log()).view(S, h_q))  # -inf without rows
    w = w / total.clamp(min=1e-30)
    st["out"].copy_(torch.matmul(w, v.permute(0, 2, 1, 3)).reshape(S, h_q, d))
    if c["mass"]:
        add = w.sum(2).transpose(1, 2)  # [S, R, H]
        new = st["mass"][pg, :, row] + add
        st["mass_out"][pg, :, row] = torch.where(valid[..., None], new, 0.0)


def _plain_evict(st):
    pg, row, valid = _rows(st)  # [S, R]
    S, R = pg.shape
    c = st["case"]
    mass, order = st["mass"][pg, :, row].transpose(1, 2), st["order"][pg, :, row].transpose(1, 2)  # [S, H, R]
    safe = (order < c["sink"]) | (order >= (st["seen"] - c["recent"])[:, None, None])
    key = torch.where(torch.isnan(mass), float("-inf"), mass)
    key = torch.where(safe, float("inf"), key).masked_fill(~valid[:, None], float("-inf"))
    # ranks by key, ties to the lower row; slots behind the last row rank after all rows
    by = key.argsort(dim=-1, descending=True, stable=True)
    rank = torch.empty_like(by).scatter_(-1, by, torch.arange(R, device=DEV).expand_as(by))
    new = torch.minimum(st["lens"], st["keep"])
    kept = valid[:, None] & (rank < new[:, None, None])
    r = torch.arange(R, device=DEV)
    hole = ~kept & (r < new[:, None, None])
    mover = kept & (r >= new[:, None, None])
    # the j-th hole takes the j-th mover; the list's unused end reads and writes the spare page
    nth_hole = torch.where(hole, hole.cumsum(-1) - 1, R)
    nth_mover = torch.where(mover, mover.cumsum(-1) - 1, R)
    lists = torch.full((2, S, c["h_kv"], R + 1), -1, dtype=torch.long, device=DEV)
    at = r.expand_as(hole)
    lists[0].scatter_(-1, nth_hole, at)
    lists[1].scatter_(-1, nth_mover, at)
    n_moves = hole.sum(-1, keepdim=True)
    real = r < n_moves  # [S, H, R]
    dst, src = lists[0, ..., :R].clamp(min=0), lists[1, ..., :R].clamp(min=0)
    seq = torch.arange(S, device=DEV)[:, None, None].expand_as(dst)
    head = torch.arange(c["h_kv"], device=DEV)[None, :, None].expand_as(dst)
    dp, dr = torch.where(real, pg[seq, dst], 0), torch.where(real, row[seq, dst], 0)
    sp, sr = torch.where(real, pg[seq, src], 0), torch.where(real, row[seq, src], 0)
    for name in ("k", "v"):
        st[name][dp, dr, head] = st[name][sp, sr, head]
    if c["int8"]:
        for name in ("k_scale", "v_scale"):
            st[name][dp, head, dr] = st[name][sp, head, sr]
    for name, x in (("mass", mass), ("order", order)):
        out = st[name + "_out"]
        stay = kept & (r < new[:, None, None])
        out[torch.where(stay, pg[:, None], 0), torch.arange(c["h_kv"], device=DEV)[None, :, None],
            torch.where(stay, row[:, None], 0)] = torch.where(stay, x, 0)
        out[dp, head, dr] = torch.where(real, st[name][sp, head, sr], 0)
    st["lens_out"].copy_(new)


# ------------------------------------------------------------------ a pass

def _plan(st):
    """The problem description and the workspace, kept with the state as a serving program keeps them per layer."""
    from lvlm_kv_cache_gb300 import aircache as A

    c = st["case"]
    cache = A.PagedCache(st["k"], st["v"], st["table"], st["lens"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                         mass=st.get("mass"), order=st.get("order"))
    if c["op"] == "rotate":
        prob = A.RotateProblem(st["q"], st["kx"], st["vx"], q_out=st["q_out"], k_out=st["k_out"], cache=cache,
                               cu_tokens=st["cu"], seen=st["seen"], positions=st["positions"],
                               sections=st["sections"], turns=A.rotation_table(st["inv_freq"]),
                               q_weight=st["q_w"], k_weight=st["k_w"], eps=1e-6, interleaved=c["inter"])
        return A.aircache_rotate, prob, torch.zeros(1, dtype=torch.int32, device=DEV)
    if c["op"] == "decode":
        prob = A.PagedDecodeProblem(st["q"], cache, out=st["out"], lse=st["lse"], mass_out=st["mass_out"])
        return A.aircache_paged_decode, prob, prob.new_workspace()
    prob = A.EvictProblem(cache, st["keep"], st["lens_out"], seen=st["seen"], sink=c["sink"], recent=c["recent"],
                          mass_out=st["mass_out"], order_out=st["order_out"])
    return A.aircache_evict, prob, prob.new_workspace()


def run(state):
    c = state["case"]
    if own:
        if "plan" not in state:
            state["plan"] = _plan(state)
        call, prob, ws = state["plan"]
        call(prob, ws)
    else:
        {"rotate": _plain_rotate, "decode": _plain_decode, "evict": _plain_evict}[c["op"]](state)
    if c["op"] == "rotate":
        return {n: state[n] for n in ("q_out", "k_out", "k", "v", "mass", "order")}
    if c["op"] == "decode":
        return {n: state[n] for n in ("out", "lse", "mass_out")}
    return {n: state[n] for n in ("k", "v", "k_scale", "v_scale", "mass_out", "order_out", "lens_out")}


def work(case):
    c = case
    lens = _lens(c)
    d, h = c["d"], c["h_kv"]
    if c["op"] == "rotate":
        T, h_q = sum(lens), c["h_q"]
        b = T * d * 2 * (2 * h_q + 4 * h + (h if c["k_out"] else 0)) + T * h * 8
        return {"bytes": b + T * 4 * (3 if c["axes"] == 3 else 0),
                "flops": T * (h_q + h) * (3 * c["rot"] + (4 * d if c["norm"] else 0))}
    if c["op"] == "decode":
        row = 2 * d * (1 if c["int8"] else 2) + (8 if c["int8"] else 0) + (8 if c["mass"] else 0)
        return {"bytes": sum(lens) * h * row + c["S"] * c["h_q"] * (d * 4 + 4), "flops": 4 * sum(lens) * c["h_q"] * d}
    b = 0
    for n, keep in zip(lens, _keeps(c)):
        keep = min(n, keep)
        # rows to move where the mass does not go by the row's place, the newest rows aside
        moves = (n - keep) * keep / n
        b += h * (n * 8 + keep * 8 + moves * 2 * (2 * d * (1 if c["int8"] else 2) + (8 if c["int8"] else 0)))
    return {"bytes": b, "flops": sum(lens) * h * 4}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in 64 bits, one sequence (and token or head) after the other."""
    st = prepare(case, seed)
    c = st["case"]
    page, h = c["page"], c["h_kv"]
    lens, table = _lens(c), st["table"].long()
    if c["op"] == "rotate":
        out = {n: st[n].double() for n in ("k", "v")}
        out.update(mass=st["mass"].double(), order=st["order"].double(), q_out=st["q_out"].double(),
                   k_out=None if st["k_out"] is None else st["k_out"].double())
        n_f, at = c["rot"] // 2, 0
        i = torch.arange(n_f, device=DEV)
        ia, ib = (2 * i, 2 * i + 1) if c["inter"] else (i, i + n_f)
        for s, n in enumerate(lens):
            tok = slice(at, at + n)
            p = torch.arange(c["past"], c["past"] + n, device=DEV).double()[:, None].expand(n, n_f)
            if st["positions"] is not None:
                p = torch.cat([st["positions"][a, tok].double()[:, None].expand(n, m) for a, m in enumerate(st["sections"])], 1)
            turn = torch.polar(torch.ones_like(p), p * st["inv_freq"])[:, None]
            ys = []
            for x, w in ((st["q"][tok].double(), st["q_w"]), (st["kx"][tok].double(), st["k_w"])):
                if w is not None:
                    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
                y = x.clone()
                z = torch.complex(x[..., ia], x[..., ib]) * turn
                y[..., ia], y[..., ib] = z.real, z.imag
                ys.append(y)
            out["q_out"][tok] = ys[0]
            if out["k_out"] is not None:
                out["k_out"][tok] = ys[1]
            first = int(st["lens"][s]) - n
            rows = torch.arange(first, first + n, device=DEV)
            pg, rr = table[s, rows // page], rows % page
            out["k"][pg, rr], out["v"][pg, rr] = ys[1], st["vx"][tok].double()
            out["mass"][pg, :, rr] = 0.0
            out["order"][pg, :, rr] = torch.arange(c["past"], c["past"] + n, device=DEV).double()[:, None]
            at += n
        out["order"] = out["order"].to(torch.int32)
        return out
    if c["op"] == "decode":
        o = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
        m_out = None if st["mass"] is None else torch.zeros(st["mass"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
        g = c["h_q"] // h
        for s, n in enumerate(lens):
            rows = torch.arange(n, device=DEV)
            pg, rr = table[s, rows // page], rows % page
            for j in range(h if n else 0):
                k, v = st["k"][pg, rr, j].double(), st["v"][pg, rr, j].double()
                if c["int8"]:
                    k, v = k * st["k_scale"][pg, j, rr].double()[:, None], v * st["v_scale"][pg, j, rr].double()[:, None]
                x = st["q"][s, j * g:(j + 1) * g].double() @ k.T / math.sqrt(c["d"])
                lse[s, j * g:(j + 1) * g] = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
                o[s, j * g:(j + 1) * g] = w @ v
                if m_out is not None:
                    m_out[pg, j, rr] = st["mass"][pg, j, rr].double() + w.sum(0)
        return {"out": o, "lse": lse, "mass_out": m_out}
    out = {n: st[n].clone() for n in ("k", "v")}
    out.update({n: None if st[n] is None else st[n].clone() for n in ("k_scale", "v_scale")})
    out.update({n + "_out": torch.zeros_like(st[n]) for n in ("mass", "order")})
    new = []
    for s, (n, keep) in enumerate(zip(lens, _keeps(c))):
        keep = min(n, keep)
        new.append(keep)
        rows = torch.arange(n, device=DEV)
        pg, rr = table[s, rows // page], rows % page
        for j in range(h):
            m, age = st["mass"][pg, j, rr].double(), st["order"][pg, j, rr]
            safe = (age < c["sink"]) | (age >= int(st["seen"][s]) - c["recent"])
            rank = torch.argsort(torch.where(safe, -math.inf, -m), stable=True)  # best first, the lower row first among equals
            stay = torch.sort(rank[:keep]).values
            gone = torch.ones(n, dtype=torch.bool, device=DEV)
            gone[stay] = False
            frm = torch.arange(keep, device=DEV)
            frm[gone[:keep]] = stay[stay >= keep]
            for name in ("k", "v"):
                out[name][pg[:keep], rr[:keep], j] = st[name][pg[frm], rr[frm], j]
            if c["int8"]:
                for name in ("k_scale", "v_scale"):
                    out[name][pg[:keep], j, rr[:keep]] = st[name][pg[frm], j, rr[frm]]
            for name in ("mass", "order"):
                out[name + "_out"][pg[:keep], j, rr[:keep]] = st[name][pg[frm], j, rr[frm]]
    out["lens_out"] = torch.tensor(new, dtype=torch.int32, device=DEV)
    return {n: x.double() if x is not None and x.dtype in (torch.bfloat16, torch.float32) else x for n, x in out.items()}
