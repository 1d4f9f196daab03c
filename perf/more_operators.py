"""Workloads of attention with several query tokens over the paged cache:
new tokens that continue a cached sequence (``extend``), text tokens over an
encoder's states (``cross``), and one decode step of a batch whose sequences
share prefixes (``shared``).

``run`` computes a pass in elementary torch operations where ``own`` is false
and through the framework's entry points where it is true.  Lengths come from
the case itself (``lens_seed``), values from the seed of ``prepare``.  Page 0
of every cache is spare: padding entries of the block table point there, as a
serving engine's do.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # four drafted tokens of each of eight chats are checked at once: the smallest call
        dict(name="extend_drafts", op="extend", S=8, lo=4, hi=4, past_lo=300, past_hi=2100, lens_seed=1, h_q=28, h_kv=4,
             d=128, page=16, int8=False, fused=False, lse=False),
        # questions behind compressed or full image prompts (the ragged compression workload's lengths)
        dict(name="extend_questions", op="extend", S=16, lo=32, hi=1024, past_lo=576, past_hi=9000, lens_seed=2, h_q=28,
             h_kv=4, d=128, page=64, int8=False, fused=True, lse=False),
        # a chunk of a prompt behind a very long cached video
        dict(name="extend_long_video", op="extend", S=1, lo=1000, hi=1000, past_lo=130000, past_hi=130000, lens_seed=3,
             h_q=28, h_kv=4, d=128, page=256, int8=False, fused=False, lse=False),
        # int8 rows, 64-wide heads, as many KV heads as query heads, one sequence without a past
        dict(name="extend_mha64_int8", op="extend", S=6, lo=17, hi=300, past_lo=0, past_hi=2880, lens_seed=4, h_q=32,
             h_kv=32, d=64, page=32, int8=True, fused=False, lse=True),
        # a few words about two small images; words before an image do not see it, some see none
        dict(name="cross_words", op="cross", S=4, lo=5, hi=40, rows_lo=1152, rows_hi=1152, images=2, latest=False,
             lens_seed=5, h_q=28, h_kv=4, d=128, page=16, int8=False, fused=False, lse=False),
        # questions over whole videos (64 frames of 196)
        dict(name="cross_videos", op="cross", S=4, lo=256, hi=256, rows_lo=12544, rows_hi=12544, images=0, latest=False,
             lens_seed=6, h_q=28, h_kv=4, d=128, page=64, int8=False, fused=False, lse=False),
        # long interleaved prompts, each token over its latest image only, int8 states of eight images
        dict(name="cross_interleaved_int8", op="cross", S=8, lo=32, hi=1024, rows_lo=2000, rows_hi=9000, images=8,
             latest=True, lens_seed=7, h_q=40, h_kv=8, d=128, page=32, int8=True, fused=False, lse=True),
        # as many KV heads as query heads
        dict(name="cross_mha", op="cross", S=8, lo=301, hi=512, rows_lo=2880, rows_hi=2880, images=0, latest=False,
             lens_seed=8, h_q=32, h_kv=32, d=128, page=32, int8=False, fused=False, lse=False),
        # eight answers to one prompt, just begun: the smallest
        dict(name="shared_8", op="shared", G=1, S=8, alone=0, p_lo=2048, p_hi=2048, lo=1, hi=64, lens_seed=9, h_q=28,
             h_kv=4, d=128, page=16, p_page=64, int8=False, mass=False, fused=False),
        # many chats about one long document
        dict(name="shared_64x16k", op="shared", G=1, S=64, alone=0, p_lo=16384, p_hi=16384, lo=100, hi=2000,
             lens_seed=10, h_q=28, h_kv=4, d=128, page=16, p_page=64, int8=False, mass=False, fused=True),
        # four prompts with their chats and a few chats alone, int8 rows, mass for a later eviction of the chats' own rows
        dict(name="shared_groups_int8", op="shared", G=4, S=48, alone=5, p_lo=577, p_hi=9000, lo=0, hi=1500,
             lens_seed=11, h_q=32, h_kv=8, d=128, page=32, p_page=128, int8=True, mass=True, fused=False),
        # questions about one very long video
        dict(name="shared_video", op="shared", G=1, S=24, alone=0, p_lo=131072, p_hi=131072, lo=1, hi=256, lens_seed=12,
             h_q=28, h_kv=4, d=128, page=16, p_page=256, int8=False, mass=False, fused=False),
    ]


HEADS = [(28, 4), (32, 32), (8, 2), (16, 1), (40, 8), (12, 4), (10, 2)]
MOST_WORK = 1.4e12      # operations of a drawn case
MOST_ROWS = 16 * 16384 * 4 * 128  # cached elements of K


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["extend", "cross", "shared"])
    h_q, h_kv = rng.choice(HEADS)
    c = dict(op=op, lens_seed=rng.randrange(1 << 30), h_q=h_q, h_kv=h_kv, d=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128, 256]), int8=rng.random() < 0.35, fused=rng.random() < 0.3)
    line = h_kv * c["d"]
    if op == "shared":
        c.update(G=_log(rng, 1, 6), p_page=rng.choice([16, 32, 64, 128, 256]), mass=rng.random() < 0.4)
        c["S"] = rng.randint(c["G"], max(c["G"], _log(rng, 2, 80)))
        c["alone"] = rng.choice([0, 0, min(3, c["S"] - c["G"])])
        p_hi = _log(rng, 20, max(21, min(131072, MOST_ROWS // (c["G"] * line))))
        hi = _log(rng, 2, max(3, min(8192, MOST_ROWS // (c["S"] * line))))
        c.update(p_lo=rng.choice([1, p_hi // 2, p_hi]), p_hi=p_hi, lo=rng.choice([0, 1, hi]), hi=hi)
        return c
    c.update(S=_log(rng, 1, 32), lse=rng.random() < 0.5)
    rows = _log(rng, 20, max(21, min(131072, MOST_ROWS // (c["S"] * line))))
    hi = _log(rng, 1, max(2, min(2000, MOST_WORK / (4 * c["S"] * h_q * c["d"] * rows))))
    c.update(lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi)
    if op == "extend":
        c.update(past_lo=rng.choice([0, rows // 2, rows]), past_hi=rows)
    else:
        images = rng.choice([0, 1, 2, 5])
        c.update(rows_lo=rng.choice([images + 1, rows // 2, rows]), rows_hi=rows, images=images,
                 latest=rng.random() < 0.5)
    return c


def _sizes(c):
    """New tokens of each sequence and rows of each cache; for shared: rows of each prefix, members of each prefix."""
    r = random.Random(c["lens_seed"])
    if c["op"] == "shared":
        cuts = sorted(r.sample(range(1, c["S"] - c["alone"]), c["G"] - 1)) if c["G"] > 1 else []
        cu = [0] + cuts + [c["S"] - c["alone"]]
        return [1] * c["S"], [r.randint(c["lo"], c["hi"]) for _ in range(c["S"])], \
            [r.randint(c["p_lo"], c["p_hi"]) for _ in range(c["G"])], cu
    new = [r.randint(c["lo"], c["hi"]) for _ in range(c["S"])]
    if c["op"] == "extend":
        return new, [r.randint(c["past_lo"], c["past_hi"]) + n for n in new], None, None
    return new, [r.randint(c["rows_lo"], c["rows_hi"]) for _ in new], None, None


def _ranges(c):
    """cross with images: the rows [begin, end) that each token sees.  Image i of a sequence stands before its token
    at[i]; what stands before the first sees nothing."""
    r = random.Random(c["lens_seed"] + 1)
    begin, end = [], []
    new, rows, _, _ = _sizes(c)
    for n, R in zip(new, rows):
        at = sorted(r.randint(0, n) for _ in range(c["images"]))
        at[0] = min(at[0], n - 1)  # (the last token sees one at least)
        edge = [R * i // c["images"] for i in range(c["images"] + 1)]
        for t in range(n):
            seen = sum(a <= t for a in at)
            begin.append(edge[max(seen - 1, 0)] if c["latest"] else 0)
            end.append(edge[seen])
    return begin, end


# ------------------------------------------------------------------ inputs

def _cache(c, lens, gen, page, fused):
    """The pages of sequences of `lens` rows, shuffled as a long-running engine's are."""
    h, d = c["h_kv"], c["d"]
    need = [max(1, -(-n // page)) for n in lens]
    total, width = sum(need) + 1, max(need)
    perm = (torch.randperm(total - 1, generator=gen, device=DEV) + 1).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    kv = torch.randn((total, 2, page, h, d), generator=gen, device=DEV,
                     dtype=torch.float32 if c["int8"] else torch.bfloat16)
    st = dict(table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), rows=lens, page=page, k_scale=None,
              v_scale=None, mass=None)
    if c["int8"]:
        top = kv.abs().amax(-1, keepdim=True)
        codes = torch.round(kv * (127.0 / top)).to(torch.int8)
        sc = top[..., 0] / 127.0 * torch.exp(0.3 * torch.randn(top.shape[:-1], generator=gen, device=DEV))
        sc = sc.transpose(2, 3).contiguous()  # [P, 2, H, page]
        st["k_scale"], st["v_scale"] = sc[:, 0].contiguous(), sc[:, 1].contiguous()
        kv = codes
    if fused:
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
    else:
        st["k"], st["v"] = kv[:, 0].contiguous(), kv[:, 1].contiguous()
    return st


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    new, rows, prefix, cu = _sizes(c)
    T, h_q, d = sum(new), c["h_q"], c["d"]
    st = dict(case=c, new=new, cache=_cache(c, rows, gen, c["page"], c["fused"]))
    # queries of about the norm that makes a few hundred rows carry most of the weight
    st["q"] = (1.5 * torch.randn((T, h_q, d), generator=gen, device=DEV)).to(torch.bfloat16)
    st["out"] = torch.zeros((T, h_q, d), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.zeros((T, h_q), dtype=torch.float32, device=DEV) if c["op"] == "shared" or c["lse"] else None
    if c["op"] == "shared":
        st["prefix"] = _cache(c, prefix, gen, c["p_page"], False)
        st["groups"] = cu
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        st["mass_out"] = None
        if c["mass"]:
            k = st["cache"]["k"]
            slots = (k.shape[0], c["h_kv"], c["page"])
            valid = torch.zeros((slots[0], c["page"]), dtype=torch.bool, device=DEV)
            pg, r, live = _places(st["cache"])
            valid[pg[live], r[live]] = True
            st["cache"]["mass"] = torch.rand(slots, generator=gen, device=DEV) * valid[:, None]
            st["mass_out"] = torch.zeros(slots, device=DEV)
        return st
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    st["at"], st["cu"] = at, torch.tensor(at, dtype=torch.int32, device=DEV)
    st["begin"] = st["end"] = None
    if c["op"] == "cross" and c["images"]:
        begin, end = _ranges(c)
        st["begin"] = torch.tensor(begin, dtype=torch.int32, device=DEV)
        st["end"] = torch.tensor(end, dtype=torch.int32, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _places(ca):
    """Page and row of every (sequence, row) of the table's capacity, and which of them hold a row."""
    R = ca["table"].shape[1] * ca["page"]
    r = torch.arange(R, device=DEV)
    pg = ca["table"].long()[:, r // ca["page"]]
    return pg, (r % ca["page"]).expand_as(pg), r[None] < ca["lens"][:, None]


def _rows(ca, s):
    """Sequence s's keys and values, [H, R, D] in 32 bits."""
    n = ca["rows"][s]
    r = torch.arange(n, device=DEV)
    pg, r = ca["table"][s].long()[r // ca["page"]], r % ca["page"]
    out = []
    for name in ("k", "v"):
        x = ca[name][pg, r].float()
        if ca[name + "_scale"] is not None:
            x = x * ca[name + "_scale"][pg, :, r][..., None]
        out.append(x.transpose(0, 1).contiguous())
    return out


def _weights(q, k, scale, seen=None):
    """q [H, M, D], k [H, R, D]: the unnormalised weights, their sum and their reference."""
    x = torch.matmul(q, k.transpose(1, 2)) * scale
    if seen is not None:
        x = x.masked_fill(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)  # nothing seen: weights of 0
    w = (x - top).exp_()
    return w, w.sum(-1, keepdim=True), top


def _plain_attend(st):
    c = st["case"]
    h, g, d, ca = c["h_kv"], c["h_q"] // c["h_kv"], c["d"], st["cache"]
    for s, n in enumerate(st["new"]):
        R, t0 = ca["rows"][s], st["at"][s]
        if R == 0:
            st["out"][t0:t0 + n] = 0
            if st["lse"] is not None:
                st["lse"][t0:t0 + n] = float("-inf")
            continue
        k, v = _rows(ca, s)
        some = max(1, min(n, (1 << 28) // (h * g * R)))  # tokens at a time: a gigabyte of logits
        r = torch.arange(R, device=DEV)
        for a in range(0, n, some):
            m = min(some, n - a)
            tok = slice(t0 + a, t0 + a + m)
            seen = None
            if c["op"] == "extend":
                seen = r < R - n + a + 1 + torch.arange(m, device=DEV)[:, None]
            elif st["end"] is not None:
                seen = (r >= st["begin"][tok, None]) & (r < st["end"][tok, None])
            if seen is not None:
                seen = seen.repeat_interleave(g, 0)  # a row for each query head of a KV head
            q = st["q"][tok].float().view(m, h, g, d).transpose(0, 1).reshape(h, m * g, d)
            w, total, top = _weights(q, k, d ** -0.5, seen)
            o = torch.matmul(w, v) / total.clamp(min=1e-30)
            st["out"][tok] = o.view(h, m, g, d).transpose(0, 1).reshape(m, h * g, d).to(torch.bfloat16)
            if st["lse"] is not None:
                st["lse"][tok] = (top + total.log()).view(h, m, g).transpose(0, 1).reshape(m, h * g)


def _plain_shared(st):
    c = st["case"]
    h, g, d, ca = c["h_kv"], c["h_q"] // c["h_kv"], c["d"], st["cache"]
    group = [-1] * c["S"]
    for i, (a, b) in enumerate(zip(st["groups"], st["groups"][1:])):
        group[a:b] = [i] * (b - a)
    shared = {}
    for i in range(c["G"]):  # the whole group's queries over its prefix
        a, b = st["groups"][i], st["groups"][i + 1]
        if b > a and st["prefix"]["rows"][i] > 0:
            k, v = _rows(st["prefix"], i)
            q = st["q"][a:b].float().view(b - a, h, g, d).transpose(0, 1).reshape(h, (b - a) * g, d)
            w, total, top = _weights(q, k, d ** -0.5)
            o = torch.matmul(w, v)
            shared[i] = [x.view(h, b - a, g, -1) for x in (o, total, top)]
    for s in range(c["S"]):
        part = None
        if group[s] in shared:
            part = [x[:, s - st["groups"][group[s]]] for x in shared[group[s]]]
        if ca["rows"][s] > 0:
            k, v = _rows(ca, s)
            w, total, top = _weights(st["q"][s].float().view(h, g, d), k, d ** -0.5)
            o = torch.matmul(w, v)
            if part is not None:
                new = torch.maximum(top, part[2])
                fo, fp = (top - new).exp(), (part[2] - new).exp()
                w, o, total, top = w * fo, o * fo + part[0] * fp, total * fo + part[1] * fp, new
            if c["mass"]:
                r = torch.arange(ca["rows"][s], device=DEV)
                pg, r = ca["table"][s].long()[r // ca["page"]], r % ca["page"]
                st["mass_out"][pg, :, r] = ca["mass"][pg, :, r] + (w / total).sum(1).T
        elif part is not None:
            o, total, top = part
        else:
            st["out"][s] = 0
            st["lse"][s] = float("-inf")
            continue
        st["out"][s] = (o / total).reshape(h * g, d).to(torch.bfloat16)
        st["lse"][s] = (top + total.log()).reshape(h * g)


# ------------------------------------------------------------------ a pass

def _plan(st):
    """The problem description and the workspace, kept with the state as a serving program keeps them per layer."""
    from lvlm_kv_cache_gb300 import aircache as A

    c = st["case"]
    ca = st["cache"]
    cache = A.PagedCache(ca["k"], ca["v"], ca["table"], ca["lens"], k_scale=ca["k_scale"], v_scale=ca["v_scale"],
                         mass=ca["mass"])
    if c["op"] == "shared":
        p = st["prefix"]
        prefix = A.PagedCache(p["k"], p["v"], p["table"], p["lens"], k_scale=p["k_scale"], v_scale=p["v_scale"])
        prob = A.SharedDecodeProblem(st["q"], cache, prefix, st["cu"], out=st["out"], lse=st["lse"],
                                     mass_out=st["mass_out"])
        return A.aircache_shared_decode, prob, prob.new_workspace()
    prob = A.PagedAttendProblem(st["q"], cache, st["cu"], out=st["out"], lse=st["lse"], causal=c["op"] == "extend",
                                row_begin=st["begin"], row_end=st["end"])
    return A.aircache_paged_attend, prob, prob.new_workspace()


def run(state):
    if own:
        if "plan" not in state:
            state["plan"] = _plan(state)
        call, prob, ws = state["plan"]
        call(prob, ws)
    else:
        (_plain_shared if state["case"]["op"] == "shared" else _plain_attend)(state)
    if state["case"]["op"] == "shared":
        return {n: state[n] for n in ("out", "lse", "mass_out")}
    return {n: state[n] for n in ("out", "lse")}


def work(case):
    c = case
    new, rows, prefix, cu = _sizes(c)
    h, d = c["h_kv"], c["d"]
    row = h * (2 * d + 8 if c["int8"] else 4 * d)
    b = sum(new) * c["h_q"] * (4 * d + (4 if c["op"] == "shared" or c["lse"] else 0))
    if c["op"] == "shared":
        members = [n - m for m, n in zip(cu, cu[1:])]
        return {"bytes": b + sum(prefix) * row + sum(rows) * (row + (8 * h if c["mass"] else 0)),
                "flops": 4 * c["h_q"] * d * (sum(rows) + sum(p * m for p, m in zip(prefix, members)))}
    if c["op"] == "extend":
        pairs = sum(n * (R - n) + n * (n + 1) // 2 for n, R in zip(new, rows))
    elif c["images"]:
        begin, end = _ranges(c)
        pairs = sum(e - a for a, e in zip(begin, end))
    else:
        pairs = sum(n * R for n, R in zip(new, rows))
    return {"bytes": b + sum(rows) * row, "flops": 4 * c["h_q"] * d * pairs}


# ------------------------------------------------------------------ 64 bits

def _softmax_rows(q, k, v, scale, lo, hi):
    """Definition over rows lo..hi-1 of each query: q [M, D], k, v [R, D], lo, hi [M]; (out [M, D], lse [M], w [M, R])."""
    x = (q @ k.T) * scale
    r = torch.arange(k.shape[0], device=DEV)
    x[(r < lo[:, None]) | (r >= hi[:, None])] = -math.inf
    lse = torch.logsumexp(x, 1)
    w = torch.where(torch.isinf(lse)[:, None], 0.0, torch.exp(x - lse[:, None]))
    return w @ v, lse, w


def _numbers(ca, s, j):
    """Keys and values of sequence s and KV head j in 64 bits, and their places."""
    r = torch.arange(int(ca["lens"][s]), device=DEV)
    pg, r = ca["table"].long()[s, r // ca["page"]], r % ca["page"]
    k, v = ca["k"][pg, r, j].double(), ca["v"][pg, r, j].double()
    if ca["k_scale"] is not None:
        k, v = k * ca["k_scale"][pg, j, r].double()[:, None], v * ca["v_scale"][pg, j, r].double()[:, None]
    return k, v, pg, r


def exact(case, seed):
    """The definitions in 64 bits, one sequence, KV head and (for attention over a sequence) query head after the other."""
    st = prepare(case, seed)
    c, ca = st["case"], st["cache"]
    h, g, d = c["h_kv"], c["h_q"] // c["h_kv"], c["d"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    if c["op"] == "shared":
        mass = None if st["mass_out"] is None else torch.zeros(st["mass_out"].shape, dtype=torch.float64, device=DEV)
        owner = torch.bucketize(torch.arange(c["S"], device=DEV), st["cu"][1:].long(), right=True).tolist()
        for j in range(h):
            shared = [_numbers(st["prefix"], i, j)[:2] for i in range(c["G"])]
            for s in range(c["S"]):
                k, v, pg, r = _numbers(ca, s, j)
                if owner[s] < c["G"]:
                    k, v = torch.cat((shared[owner[s]][0], k)), torch.cat((shared[owner[s]][1], v))
                if len(k) == 0:
                    continue
                x = st["q"][s, j * g:(j + 1) * g].double() @ k.T / math.sqrt(d)
                lse[s, j * g:(j + 1) * g] = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
                out[s, j * g:(j + 1) * g] = w @ v
                if mass is not None:
                    mass[pg, j, r] = ca["mass"][pg, j, r].double() + w[:, len(k) - len(r):].sum(0)
        return {"out": out, "lse": lse, "mass_out": mass}
    for s, n in enumerate(st["new"]):
        R, t0 = int(ca["lens"][s]), st["at"][s]
        if R == 0:
            continue
        if c["op"] == "extend":
            hi = R - n + 1 + torch.arange(n, device=DEV)
            lo = torch.zeros_like(hi)
        elif st["end"] is not None:
            lo, hi = st["begin"][t0:t0 + n].long(), st["end"][t0:t0 + n].long()
        else:
            lo, hi = torch.zeros(n, dtype=torch.long, device=DEV), torch.full((n,), R, device=DEV)
        for j in range(h):
            k, v, _, _ = _numbers(ca, s, j)
            for i in range(j * g, (j + 1) * g):
                for a in range(0, n, 512):
                    tok = slice(t0 + a, t0 + min(n, a + 512))
                    part = slice(a, min(n, a + 512))
                    out[tok, i], lse[tok, i], _ = _softmax_rows(st["q"][tok, i].double(), k, v, d ** -0.5, lo[part], hi[part])
    return {"out": out, "lse": None if st["lse"] is None else lse}
