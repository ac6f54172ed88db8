"""Measured cases of the bounded-cache operators: attention under a sliding window with sink
tokens that stay visible, attention that also accumulates every key's attention weight, and the
eviction of a paged cache by that weight (choose the keys to keep, then compact the pages).

Each case is one call as a serving loop makes it. ``prepare`` makes the inputs from a seed: the
query rows, a paged K/V pool with shuffled pages, the per-key statistics, and the batch's plan.
``run`` makes one pass: with ``own`` false in plain torch operations, with ``own`` true through
this library. ``exact`` computes the same outputs in 64 bits, request by request.

Definitions (position p of a query, j of a key, g the KV head of query head h):
  visible(p, j) = j <= p and (window < 0 or p - j <= window or j < sinks)
  w(t, h, j)    = exp(scale <q, k_j>) / sum of the same over the keys visible from p
  out = sum_j w v_j,  lse = log sum_j exp(scale <q, k_j>)
  mass[g][j] (+)= sum over the step's rows t and the heads h of g of w(t, h, j); keys that the
                  step itself wrote start from zero, older keys add
  evict: of a request's n keys keep min(n, budget): first those among the first `sinks` or the
         last `recent` positions, then by mass, larger first, ties by lower slot; the kept keys
         of slots at or past the new length move, in order, into the evicted slots before it.
"""
import math

import numpy as np
import torch

own = False  # set by the caller: True runs the library's operators

LAYERS_ATTN = 1  # attention cases hold one layer's pool


# ------------------------------------------------------------------------------- the cases
def _attn(op, name, head_dim, hkv, mode, reqs, lo, hi, start_lo, start_hi, window, sinks, lens,
          page=16, hq=16, gain=2.0):
    return {"name": name, "op": op, "head_dim": head_dim, "hq": hq, "hkv": hkv, "mode": mode,
            "reqs": reqs, "lo": lo, "hi": hi, "start_lo": start_lo, "start_hi": start_hi,
            "window": window, "sinks": sinks, "lens": lens, "page": page, "gain": gain}


def _evict(op, name, head_dim, hkv, layers, reqs, lo, hi, budget, sinks, recent, evicted, lens,
           page=16):
    return {"name": name, "op": op, "head_dim": head_dim, "hkv": hkv, "layers": layers,
            "reqs": reqs, "lo": lo, "hi": hi, "budget": budget, "sinks": sinks, "recent": recent,
            "evicted": evicted, "lens": lens, "page": page}


def listed():
    return [
        # one user's next token on a local layer, long past the window: latency
        _attn("sink", "sink decode 1 hd256", 256, 8, "decode", 1, 1, 1, 5000, 5000, 1023, 4, 1),
        # a serving step of 64 requests on a local layer
        _attn("sink", "sink decode 64 hd256", 256, 8, "decode", 64, 1, 1, 0, 16383, 1023, 4, 2),
        # a ragged batch of prompts
        _attn("sink", "sink prefill 8 hd256", 256, 8, "prefill", 8, 128, 2048, 0, 0, 1023, 4, 3),
        # one long prompt, a page-sized block of sinks
        _attn("sink", "sink prefill 16384 hd256", 256, 8, "prefill", 1, 16384, 16384, 0, 0, 1023,
              64, 4),
        # one user's next token on a global layer whose cache is being scored
        _attn("mass", "mass decode 1 hd512", 512, 1, "decode", 1, 1, 1, 4095, 4095, -1, 0, 5),
        # a serving step of 64 requests on a global layer
        _attn("mass", "mass decode 64 hd512", 512, 1, "decode", 64, 1, 1, 0, 16383, -1, 0, 6),
        # a short prompt, and the next chunk of a longer one beside it
        _attn("mass", "mass prefill 2 hd512", 512, 1, "prefill", 2, 250, 512, 0, 1500, -1, 0, 7),
        # a long prompt scored as it is read
        _attn("mass", "mass prefill 8192 hd512", 512, 1, "prefill", 1, 8192, 8192, 0, 0, -1, 0, 8),
        # one request of one layer over its budget
        _evict("select", "select 1", 512, 1, 1, 1, 2048, 2048, 1024, 4, 128, 0, 9),
        # every layer and request of a serving step, each over its budget
        _evict("select", "select 64 x 8 layers", 512, 1, 8, 64, 4097, 16384, 4096, 4, 512, 777,
               10),
        # the steady state: each step brings one key and takes one away
        _evict("apply", "apply 64 x 8 layers, one key", 512, 1, 8, 64, 4097, 4097, 4096, 4, 512,
               777, 11),
        # half of a long cache goes at once
        _evict("apply", "apply 16 x 4 layers, half", 512, 1, 4, 16, 16384, 16384, 8192, 4, 512, 0,
               12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["sink", "sink", "mass", "mass", "select", "apply"])
    lens = rng.randrange(1 << 20)
    page = rng.choice([8, 16, 16, 16, 32, 64])
    head_dim = rng.choice([256, 512])
    if op in ("sink", "mass"):
        hq, hkv = rng.choice([(16, 8), (16, 4), (8, 8)] if head_dim == 256 else
                             [(16, 1), (16, 2), (8, 1)])
        mode = rng.choice(["decode", "prefill"])
        reqs = _log(rng, 1, 64 if mode == "decode" else 8)
        if op == "sink":
            window, sinks = _log(rng, 15, 2048), rng.choice([1, 4, 4, 16, 64, _log(rng, 1, 300)])
        else:
            window, sinks = rng.choice([(-1, 0), (-1, 0), (_log(rng, 100, 4096), 4)])
        if mode == "decode":
            top = _log(rng, 1, 16383 if head_dim == 512 or hkv < 8 else 8191)
            return _attn(op, None, head_dim, hkv, mode, reqs, 1, 1, 0, top, window, sinks, lens,
                         page, hq, rng.choice([1.0, 2.0, 3.0]))
        hi = _log(rng, 2, 4096 // reqs)
        lo = rng.randint(1, hi)
        top = _log(rng, 1, 2000) if rng.random() < 0.5 else 0
        return _attn(op, None, head_dim, hkv, mode, reqs, lo, hi, 0, top, window, sinks, lens,
                     page, hq, rng.choice([1.0, 2.0, 3.0]))
    hkv = rng.choice([1, 2]) if head_dim == 512 else rng.choice([4, 8])
    layers, reqs = rng.randint(1, 8 if hkv == 1 else 2), _log(rng, 1, 32)
    top = _log(rng, 64, 16384 if hkv == 1 else 4096)
    while layers * reqs * hkv * top > 4_000_000:  # the largest listed case's cost
        layers, reqs = max(1, layers // 2), max(1, reqs - reqs // 3) if layers == 1 else reqs
    budget = rng.randint(top // 8 + 4, top * 2 // 3)
    sinks = rng.choice([0, 4])
    recent = rng.randint(0, (budget - sinks) * 3 // 4)
    lo = rng.randint(1, budget) if reqs >= 8 else budget + 1  # some requests inside the budget
    return _evict(op, None, head_dim, hkv, layers, reqs, lo, top, budget, sinks,
                  recent, rng.choice([0, _log(rng, 1, 5000)]), lens, page)


# ------------------------------------------------------------------------------- the inputs
def _lengths(case):
    """(query tokens, first query position) of each request: the case alone says them."""
    r = np.random.RandomState(case["lens"] % (1 << 31))
    n = case["reqs"]
    if case["op"] in ("sink", "mass"):
        return (r.randint(case["lo"], case["hi"] + 1, n).astype(np.int64),
                r.randint(case["start_lo"], case["start_hi"] + 1, n).astype(np.int64))
    keys = r.randint(case["lo"], case["hi"] + 1, n).astype(np.int64)
    # after the step that wrote the last key: one query token, at the last position
    return np.ones(n, np.int64), keys - 1 + case["evicted"]


def _plan(case):
    """The batch's ragged geometry on the host."""
    qo, start = _lengths(case)
    evicted = case.get("evicted", 0)
    keys = start + qo - evicted  # keys held; slot = position - evicted
    ps = case["page"]
    npg = (keys + ps - 1) // ps
    return {"qo": qo, "start": start, "keys": keys, "npg": npg,
            "qo_indptr": np.concatenate([[0], np.cumsum(qo)]).astype(np.int64),
            "pg_indptr": np.concatenate([[0], np.cumsum(npg)]).astype(np.int64),
            "last": (keys - (npg - 1) * ps).astype(np.int32),
            "kv_start": np.full(len(qo), evicted, np.int64)}


def _normal(gen, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    p = _plan(case)
    ps, hkv, D, R = case["page"], case["hkv"], case["head_dim"], case["reqs"]
    layers = case.get("layers", LAYERS_ATTN)
    need = int(p["pg_indptr"][-1])
    num_pages = need + 3
    perm = torch.randperm(num_pages, device="cuda", generator=gen).to(torch.int32)
    ids = perm[:need].clone()
    # spare: a page of the pool that no request holds
    st = {"case": dict(case), "plan_host": p, "ids": ids, "spare": int(perm[need])}
    op = case["op"]
    if op != "select":
        # rows as prep leaves them: every key and value row has unit mean square
        st["pool"] = _normal(gen, (layers, num_pages, 2, hkv, ps, D))
    T = int(p["qo_indptr"][-1])
    if op in ("sink", "mass"):
        # the norm weights of queries and keys carry the scale (the attention itself is
        # unscaled): logits of standard deviation `gain`
        st["q"] = _normal(gen, (T, case["hq"], D), case["gain"] / math.sqrt(D))
        st["out"] = torch.zeros((T, case["hq"], D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros((T, case["hq"]), dtype=torch.float32, device="cuda")
    if op != "sink":
        shape = (layers, num_pages, hkv, ps)
        # accumulated weights: heavy-tailed, with exact zeros and equal values among them
        m = torch.empty(shape, device="cuda").normal_(0.0, 1.5, generator=gen).exp_()
        u = torch.rand(shape, device="cuda", generator=gen)
        m = torch.where(u < 0.03, torch.zeros_like(m), m)
        st["mass"] = torch.where(u > 0.95, torch.full_like(m, 0.25), m)
        st["pos"] = torch.full(shape, -1, dtype=torch.int32, device="cuda")
    # the batch's index tensors: every key held, with its request, slot, page and offset
    keys = torch.from_numpy(p["keys"]).cuda()
    kmax = int(p["keys"].max())
    slot = torch.arange(kmax, device="cuda")
    st["kmask"] = slot[None, :] < keys[:, None]                       # [R, kmax]
    pgi = torch.from_numpy(p["pg_indptr"][:-1].copy()).cuda()
    lp = torch.minimum(slot[None, :] // ps, (torch.from_numpy(p["npg"]).cuda() - 1)[:, None])
    st["kpage"] = ids.long()[pgi[:, None] + lp]                       # [R, kmax]
    st["koff"] = (slot % ps)[None, :].expand(R, kmax)
    flat = torch.nonzero(st["kmask"])
    st["kreq"], st["kslot"] = flat[:, 0].contiguous(), flat[:, 1].contiguous()
    st["start"] = torch.from_numpy(p["start"]).cuda()
    st["keys"] = keys
    if op in ("sink", "mass"):
        tmax = int(p["qo"].max())
        t = torch.arange(tmax, device="cuda")
        qo = torch.from_numpy(p["qo"]).cuda()
        st["tmask"] = t[None, :] < qo[:, None]                        # [R, tmax]
        q0 = torch.from_numpy(p["qo_indptr"][:-1].copy()).cuda()
        st["trow"] = torch.where(st["tmask"], q0[:, None] + t[None, :], 0)
        # the columns of keys that the plain form reads: a decode step under a window takes the
        # sinks before the window and the window, everything else every key held
        st["kcol"] = slot[None, :].expand(R, kmax)
        if op == "sink" and case["mode"] == "decode" and case["window"] >= 0:
            lo = (st["start"] - case["window"]).clamp_min(0)[:, None]
            a = torch.arange(min(case["sinks"], kmax), device="cuda")[None, :].expand(R, -1)
            b = lo + torch.arange(min(case["window"] + 1, kmax), device="cuda")[None, :]
            st["kcol"] = torch.cat([a, b.clamp_max(kmax - 1)], 1)
            st["cmask"] = torch.cat([a < lo, b < keys[:, None]], 1)
        else:
            st["cmask"] = st["kmask"]
        tf = torch.nonzero(st["tmask"])
        st["treq"], st["ttok"] = tf[:, 0].contiguous(), tf[:, 1].contiguous()
    else:
        # positions of the keys held: the first and the last ones are all there, others thinned
        # by earlier evictions, and an eighth of the slots out of order
        e = case["evicted"]
        n = keys[:, None].double()
        pos = torch.floor(slot[None, :].double() * ((n + e) / n)).long()
        tail = e + slot[None, :]
        pos = torch.where((slot[None, :] >= keys[:, None] - case["recent"]), tail, pos)
        pos = torch.where(slot[None, :] < case["sinks"], slot[None, :], pos)
        S = layers * R * hkv
        pos = pos[None, :, None, :].expand(layers, R, hkv, kmax).reshape(S, kmax)
        mask = st["kmask"][None, :, None, :].expand(layers, R, hkv, kmax).reshape(S, kmax)
        order = torch.rand((S, kmax), device="cuda", generator=gen)
        moved = (torch.rand((S, kmax), device="cuda", generator=gen) < 0.125) & mask
        # permute the moved slots among themselves: rank by slot against rank by random number
        by_slot = torch.sort(torch.where(moved, slot[None, :].double(), 2.0 * kmax), 1)[1]
        by_rand = torch.sort(torch.where(moved, order.double(), 2.0), 1)[1]
        shuffled = pos.clone()
        shuffled.scatter_(1, by_slot, torch.where(moved.gather(1, by_slot), pos.gather(1, by_rand),
                                                  pos.gather(1, by_slot)))
        val = shuffled.reshape(layers, R, hkv, kmax)[:, st["kreq"], :, st["kslot"]]
        st["pos"][:, st["kpage"][st["kreq"], st["kslot"]], :, st["koff"][st["kreq"], st["kslot"]]] = \
            val.to(torch.int32)
        st["src"] = torch.full((layers, R, hkv, case["budget"]), -1, dtype=torch.int32,
                               device="cuda")
        if op == "apply":
            st["src"].copy_(_select(st))
    if own:
        # the handles that a serving loop keeps: the plan, the descriptors and the workspace
        from paged_sliding_window_qkv_gb300 import pg
        hq = case.get("hq", hkv)
        rc, plan = pg.pg_plan_paged_segment(None, R, p["qo_indptr"], p["pg_indptr"],
                                            ids.cpu().numpy(), p["last"], p["kv_start"],
                                            p["start"], hq, hkv, D, ps)
        pg.check(rc, "pg_plan_paged_segment")
        st["plan"] = plan
        if op != "select":
            st["desc"] = pg.pool_descriptor(st["pool"])
        if op != "sink":
            st["stats"] = pg.stats_descriptor(st["mass"], st["pos"])
        if op in ("sink", "mass"):
            size = (pg.pg_workspace_bytes if op == "sink" else pg.pg_mass_workspace_bytes)(plan)
            st["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------- one pass
def _attention(st):
    """(out, lse, weights) of the padded batch in 32 bits: out [R, T, Hq, D], lse [R, T, Hq],
    weights [R, Hkv, G, T, K]."""
    c = st["case"]
    R, hq, hkv, D = c["reqs"], c["hq"], c["hkv"], c["head_dim"]
    G = hq // hkv
    rows = st["pool"][0].transpose(2, 3)  # [P, 2, ps, Hkv, D]
    page, off = st["kpage"].gather(1, st["kcol"]), st["koff"].gather(1, st["kcol"])
    K = rows[page, 0, off].float()  # [R, K, Hkv, D]
    V = rows[page, 1, off].float()
    T = st["trow"].shape[1]
    q = st["q"][st["trow"]].float().reshape(R, T, hkv, G, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.reshape(R, hkv, G * T, D), K.permute(0, 2, 3, 1)).reshape(R, hkv, G, T, -1)
    j = st["kcol"][:, None, :]
    p = (st["start"][:, None] + torch.arange(T, device="cuda")[None, :])[:, :, None]
    vis = (j <= p) & st["cmask"][:, None, :]
    if c["window"] >= 0:
        vis &= (p - j <= c["window"]) | (j < c["sinks"])
    s.masked_fill_(~vis[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_min(-3.0e38)
    w = s.sub_(m).exp_()
    den = w.sum(-1, keepdim=True)
    lse = (m + den.log())[..., 0]                       # [R, Hkv, G, T]
    w = w.div_(den.clamp_min(1e-38))
    o = torch.matmul(w.reshape(R, hkv, G * T, -1), V.permute(0, 2, 1, 3)).reshape(R, hkv, G, T, D)
    return o.permute(0, 3, 1, 2, 4).reshape(R, T, hq, D), lse.permute(0, 3, 1, 2).reshape(R, T, hq), w


def _select(st):
    """The source slot of each kept slot, [layers, R, Hkv, budget] (-1 past the keys kept)."""
    c = st["case"]
    L, R, hkv, budget = c["layers"], c["reqs"], c["hkv"], c["budget"]
    take = lambda x: x.transpose(2, 3)[:, st["kpage"], st["koff"]].permute(0, 1, 3, 2)  # noqa: E731
    mass, pos = take(st["mass"]), take(st["pos"])       # [L, R, Hkv, K]
    n = st["keys"][None, :, None, None]
    end = st["start"][None, :, None, None] + 1
    slot = torch.arange(mass.shape[-1], device="cuda")[None, None, None, :]
    held = slot < n
    kept_first = (pos < c["sinks"]) | (pos >= end - c["recent"])
    held = held.expand(mass.shape)
    rank = torch.where(held, torch.where(kept_first, 2, 1), 0)
    mass = torch.where(torch.isnan(mass), float("-inf"), mass)
    by_mass = torch.sort(mass, dim=-1, descending=True, stable=True)[1]
    order = by_mass.gather(-1, torch.sort(rank.gather(-1, by_mass), dim=-1, descending=True,
                                          stable=True)[1])
    new = n.clamp_max(budget)
    kept = torch.zeros_like(held).scatter_(-1, order, (slot < new).expand(held.shape))
    hole, mover = (slot < new) & ~kept, (slot >= new) & kept
    K = mass.shape[-1]
    movers = torch.full((L, R, hkv, K + 1), -1, device="cuda")
    movers.scatter_(-1, torch.where(mover, mover.cumsum(-1) - 1, K), slot.expand(mover.shape))
    src = torch.where(hole, movers.gather(-1, (hole.cumsum(-1) - 1).clamp_min(0)), slot)
    src = torch.where(slot < new, src, -1)
    src = src[..., :budget].to(torch.int32)
    return torch.nn.functional.pad(src, (0, budget - src.shape[-1]), value=-1)


def _apply(st):
    """Copy each moved key's rows, weight and position into its new slot."""
    c = st["case"]
    b = min(c["budget"], st["kpage"].shape[1])
    most = min(b, st["kpage"].shape[1] - b)              # moves of one head of one request
    if most <= 0:
        return
    src = st["src"][..., :b].long()                      # [L, R, Hkv, b]
    slot = torch.arange(b, device="cuda")[None, None, None, :]
    moved = (src >= 0) & (src != slot)
    to = torch.sort(moved.to(torch.uint8), dim=-1, descending=True, stable=True)[1][..., :most]
    src = src.gather(-1, to)
    src = torch.where(src >= 0, src, to)                 # unmoved slots copy themselves
    R = torch.arange(c["reqs"], device="cuda")[None, :, None, None]
    L = torch.arange(c["layers"], device="cuda")[:, None, None, None]
    H = torch.arange(c["hkv"], device="cuda")[None, None, :, None]
    live = st["kmask"][R, to]
    fp, fo = st["kpage"][R, src], st["koff"][R, src]
    tp, to = st["kpage"][R, to], st["koff"][R, to]
    # padding columns of short requests write to a page that no request holds
    spare = st["spare"]
    tp, to = torch.where(live, tp, spare), torch.where(live, to, 0)
    for_rows = st["pool"].transpose(2, 3)                # [L, P, Hkv, 2, ps, D]
    keep = st["pool"][:, spare, :, :, 0].clone(), st["mass"][:, spare, :, 0].clone(), \
        st["pos"][:, spare, :, 0].clone()
    for_rows[L, tp, H, 0, to] = for_rows[L, fp, H, 0, fo]
    for_rows[L, tp, H, 1, to] = for_rows[L, fp, H, 1, fo]
    st["mass"][L, tp, H, to] = st["mass"][L, fp, H, fo]
    st["pos"][L, tp, H, to] = st["pos"][L, fp, H, fo]
    st["pool"][:, spare, :, :, 0], st["mass"][:, spare, :, 0], st["pos"][:, spare, :, 0] = keep


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        from paged_sliding_window_qkv_gb300 import pg
        if op == "sink":
            pg.check(pg.pg_attn_paged_sink(st["plan"], st["desc"], 0, st["q"], st["out"], st["lse"],
                                           c["window"], c["sinks"], 1.0, st["ws"],
                                           st["ws"].numel()))
            return {"out": st["out"], "lse": st["lse"]}
        if op == "mass":
            pg.check(pg.pg_attn_paged_mass(st["plan"], st["desc"], 0, st["q"], st["out"], st["lse"],
                                           st["stats"], c["window"], c["sinks"], 1.0, st["ws"],
                                           st["ws"].numel()))
            return {"out": st["out"], "lse": st["lse"], "mass": st["mass"], "pos": st["pos"]}
        if op == "select":
            pg.check(pg.pg_kv_evict_select(st["plan"], st["stats"], 0, c["layers"], c["budget"],
                                           c["sinks"], c["recent"], st["src"]))
            return {"src": st["src"]}
        pg.check(pg.pg_kv_evict_apply(st["plan"], st["desc"], st["stats"], 0, c["layers"],
                                      c["budget"], st["src"]))
        return {"pool": st["pool"], "mass": st["mass"], "pos": st["pos"]}
    if op == "select":
        return {"src": _select(st)}
    if op == "apply":
        _apply(st)
        return {"pool": st["pool"], "mass": st["mass"], "pos": st["pos"]}
    o, lse, w = _attention(st)
    out = {"out": o[st["treq"], st["ttok"]].to(torch.bfloat16), "lse": lse[st["treq"], st["ttok"]]}
    if op == "mass":
        w = torch.where(st["tmask"][:, None, None, :, None], w, 0.0)
        add = w.sum((2, 3))                              # [R, Hkv, K]
        r, s = st["kreq"], st["kslot"]
        page, off = st["kpage"][r, s], st["koff"][r, s]
        new = (s >= st["start"][r])[:, None]
        mass, pos = st["mass"][0], st["pos"][0]
        mass[page, :, off] = torch.where(new, 0.0, mass[page, :, off]) + add[r, :, s]
        pos[page, :, off] = torch.where(new, s[:, None].to(torch.int32), pos[page, :, off])
        out |= {"mass": st["mass"], "pos": st["pos"]}
    return out


# ------------------------------------------------------------------------------- its work
def work(case):
    p = _plan(case)
    D, hkv = case["head_dim"], case["hkv"]
    if case["op"] in ("sink", "mass"):
        hq, W, ns = case["hq"], case["window"], case["sinks"]
        pairs = read = 0
        for t, s in zip(p["qo"], p["start"]):
            pos = np.arange(s, s + t)
            lo = np.maximum(pos - W, 0) if W >= 0 else np.zeros_like(pos)
            extra = np.minimum(lo, ns) if W >= 0 else 0
            pairs += int((pos - lo + 1 + extra).sum())
            first = int(lo[0])
            read += int(s + t - first) + (min(first, ns) if W >= 0 else 0)
        T = int(p["qo"].sum())
        nbytes = read * hkv * D * 2 * 2 + 2 * T * hq * D * 2 + T * hq * 4 + len(p["npg"]) * 32
        if case["op"] == "mass":
            old = int(p["start"].sum())
            nbytes += hkv * (read * 4 + min(read, old) * 4 + T * 4)
        return {"bytes": nbytes, "flops": 4 * D * hq * pairs}
    segs = case["layers"] * hkv
    n, b = p["keys"], np.minimum(p["keys"], case["budget"])
    if case["op"] == "select":
        return {"bytes": int(segs * (n.sum() * 8 + case["reqs"] * case["budget"] * 4)), "flops": 0}
    moves = float((b * (n - b) / n).sum()) * segs  # kept keys past the new length, on average
    return {"bytes": segs * case["reqs"] * case["budget"] * 4 + moves * 2 * (2 * D * 2 + 8),
            "flops": 0}


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    p, op = st["plan_host"], case["op"]
    if op == "select":
        return None  # whole numbers alone
    ps, hkv = case["page"], case["hkv"]
    ids = st["ids"].long()
    if op == "apply":
        pool, mass, pos = st["pool"].clone(), st["mass"].double(), st["pos"].clone()
        old_pool, old_mass = st["pool"], mass.clone()
        for r in range(case["reqs"]):
            pages = ids[int(p["pg_indptr"][r]):int(p["pg_indptr"][r + 1])]
            for layer in range(case["layers"]):
                for g in range(hkv):
                    src = st["src"][layer, r, g].long()
                    src = src[src >= 0]
                    to = torch.arange(len(src), device="cuda")
                    a, b = pages[to // ps], to % ps
                    x, y = pages[src // ps], src % ps
                    pool[layer, a, :, g, b] = old_pool[layer, x, :, g, y]
                    mass[layer, a, g, b] = old_mass[layer, x, g, y]
        return {"pool": pool, "mass": mass, "pos": None}
    T, hq, D = st["q"].shape
    G = hq // hkv
    out = torch.zeros((T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, hq), dtype=torch.float64, device="cuda")
    mass = st["mass"].double() if op == "mass" else None
    for r in range(case["reqs"]):
        n, t0, t1 = int(p["keys"][r]), int(p["qo_indptr"][r]), int(p["qo_indptr"][r + 1])
        start = int(p["start"][r])
        pages = ids[int(p["pg_indptr"][r]):int(p["pg_indptr"][r + 1])]
        where = torch.arange(n, device="cuda")
        position = torch.arange(start, start + t1 - t0, device="cuda")[:, None]
        hidden = where[None, :] > position
        if case["window"] >= 0:
            hidden |= (position - where[None, :] > case["window"]) & (where[None, :] >= case["sinks"])
        for g in range(hkv):
            k = st["pool"][0, pages, 0, g].reshape(-1, D)[:n].double()
            v = st["pool"][0, pages, 1, g].reshape(-1, D)[:n].double()
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for h in range(g * G, (g + 1) * G):
                z = (st["q"][t0:t1, h].double() @ k.T).masked_fill(hidden, float("-inf"))
                norm = torch.logsumexp(z, 1)
                z = torch.exp(z - norm[:, None])
                out[t0:t1, h] = z @ v
                lse[t0:t1, h] = norm
                got += z.sum(0)
                del z
            if op == "mass":
                a, b = pages[where // ps], where % ps
                mass[0, a, g, b] = torch.where(where >= start, 0.0, mass[0, a, g, b]) + got
    res = {"out": out, "lse": lse}
    return res | {"mass": mass, "pos": None} if op == "mass" else res
