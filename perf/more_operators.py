"""Measured cases of the operators that let a serving step read less of its cache: prep that writes
K and V into an 8-bit pool, attention that reads such a pool, the way back into a bf16 pool, and
attention for requests that share a prefix, whose keys are read once for all of them.

``prepare`` makes a case's inputs from a seed: raw or prepared rows, a pool with shuffled pages, and
the batch's plan. ``run`` makes one pass: with ``own`` false in plain torch operations, with ``own``
true through this library. ``exact`` computes the same outputs in 64 bits, request by request.

Definitions. A quantised row y[0..D) is a scale 2^e and D e4m3 codes:
  e = the least integer with max|y| <= 448 * 2^e, held to [-110, 120] (the least for a row of zeros)
  code = y * 2^-e rounded to nearest even, and the row stands for code * 2^e
Prep: K = rope(x / rms(x) * w), V = v / rms(v) (head_dim 512: of the same raw K), q = rope(...) in bf16.
Attention from position p, of a request's keys j held in slots j - kv_start:
  visible(p, j) = j <= p and (window < 0 or p - j <= window or j < sinks)
  out = sum_j w_j v_j, w = softmax over the visible keys of scale <q, k_j>; lse the log normaliser
Shared prefix: the first keys of every request of a group are the same pages; nothing else changes.
"""
import math

import numpy as np
import torch

own = False  # set by the caller: True runs the library's operators

EPS = 1e-6


# ------------------------------------------------------------------------------- the cases
def _write(name, head_dim, hq, hkv, reqs, lo, hi, start_hi, lens, page=16):
    return {"name": name, "op": "write", "head_dim": head_dim, "hq": hq, "hkv": hkv, "reqs": reqs,
            "lo": lo, "hi": hi, "start_lo": 0, "start_hi": start_hi, "lens": lens, "page": page}


def _read(name, head_dim, hkv, layers, reqs, lo, hi, lens, page=16):
    return {"name": name, "op": "read", "head_dim": head_dim, "hq": hkv, "hkv": hkv,
            "layers": layers, "reqs": reqs, "lo": 1, "hi": 1, "start_lo": lo - 1,
            "start_hi": hi - 1, "lens": lens, "page": page}


def _attn(name, head_dim, hq, hkv, reqs, lo, hi, start_lo, start_hi, window, sinks, lens, page=16,
          gain=2.0, evicted=0):
    return {"name": name, "op": "attn", "head_dim": head_dim, "hq": hq, "hkv": hkv, "reqs": reqs,
            "lo": lo, "hi": hi, "start_lo": start_lo, "start_hi": start_hi, "window": window,
            "sinks": sinks, "evicted": evicted, "lens": lens, "page": page, "gain": gain}


def _shared(name, head_dim, hq, hkv, groups, reqs, prefix_lo, prefix_hi, lo, hi, start_hi, q8, lens,
            page=16, gain=2.0):
    """prefix_lo..prefix_hi: pages of a group's prefix; start_hi: own keys before the step."""
    return {"name": name, "op": "shared", "head_dim": head_dim, "hq": hq, "hkv": hkv,
            "groups": groups, "reqs": reqs, "prefix_lo": prefix_lo, "prefix_hi": prefix_hi,
            "lo": lo, "hi": hi, "start_lo": 0, "start_hi": start_hi, "q8": q8, "lens": lens,
            "page": page, "gain": gain, "window": -1, "sinks": 0}


def listed():
    return [
        # a serving step's new tokens on a global layer: latency
        _write("write decode 64 hd512", 512, 16, 1, 64, 1, 1, 16383, 1),
        # a long prompt on a local layer
        _write("write prefill 16384 hd256", 256, 16, 8, 1, 16384, 16384, 0, 2),
        # one request's cache back into a bf16 pool (to be weighed and evicted there)
        _read("read 1 hd512", 512, 1, 1, 1, 4097, 4097, 3),
        # two layers' caches of a batch
        _read("read 32 x 2 layers hd512", 512, 1, 2, 32, 1, 16384, 4),
        # one user's next token on a global layer: latency
        _attn("q8 decode 1 hd512", 512, 16, 1, 1, 1, 1, 8000, 8000, -1, 0, 5),
        # a serving step of 64 requests on a global layer
        _attn("q8 decode 64 hd512", 512, 16, 1, 64, 1, 1, 0, 16383, -1, 0, 6),
        # the same step on a local layer: window and sinks
        _attn("q8 decode 64 hd256", 256, 16, 8, 64, 1, 1, 0, 16383, 1023, 4, 7),
        # the next chunks of four long prompts
        _attn("q8 chunks 4 hd512", 512, 16, 1, 4, 100, 512, 0, 8000, -1, 0, 8),
        # a few requests on one system prompt, local head geometry: latency
        _shared("shared decode 4 hd256", 256, 16, 8, 1, 4, 128, 128, 1, 1, 200, False, 9),
        # a serving step of 64 requests on one long document
        _shared("shared decode 64 hd512", 512, 16, 1, 1, 64, 512, 512, 1, 1, 1023, False, 10),
        # eight prompts behind the same long instructions
        _shared("shared prefill 8 hd512", 512, 16, 1, 1, 8, 256, 256, 1, 512, 0, False, 11),
        # four documents with sixteen requests each, over a quantised cache
        _shared("shared q8 decode 64 hd512", 512, 16, 1, 4, 64, 200, 600, 1, 1, 1023, True, 12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["write", "read", "attn", "attn", "shared", "shared"])
    lens = rng.randrange(1 << 20)
    page = rng.choice([8, 16, 16, 16, 32, 64])
    head_dim = rng.choice([256, 512])
    hq, hkv = rng.choice([(16, 8), (16, 4), (8, 8)] if head_dim == 256 else
                         [(16, 1), (16, 2), (8, 1)])
    gain = rng.choice([1.0, 2.0, 3.0])
    if op == "write":
        reqs = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 8192 // reqs))
        top = min(8000, 250_000_000 // (reqs * hkv * head_dim))  # a pool of half a gigabyte
        return _write(None, head_dim, hq, hkv, reqs, rng.randint(1, hi), hi,
                      rng.choice([0, _log(rng, 1, top)]), lens, page)
    if op == "read":
        layers, reqs = rng.randint(1, 4), _log(rng, 1, 32)
        top = _log(rng, 1, max(2, 500_000 // (layers * reqs * hkv)))
        return _read(None, head_dim, hkv, layers, reqs, rng.randint(1, top), min(top, 16384), lens,
                     page) if top <= 16384 else \
            _read(None, head_dim, hkv, layers, reqs, 1, 16384, lens, page)
    decode = rng.random() < 0.6
    reqs = _log(rng, 1, 64 if decode else 8)
    if op == "attn":
        window, sinks = rng.choice([(-1, 0), (-1, 0), (_log(rng, 15, 2048), rng.choice([0, 4, 64]))])
        evicted = rng.choice([0, 0, _log(rng, 1, 3000)])
        if decode:
            top = _log(rng, 1, 16383 if hkv <= 2 else 4000)
            return _attn(None, head_dim, hq, hkv, reqs, 1, 1, 0, top, window, sinks, lens, page,
                         gain, evicted)
        hi = _log(rng, 2, 2048 // reqs)
        top = _log(rng, 1, 4000) if rng.random() < 0.6 else 0
        return _attn(None, head_dim, hq, hkv, reqs, rng.randint(1, hi), hi, 0, top, window, sinks,
                     lens, page, gain, evicted)
    groups = rng.randint(1, min(4, reqs))
    top = max(1, _log(rng, 16, 8192 if hkv <= 2 else 3000) // page)
    low = rng.randint(0, top)
    q8 = rng.random() < 0.5
    if decode:
        return _shared(None, head_dim, hq, hkv, groups, reqs, low, top, 1, 1, _log(rng, 1, 1000),
                       q8, lens, page, gain)
    hi = _log(rng, 2, 2048 // reqs)
    return _shared(None, head_dim, hq, hkv, groups, reqs, low, top, rng.randint(1, hi), hi,
                   rng.choice([0, _log(rng, 1, 500)]), q8, lens, page, gain)


# ------------------------------------------------------------------------------- the inputs
def _plan(case):
    """The batch's ragged geometry on the host: the case alone says it."""
    r = np.random.RandomState(case["lens"] % (1 << 31))
    n, ps = case["reqs"], case["page"]
    qo = r.randint(case["lo"], case["hi"] + 1, n).astype(np.int64)
    start = r.randint(case["start_lo"], case["start_hi"] + 1, n).astype(np.int64)
    p = {"qo": qo}
    if case["op"] == "shared":
        g = case["groups"]
        cuts = np.sort(r.permutation(n - 1)[:g - 1] + 1) if g > 1 else np.zeros(0, np.int64)
        p["group_indptr"] = np.concatenate([[0], cuts, [n]]).astype(np.int64)
        pages = r.randint(case["prefix_lo"], case["prefix_hi"] + 1, g).astype(np.int64)
        p["prefix"] = pages * ps
        p["of"] = np.repeat(np.arange(g), np.diff(p["group_indptr"]))
        start = start + p["prefix"][p["of"]]
    evicted = np.minimum(case.get("evicted", 0), start)
    keys = start + qo - evicted
    npg = (keys + ps - 1) // ps
    p |= {"start": start, "keys": keys, "npg": npg, "kv_start": evicted,
          "qo_indptr": np.concatenate([[0], np.cumsum(qo)]).astype(np.int64),
          "pg_indptr": np.concatenate([[0], np.cumsum(npg)]).astype(np.int64),
          "last": (keys - (npg - 1) * ps).astype(np.int32)}
    return p


def _normal(gen, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def _pages(case, p, gen):
    """Page ids of the batch, shuffled; a group's requests list the same prefix pages."""
    total = int(p["pg_indptr"][-1])
    perm = torch.randperm(total + 3, device="cuda", generator=gen).to(torch.int32)
    ids = perm[:total].clone()
    if case["op"] == "shared":
        take = np.arange(total)
        for r in range(case["reqs"]):
            first = int(p["group_indptr"][p["of"][r]])
            k = int(p["prefix"][p["of"][r]]) // case["page"]
            a, b = int(p["pg_indptr"][first]), int(p["pg_indptr"][r])
            take[b:b + k] = np.arange(a, a + k)
        ids = ids[torch.from_numpy(take).cuda()]
    return ids, total + 3


def _quantise(y):
    """e4m3 codes and e8m0 scales of the rows of y (float32 or float64)."""
    m, x = torch.frexp(y.abs().amax(-1))
    e = torch.where(m > 0, x - 9 + (m > 0.875), -110).clamp(-110, 120)
    code = torch.ldexp(y, -e[..., None]).float().to(torch.float8_e4m3fn)
    return code, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(codes, scales, dtype=torch.float32):
    return codes.to(dtype) * scales.to(dtype)[..., None]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    p = _plan(case)
    op, ps, hq, hkv, D, R = (case[k] for k in ("op", "page", "hq", "hkv", "head_dim", "reqs"))
    layers = case.get("layers", 1)
    ids, num_pages = _pages(case, p, gen)
    T = int(p["qo_indptr"][-1])
    st = {"case": dict(case), "plan_host": p, "ids": ids}
    rows = (layers, num_pages, 2, hkv, ps)
    if op == "write":
        # rows of one fused projection: q, k and v side by side, a common token stride
        cols = (hq + (2 if D == 256 else 1) * hkv) * D
        raw = _normal(gen, (T, cols))
        st["q_raw"] = raw[:, :hq * D].unflatten(1, (hq, D))
        st["k_raw"] = raw[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        st["v_raw"] = raw[:, (hq + hkv) * D:].unflatten(1, (hkv, D)) if D == 256 else None
        st["stride"] = cols
        st["w_q"], st["w_k"] = (1.0 + 0.1 * _normal(gen, (2, D)).float()).to(torch.bfloat16)
        top = int((p["start"] + p["qo"]).max())
        freq = (1e4 if D == 256 else 1e6) ** (-2.0 * torch.arange(D // 2, device="cuda").double() / D)
        angle = torch.arange(top, device="cuda").double()[:, None] * freq
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
        st["codes"] = torch.zeros(rows + (D,), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.full(rows, 127, dtype=torch.uint8, device="cuda")
        st["q"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
    elif op == "shared" and not case["q8"]:
        st["pool"] = _normal(gen, rows + (D,))
    else:
        # rows as prep leaves them: unit mean square before they are rounded to codes
        st["codes"] = torch.empty(rows + (D,), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(rows, dtype=torch.uint8, device="cuda")
        for i in range(layers):
            for a in range(0, num_pages, 4096):
                c, s = _quantise(_normal(gen, (min(4096, num_pages - a),) + rows[2:] + (D,)).float())
                st["codes"][i, a:a + 4096] = c.view(torch.uint8)
                st["scales"][i, a:a + 4096] = s.view(torch.uint8)
    if op == "read":
        st["pool"] = torch.zeros(rows + (D,), dtype=torch.bfloat16, device="cuda")
    if op in ("attn", "shared"):
        # the norm weights of queries and keys carry the scale: logits of standard deviation `gain`
        st["q"] = _normal(gen, (T, hq, D), case["gain"] / math.sqrt(D))
        st["out"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros((T, hq), dtype=torch.float32, device="cuda")
    # the batch's index tensors
    pgi = torch.from_numpy(p["pg_indptr"][:-1].copy()).cuda()
    npg = torch.from_numpy(p["npg"]).cuda()
    keys, start, ks = (torch.from_numpy(p[k]).cuda() for k in ("keys", "start", "kv_start"))
    qo = torch.from_numpy(p["qo"]).cuda()
    if op == "write":
        req = torch.repeat_interleave(torch.arange(R, device="cuda"), qo)
        t = torch.arange(T, device="cuda") - torch.from_numpy(p["qo_indptr"][:-1].copy()).cuda()[req]
        st["tpos"] = start[req] + t
        st["tpage"] = ids.long()[pgi[req] + st["tpos"] // ps]
        st["toff"] = st["tpos"] % ps
    else:
        slot = torch.arange(int(p["keys"].max()), device="cuda")
        held = slot[None, :] < keys[:, None]
        st["kreq"], st["kslot"] = torch.nonzero(held, as_tuple=True)
        lp = torch.minimum(slot[None, :] // ps, npg[:, None] - 1)
        st["kpage"] = ids.long()[pgi[:, None] + lp]
        st["koff"] = (slot % ps)[None, :].expand(R, -1)
        if op != "read":
            kpos = ks[:, None] + slot[None, :]
            W = case["window"]
            # a decode step under a window reads the sinks before it and the window alone
            if case["hi"] == 1 and W >= 0:
                lo = (start - W - ks).clamp_min(0)[:, None]
                a = slot[None, :min(case["sinks"], len(slot))].expand(R, -1)
                b = lo + slot[None, :min(W + 1, len(slot))]
                col = torch.cat([a, b.clamp_max(len(slot) - 1)], 1)
                live = torch.cat([(a < lo) & (a < keys[:, None]), b < keys[:, None]], 1)
                st["kpage"], st["koff"] = st["kpage"].gather(1, col), st["koff"].gather(1, col)
                kpos, held = kpos.gather(1, col), live
            st["kpos"], st["held"] = kpos, held
            t = torch.arange(int(p["qo"].max()), device="cuda")
            tmask = t[None, :] < qo[:, None]
            q0 = torch.from_numpy(p["qo_indptr"][:-1].copy()).cuda()
            st["trow"] = torch.where(tmask, q0[:, None] + t[None, :], 0)
            st["tpos"] = start[:, None] + t[None, :]
            st["treq"], st["ttok"] = torch.nonzero(tmask, as_tuple=True)
    if own:
        # the handles that a serving loop keeps: the plan, the descriptors and the workspace
        from paged_sliding_window_qkv_gb300 import pg
        host = ids.cpu().numpy()
        if op == "shared":
            rc, plan = pg.pg_plan_paged_shared(None, R, p["qo_indptr"], p["pg_indptr"], host,
                                               p["last"], p["start"], case["groups"],
                                               p["group_indptr"], p["prefix"], hq, hkv, D, ps)
            pg.check(rc, "pg_plan_paged_shared")
        else:
            rc, plan = pg.pg_plan_paged_segment(None, R, p["qo_indptr"], p["pg_indptr"], host,
                                                p["last"], p["kv_start"], p["start"], hq, hkv, D, ps)
            pg.check(rc, "pg_plan_paged_segment")
        st["plan"] = plan
        if "codes" in st:
            st["q8"] = pg.q8_descriptor(st["codes"], st["scales"])
        if "pool" in st:
            st["desc"] = pg.pool_descriptor(st["pool"])
        if op in ("attn", "shared"):
            size = pg.pg_q8_workspace_bytes(plan) if op == "attn" else \
                pg.pg_shared_q8_workspace_bytes(plan) if case["q8"] else \
                pg.pg_shared_workspace_bytes(plan)
            st["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------- one pass
def _normed(x, dtype):
    x = x.to(dtype)
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _roped(x, w, cos, sin):
    x = x * w.to(x.dtype)
    a, b = x.chunk(2, -1)
    c, s = cos[:, None].to(x.dtype), sin[:, None].to(x.dtype)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _prep(st, dtype):
    """q, K and V of the step's tokens, not yet rounded."""
    cos, sin = st["cos"][st["tpos"]], st["sin"][st["tpos"]]
    q = _roped(_normed(st["q_raw"], dtype), st["w_q"], cos, sin)
    k = _normed(st["k_raw"], dtype)
    v = _normed(st["v_raw"], dtype) if st["v_raw"] is not None else k
    return q, _roped(k, st["w_k"], cos, sin), v


def _codes(st):
    return st["codes"].view(torch.float8_e4m3fn), st["scales"].view(torch.float8_e8m0fnu)


def _attention(st):
    c = st["case"]
    R, hq, hkv, D = c["reqs"], c["hq"], c["hkv"], c["head_dim"]
    G = hq // hkv

    def rows(kv):  # [R, K, Hkv, D]
        if "pool" in st:
            return st["pool"][0].transpose(2, 3)[st["kpage"], kv, st["koff"]].float()
        codes, scales = st["codes"][0].transpose(2, 3), st["scales"][0].transpose(2, 3)
        at = (st["kpage"], kv, st["koff"])
        return _values(codes[at].view(torch.float8_e4m3fn), scales[at].view(torch.float8_e8m0fnu))

    T = st["trow"].shape[1]
    q = st["q"][st["trow"]].float().reshape(R, T, hkv, G, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.reshape(R, hkv, G * T, D), rows(0).permute(0, 2, 3, 1)).reshape(R, hkv, G, T, -1)
    j, p = st["kpos"][:, None, :], st["tpos"][:, :, None]
    vis = (j <= p) & st["held"][:, None, :]
    if c["window"] >= 0:
        vis &= (p - j <= c["window"]) | (j < c["sinks"])
    s.masked_fill_(~vis[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_min(-3.0e38)
    w = s.sub_(m).exp_()
    den = w.sum(-1, keepdim=True)
    lse = (m + den.log())[..., 0]
    w = w.div_(den.clamp_min(1e-38))
    o = torch.matmul(w.reshape(R, hkv, G * T, -1), rows(1).permute(0, 2, 1, 3)).reshape(R, hkv, G, T, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(R, T, hq, D)
    lse = lse.permute(0, 3, 1, 2).reshape(R, T, hq)
    at = (st["treq"], st["ttok"])
    return {"out": o[at].to(torch.bfloat16), "lse": lse[at]}


def _run_own(st):
    from paged_sliding_window_qkv_gb300 import pg
    c = st["case"]
    op = c["op"]
    if op == "write":
        pg.check(pg.pg_prep_paged_q8(st["plan"], st["q8"], 0, st["q_raw"], st["stride"], st["k_raw"],
                                     st["stride"], st["v_raw"], st["stride"], st["w_q"], st["w_k"],
                                     EPS, st["cos"], st["sin"], st["cos"].shape[0], st["q"]))
        codes, scales = _codes(st)
        return {"q": st["q"], "codes": codes, "scales": scales}
    if op == "read":
        pg.check(pg.pg_kv_dequantize(st["plan"], st["q8"], st["desc"], 0, c["layers"]))
        return {"pool": st["pool"]}
    if op == "attn":
        pg.check(pg.pg_attn_paged_q8(st["plan"], st["q8"], 0, st["q"], st["out"], st["lse"],
                                     c["window"], c["sinks"], 1.0, st["ws"], st["ws"].numel()))
    elif c["q8"]:
        pg.check(pg.pg_attn_paged_shared_q8(st["plan"], st["q8"], 0, st["q"], st["out"], st["lse"],
                                            1.0, st["ws"], st["ws"].numel()))
    else:
        pg.check(pg.pg_attn_paged_shared(st["plan"], st["desc"], 0, st["q"], st["out"], st["lse"],
                                         1.0, st["ws"], st["ws"].numel()))
    return {"out": st["out"], "lse": st["lse"]}


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "write":
        q, k, v = _prep(st, torch.float32)
        st["q"].copy_(q)
        for i, y in enumerate((k, v)):
            c, s = _quantise(y)
            st["codes"][0, st["tpage"], i, :, st["toff"]] = c.view(torch.uint8)
            st["scales"][0, st["tpage"], i, :, st["toff"]] = s.view(torch.uint8)
        codes, scales = _codes(st)
        return {"q": st["q"], "codes": codes, "scales": scales}
    if op == "read":
        page, off = (st[k][st["kreq"], st["kslot"]] for k in ("kpage", "koff"))
        for i in range(st["case"]["layers"]):
            y = _values(st["codes"][i].transpose(2, 3)[page, :, off].view(torch.float8_e4m3fn),
                        st["scales"][i].transpose(2, 3)[page, :, off].view(torch.float8_e8m0fnu))
            st["pool"][i].transpose(2, 3)[page, :, off] = y.to(torch.bfloat16)
        return {"pool": st["pool"]}
    return _attention(st)


# ------------------------------------------------------------------------------- its work
def work(case):
    p = _plan(case)
    D, hq, hkv, op = case["head_dim"], case["hq"], case["hkv"], case["op"]
    T = int(p["qo"].sum())
    row = D + 1  # a quantised row: codes and scale
    if op == "write":
        raw = (hq + (2 if D == 256 else 1) * hkv) * D * 2
        rope = len(np.unique(np.concatenate([np.arange(s, s + t) for s, t in zip(p["start"], p["qo"])])))
        return {"bytes": T * (raw + hq * D * 2 + 2 * hkv * row) + rope * D * 4, "flops": 0}
    if op == "read":
        return {"bytes": int(p["keys"].sum()) * case["layers"] * 2 * hkv * (row + 2 * D), "flops": 0}
    W, ns = case["window"], case["sinks"]
    pairs = read = 0
    for t, s, e in zip(p["qo"], p["start"], p["kv_start"]):
        pos = np.arange(s, s + t)
        lo = np.maximum(pos - W, e) if W >= 0 else np.full_like(pos, e)
        extra = np.clip(np.minimum(lo, ns) - e, 0, None) if W >= 0 else 0
        pairs += int((pos - lo + 1 + extra).sum())
        first = int(lo[0])
        read += int(s + t - first) + (max(min(first, ns) - int(e), 0) if W >= 0 else 0)
    if op == "shared":
        read -= int((p["prefix"] * (np.diff(p["group_indptr"]) - 1)).sum())
    key = 2 * hkv * (row if op == "attn" or case["q8"] else 2 * D)
    return {"bytes": read * key + T * hq * (4 * D + 4) + len(p["npg"]) * 32,
            "flops": 4 * D * hq * pairs}


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    p, op, ps, hkv = st["plan_host"], case["op"], case["page"], case["hkv"]
    if op == "write":
        q, k, v = _prep(st, torch.float64)
        codes, scales = (x.double() for x in _codes(st))
        for i, y in enumerate((k, v)):
            c, s = _quantise(y)
            codes[0, st["tpage"], i, :, st["toff"]] = c.double()
            scales[0, st["tpage"], i, :, st["toff"]] = s.double()
        return {"q": q, "codes": codes, "scales": scales}
    ids = st["ids"].long()
    if op == "read":
        pool = st["pool"].double()
        for r in range(case["reqs"]):
            n = int(p["keys"][r])
            pages = ids[int(p["pg_indptr"][r]):int(p["pg_indptr"][r + 1])]
            for a in range(0, len(pages), 256):
                part = pages[a:a + 256]
                y = _values(st["codes"][:, part].view(torch.float8_e4m3fn),
                            st["scales"][:, part].view(torch.float8_e8m0fnu), torch.float64)
                live = (a * ps + torch.arange(len(part) * ps, device="cuda") < n).reshape(-1, ps)
                pool[:, part] = torch.where(live[None, :, None, None, :, None], y, pool[:, part])
        return {"pool": pool}
    T, hq, D = st["q"].shape
    G = hq // hkv
    out = torch.zeros((T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, hq), dtype=torch.float64, device="cuda")
    for r in range(case["reqs"]):
        n, t0, t1 = int(p["keys"][r]), int(p["qo_indptr"][r]), int(p["qo_indptr"][r + 1])
        pages = ids[int(p["pg_indptr"][r]):int(p["pg_indptr"][r + 1])]
        if "pool" in st:
            kv = st["pool"][0, pages].double()
        else:
            kv = _values(st["codes"][0, pages].view(torch.float8_e4m3fn),
                         st["scales"][0, pages].view(torch.float8_e8m0fnu), torch.float64)
        position = int(p["start"][r]) + torch.arange(t1 - t0, device="cuda")[:, None]
        where = int(p["kv_start"][r]) + torch.arange(n, device="cuda")[None, :]
        hidden = where > position
        if case["window"] >= 0:
            hidden |= (position - where > case["window"]) & (where >= case["sinks"])
        for g in range(hkv):
            k, v = (kv[:, i, g].reshape(-1, D)[:n] for i in (0, 1))
            for h in range(g * G, (g + 1) * G):
                z = (st["q"][t0:t1, h].double() @ k.T).masked_fill(hidden, float("-inf"))
                norm = torch.logsumexp(z, 1)
                out[t0:t1, h] = torch.exp(z - norm[:, None]) @ v
                lse[t0:t1, h] = norm
    return {"out": out, "lse": lse}
