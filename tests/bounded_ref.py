"""Plain 64-bit restatement of the bounded-cache operators, and the set-up their tests share.

Tolerances (derived before any run). A score is a sum of D exact bf16 products in fp32: its error
is at most 16 * 2^-23 * sum_d |q_d k_d| times the scale (fp32 accumulation in 16-term steps, each
off by at most a step of the largest partial sum). With d that bound over the case's rows plus the
rounding of score * log2(e) against the row's reference and normaliser (2^-21 * (|lse| + 64) with
the 2^64 headroom):
  weight   relative error  e = 2 d + 2^-20          (2^x is good to 2^-22)
  out      2^-8 * A + 2^-8 * |ref| + e * A, A = sum_j w_j |v_j|: the bf16 rounding of each
           weight (half a step, 2^-8 of it), of the output, and the weights' own error
  lse      e + 2^-22 * |lse|
  mass     2 e * ref + 2^-22 * (|old| + ref): weights and their normaliser, fp32 sums
"""
from __future__ import annotations

import numpy as np
import torch

from paged_sliding_window_qkv_gb300 import pg


class Case:
    """One batch on the GPU and its 64-bit reference."""

    def __init__(self, D, hq, hkv, qo, start, ps=16, evicted=0, held=None, layers=1, layer=0,
                 gain=2.0, seed=0, stream=None, spare=3):
        g = np.random.Generator(np.random.PCG64(seed))
        self.D, self.hq, self.hkv, self.ps, self.layer, self.layers = D, hq, hkv, ps, layer, layers
        self.qo = np.asarray(qo, np.int64)
        self.start = np.asarray(start, np.int64)
        R = len(self.qo)
        self.ks = np.broadcast_to(np.asarray(evicted, np.int64), (R,)).copy()
        # keys held: up to the step's end unless a shorter segment is asked for
        self.n = self.start + self.qo - self.ks if held is None else np.asarray(held, np.int64)
        npg = (self.n + ps - 1) // ps
        self.pg_indptr = np.concatenate([[0], np.cumsum(npg)])
        self.qo_indptr = np.concatenate([[0], np.cumsum(self.qo)])
        need = int(self.pg_indptr[-1])
        self.P = need + spare
        self.ids = g.permutation(self.P)[:need].astype(np.int32)
        self.last = (self.n - (npg - 1) * ps).astype(np.int32)
        t = lambda shape, std=1.0: torch.from_numpy(  # noqa: E731
            (g.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)
        self.pool_cpu = t((layers, self.P, 2, hkv, ps, D))
        self.q_cpu = t((int(self.qo_indptr[-1]), hq, D), gain / np.sqrt(D))
        self.mass_cpu = torch.from_numpy(g.exponential(1.0, (layers, self.P, hkv, ps)).astype(np.float32))
        self.pos_cpu = torch.full((layers, self.P, hkv, ps), -7, dtype=torch.int32)
        self.stream = stream
        self.plan = None

    # ---- device side
    def build(self):
        rc, self.plan = pg.pg_plan_paged_segment(
            None, len(self.qo), self.qo_indptr, self.pg_indptr, self.ids, self.last, self.ks,
            self.start, self.hq, self.hkv, self.D, self.ps, self.stream)
        pg.check(rc, "plan")
        self.upload()
        return self

    def upload(self):
        self.pool, self.q = self.pool_cpu.cuda(), self.q_cpu.cuda()
        self.mass, self.pos = self.mass_cpu.cuda(), self.pos_cpu.cuda()
        self.desc = pg.pool_descriptor(self.pool)
        self.stats = pg.stats_descriptor(self.mass, self.pos)
        T = self.q.shape[0]
        # rows are written whole: what is not shows as NaN
        self.out = torch.full((T, self.hq, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, self.hq), float("nan"), device="cuda")
        n = max(pg.pg_workspace_bytes(self.plan), pg.pg_mass_workspace_bytes(self.plan), 16)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def sink(self, window, sinks, scale=1.0, lse=True):
        pg.check(pg.pg_attn_paged_sink(self.plan, self.desc, self.layer, self.q, self.out,
                                       self.lse if lse else None, window, sinks, scale, self.ws,
                                       pg.pg_workspace_bytes(self.plan), self.stream), "sink")

    def weigh(self, window=-1, sinks=0, scale=1.0):
        pg.check(pg.pg_attn_paged_mass(self.plan, self.desc, self.layer, self.q, self.out, self.lse,
                                       self.stats, window, sinks, scale, self.ws,
                                       pg.pg_mass_workspace_bytes(self.plan), self.stream), "mass")

    def close(self):
        self.plan.close()

    # ---- 64 bits
    def rows_of(self, r):
        """(page, offset) of the request's slots."""
        s = np.arange(self.n[r])
        return self.ids[self.pg_indptr[r] + s // self.ps].astype(np.int64), s % self.ps

    def reference(self, window, sinks, scale=1.0, mass=None, pos=None):
        T = self.q_cpu.shape[0]
        G = self.hq // self.hkv
        out, lse = np.zeros((T, self.hq, self.D)), np.full((T, self.hq), -np.inf)
        wabs = np.zeros((T, self.hq, self.D))
        mass = (self.mass_cpu if mass is None else mass).double().numpy().copy()
        pos = (self.pos_cpu if pos is None else pos).numpy().copy()
        pool, q = self.pool_cpu[self.layer].double().numpy(), self.q_cpu.double().numpy()
        err = 0.0
        self.touched = np.zeros(mass.shape, bool)
        for r in range(len(self.qo)):
            page, off = self.rows_of(r)
            j = self.ks[r] + np.arange(self.n[r])
            t = slice(self.qo_indptr[r], self.qo_indptr[r + 1])
            p = (self.start[r] + np.arange(self.qo[r]))[:, None]
            vis = j[None, :] <= p
            if window >= 0:
                vis &= (p - j <= window) | (j < sinks)[None, :]
            for g in range(self.hkv):
                k, v = pool[page, 0, g, off], pool[page, 1, g, off]
                add = np.zeros(self.n[r])
                for h in range(g * G, (g + 1) * G):
                    z = np.where(vis, scale * (q[t, h] @ np.where(np.isfinite(k), k, 0).T), -np.inf)
                    live = vis.any(1)
                    m = np.where(live, z.max(1, initial=-np.inf), 0.0)
                    w = np.exp(z - m[:, None])
                    den = w.sum(1)
                    w = w / np.where(live, den, 1.0)[:, None]
                    vv = np.where(np.isfinite(v), v, 0)
                    out[t, h], wabs[t, h] = w @ vv, w @ np.abs(vv)
                    with np.errstate(divide="ignore"):
                        lse[t, h] = np.where(live, m + np.log(den), -np.inf)
                    add += w.sum(0)
                    err = max(err, float((np.abs(q[t, h]) @ np.abs(np.where(np.isfinite(k), k, 0)).T).max(initial=0)))
                new = j >= self.start[r]
                seen = vis.any(0)
                at = (self.layer, page, g, off)
                mass[at] = np.where(seen, np.where(new, 0, mass[at]) + add, mass[at])
                pos[at] = np.where(new & seen, j, pos[at])
                self.touched[self.layer, page[seen], g, off[seen]] = True
        fin = lse[np.isfinite(lse)]
        big = float(np.abs(fin).max()) if fin.size else 0.0
        self.e = 2 * (16 * 2.0 ** -23 * err * abs(scale) + 2.0 ** -21 * (big + 64)) + 2.0 ** -20
        self.ref = (out, lse, mass, pos, wabs)
        return self.ref

    def check_attention(self, what="", rows=None):
        out, lse, _, _, wabs = self.ref
        rows = slice(None) if rows is None else rows
        got = self.out.double().cpu().numpy()[rows]
        tol = 2.0 ** -8 * (wabs + np.abs(out)) + self.e * wabs + 1e-30
        bad = ~(np.abs(got - out[rows]) <= tol[rows])
        assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist())
        gl, rl = self.lse.double().cpu().numpy()[rows], lse[rows]
        none = np.isneginf(rl)
        assert (np.isneginf(gl) == none).all(), (what, "rows without keys")
        d = np.abs(np.where(none, 0, gl) - np.where(none, 0, rl))
        lim = self.e + 2.0 ** -22 * np.where(none, 0, np.abs(rl))
        assert (d <= lim).all(), (what, "lse", float((d - lim).max()))

    def check_mass(self, what="", old=None):
        _, _, mass, pos, _ = self.ref
        old = (self.mass_cpu if old is None else old).double().numpy()
        got = self.mass.double().cpu().numpy()
        assert (self.pos.cpu().numpy() == pos).all(), (what, "positions")
        same = ~self.touched
        assert (got[same] == old[same]).all(), (what, "statistics of other keys changed")
        lim = 2 * self.e * mass + 2.0 ** -22 * (np.abs(old) + mass) + 1e-30
        bad = ~(np.abs(got - mass) <= lim) & ~same
        assert not bad.any(), (what, "mass", int(bad.sum()), float((np.abs(got - mass) / lim).max()))


def select_reference(case, budget, sinks, recent, mass, pos, layers):
    """The source slot of every kept slot, by sorting."""
    R, H = len(case.qo), case.hkv
    src = np.full((len(layers), R, H, budget), -1, np.int32)
    for i, layer in enumerate(layers):
        for r in range(R):
            page, off = case.rows_of(r)
            n, end = int(case.n[r]), int(case.start[r] + case.qo[r])
            keep = min(n, budget)
            for g in range(H):
                m = mass[layer][page, g, off].astype(np.float64)
                m = np.where(np.isnan(m), -np.inf, m)
                p = pos[layer][page, g, off].astype(np.int64)
                first = (p < sinks) | (p >= end - recent)
                order = sorted(range(n), key=lambda s: (not first[s], 0 if first[s] else -m[s], s))
                kept = np.zeros(n, bool)
                kept[order[:keep]] = True
                move = [s for s in range(keep, n) if kept[s]]
                hole = [s for s in range(keep) if not kept[s]]
                row = np.arange(keep)
                row[hole] = move
                src[i, r, g, :keep] = row
    return src


def apply_reference(case, src, layers, pool, mass, pos):
    """Pool, mass and pos after the moves (numpy copies)."""
    pool, mass, pos = pool.clone(), mass.clone(), pos.clone()
    for i, layer in enumerate(layers):
        for r in range(len(case.qo)):
            page, off = case.rows_of(r)
            for g in range(case.hkv):
                for s, f in enumerate(src[i, r, g]):
                    if f >= 0 and f != s:
                        pool[layer, page[s], :, g, off[s]] = pool[layer, page[f], :, g, off[f]]
                        mass[layer, page[s], g, off[s]] = mass[layer, page[f], g, off[f]]
                        pos[layer, page[s], g, off[s]] = pos[layer, page[f], g, off[f]]
    return pool, mass, pos
