"""Attention for batches that share prefixes, on bf16 and 8-bit pools (GPU), against the plain 64-bit
reference of bounded_ref.py, request by request over all its keys.

Tolerance: bounded_ref's, with one more rounding: the part of a row's own keys is rounded to bf16
before the join, by at most half a step, 2^-8 of it, so 2^-8 * A more (A = sum_j w_j |v_j|)."""
import numpy as np
import pytest
import torch

from bounded_ref import Case
from paged_sliding_window_qkv_gb300 import pg
from q8_ref import Q8Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def parts():
    """The tests' batches are small: what is tested here is the prefixes' parts, unless a test says otherwise."""
    assert pg.pg_test_shared_form(1) == pg.PG_OK
    yield
    assert pg.pg_test_shared_form(0) == pg.PG_OK


HEADS = {256: [(16, 8), (8, 8), (16, 1), (8, 2)], 512: [(16, 1), (8, 1), (4, 2), (2, 2)]}


def ok():
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK


def shared(base):
    class Shared(base):
        """groups: (requests, prefix pages) in order; own: keys of each request before the step."""

        def __init__(self, D, hq, hkv, qo, own, groups, ps=16, seed=0, **kw):
            self.group_indptr = np.concatenate([[0], np.cumsum([g for g, _ in groups])])
            self.prefix = np.asarray([p * ps for _, p in groups], np.int64)
            of = np.repeat(np.arange(len(groups)), [g for g, _ in groups])
            super().__init__(D, hq, hkv, qo, np.asarray(own) + self.prefix[of], ps=ps, seed=seed, **kw)
            for r in range(len(self.qo)):
                k, first = int(self.prefix[of[r]]) // ps, int(self.group_indptr[of[r]])
                a, b = int(self.pg_indptr[r]), int(self.pg_indptr[first])
                self.ids[a:a + k] = self.ids[b:b + k]

        def replan(self, plan=None, **kw):
            a = dict(num_req=len(self.qo), qo_indptr=self.qo_indptr, kv_page_indptr=self.pg_indptr,
                     page_ids=self.ids, last_page_len=self.last, start_pos=self.start,
                     num_groups=len(self.prefix), group_indptr=self.group_indptr, prefix_len=self.prefix,
                     num_qo_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.D, page_size=self.ps) | kw
            return pg.pg_plan_paged_shared(plan, stream=self.stream, **a)

        def build(self):
            rc, self.plan = self.replan()
            pg.check(rc, "shared plan")
            self.upload()
            return self

        def upload(self):
            super().upload()
            q8 = isinstance(self, Q8Case)
            self.ws_bytes = (pg.pg_shared_q8_workspace_bytes if q8 else pg.pg_shared_workspace_bytes)(self.plan)
            self.ws = torch.full((self.ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")

        def attend(self, scale=1.0, lse=True):
            f, pool = (pg.pg_attn_paged_shared_q8, self.q8) if isinstance(self, Q8Case) else \
                (pg.pg_attn_paged_shared, self.desc)
            pg.check(f(self.plan, pool, self.layer, self.q, self.out, self.lse if lse else None, scale,
                       self.ws, self.ws_bytes, self.stream), "shared")

        def check(self, what="", scale=1.0):
            out, lse, m, p, wabs = self.reference(-1, 0, scale)
            self.ref = (out, lse, m, p, 2 * wabs)
            self.check_attention(what)

    return Shared


Bf16, Q8 = shared(Case), shared(Q8Case)
KINDS = [Bf16, Q8]


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("qo,own,groups", [
    ([1] * 6, [0, 3, 15, 16, 100, 333], [(6, 40)]),
    ([1] * 7, [5, 0, 0, 64, 1, 300, 17], [(1, 9), (3, 1), (2, 33), (1, 0)]),
    ([1], [0], [(1, 1)]),
    ([1] * 40, list(range(40)), [(20, 13), (20, 70)]),
    ([5, 130, 1, 64], [0, 7, 200, 0], [(3, 25), (1, 4)]),
    ([300, 2, 17], [0, 0, 40], [(3, 64)]),
    ([3, 1], [9, 0], [(1, 0), (1, 0)]),
])
def test_shared_prefixes(kind, D, qo, own, groups):
    hq, hkv = HEADS[D][0]
    c = kind(D, hq, hkv, qo, own, groups, seed=len(qo)).build()
    c.attend()
    ok()
    c.check()
    c.close()


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
@pytest.mark.parametrize("D,hq,hkv", [(d, *h) for d in (256, 512) for h in HEADS[d]])
def test_head_groups_and_layers(kind, D, hq, hkv):
    for qo in ([1, 1, 1], [20, 3, 70]):
        c = kind(D, hq, hkv, qo, [10, 0, 99], [(2, 21), (1, 3)], seed=hq + hkv, layers=2, layer=1).build()
        c.attend()
        ok()
        c.check(f"{qo}")
        c.close()


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("ps", [8, 32, 128])
def test_page_sizes(kind, D, ps):
    hq, hkv = HEADS[D][0]
    for qo in ([1, 1, 1], [33, 1, 80]):
        c = kind(D, hq, hkv, qo, [10, 0, 77], [(3, 5)], ps=ps, seed=ps).build()
        c.attend()
        ok()
        c.check(f"{qo}")
        c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("scale", [0.0, -1.0, 0.25])
def test_scales_and_no_lse(D, scale):
    hq, hkv = HEADS[D][0]
    for qo in ([1, 1], [90, 4]):
        c = Bf16(D, hq, hkv, qo, [30, 2], [(2, 30)], seed=3).build()
        c.attend(scale)
        ok()
        c.check(scale=scale)
        first = c.out.clone()
        c.out.fill_(float("nan"))
        c.attend(scale, lse=False)
        ok()
        assert torch.equal(c.out, first)  # the parts and their order are fixed
        c.close()


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
def test_a_long_prefix_is_cut_into_many_parts(kind):
    for D in (256, 512):
        hq, hkv = HEADS[D][0]
        c = kind(D, hq, hkv, [1, 1], [3, 40], [(2, 500)], seed=6).build()
        c.attend()
        ok()
        c.check()
        c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_a_prefix_that_outweighs_the_own_keys_and_the_other_way(D):
    """Scores of the two parts far apart: one part's weights underflow beside the other's."""
    hq, hkv = HEADS[D][0]
    for sign in (1.0, -1.0):
        c = Bf16(D, hq, hkv, [1, 1, 30], [60, 20, 50], [(3, 12)], seed=9)
        pre = c.ids[:12].astype(int)
        c.q_cpu[:] = torch.abs(c.q_cpu)
        c.pool_cpu[0, pre, 0] = torch.abs(c.pool_cpu[0, pre, 0]) * sign * 4
        c.build()
        c.attend()
        ok()
        c.check(f"{sign}")
        c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_the_plan_serves_the_other_entries(D):
    """A shared plan is its plain plan everywhere else: attention of both entries agrees, and prep
    writes the rows that the plain plan's writes."""
    hq, hkv = HEADS[D][0]
    c = Bf16(D, hq, hkv, [1, 1, 1], [10, 0, 99], [(2, 21), (1, 3)], seed=5).build()
    ws = torch.empty(max(16, pg.pg_sink_workspace_bytes(c.plan)), dtype=torch.uint8, device="cuda")
    pg.check(pg.pg_attn_paged_sink(c.plan, c.desc, 0, c.q, c.out, c.lse, -1, 0, 1.0, ws, ws.numel()))
    ok()
    c.check("sink entry")
    c.close()


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("D", [256, 512])
def test_captured_call_follows_its_plan(kind, decode, D):
    """Replayed after an update to as many groups, requests, tokens and pages, spread otherwise."""
    hq, hkv = HEADS[D][0]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        qo = [1, 1, 1, 1] if decode else [40, 1, 9, 2]
        a = kind(D, hq, hkv, qo, [0, 15, 40, 8], [(2, 30), (2, 2)], seed=1, stream=stream).build()
        extra = 64 * 4 * hkv * 16 * D  # room for more pages in prefixes
        a.ws_bytes += extra
        a.ws = torch.full((a.ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        a.attend()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            a.attend()
        total = len(a.ids)
        for groups, seed in (([(1, 3), (3, 14)], 2), ([(3, 0), (1, 40)], 3), ([(2, 0), (2, 0)], 4)):
            own = [0, 15, 40, 8]
            need = sum(r * p for r, p in groups)
            qb = qo if decode else [2, 9, 1, 40]
            left = total - need - sum(-(-(o + q) // 16) for o, q in zip(own, qb))
            own[0] += 16 * left
            b = kind(D, hq, hkv, qb, own, groups, seed=seed, stream=stream)
            assert left >= 0 and len(b.ids) == total and b.P == a.P, (left, len(b.ids), total)
            rc, _ = b.replan(a.plan)
            pg.check(rc)
            a.q.copy_(b.q_cpu)
            if kind is Q8:
                a.codes.copy_(b.codes_cpu)
                a.scales.copy_(b.scales_cpu)
            else:
                a.pool.copy_(b.pool_cpu)
            a.out.fill_(float("nan"))
            a.ws.fill_(0xFF)
            g.replay()
            stream.synchronize()
            assert pg.pg_device_status(stream) == pg.PG_OK
            b.out, b.lse = a.out, a.lse
            b.check(f"{groups}")
    a.close()


def test_plans_change_kind_in_place():
    c = Bf16(512, 16, 1, [1, 1], [10, 20], [(2, 4)], seed=2).build()
    rc, _ = pg.pg_plan_paged_prefill(c.plan, 2, c.qo_indptr, c.pg_indptr, c.ids, c.last, c.start, 16, 1, 512, 16)
    pg.check(rc)
    assert pg.pg_shared_workspace_bytes(c.plan) == 0
    assert pg.pg_attn_paged_shared(c.plan, c.desc, 0, c.q, c.out, None, 1.0, c.ws, c.ws_bytes) == \
        pg.PG_ERR_PLAN_MISMATCH
    rc, _ = c.replan(c.plan)
    pg.check(rc)
    c.attend()
    ok()
    c.check()
    c.close()


def test_a_refused_update_leaves_the_plan_as_it_was():
    c = Bf16(256, 16, 8, [1, 1, 1], [10, 20, 0], [(2, 4), (1, 2)], seed=2).build()
    rc, _ = c.replan(c.plan, prefix_len=[64, 40])
    assert rc == pg.PG_ERR_COVERAGE
    c.attend()
    ok()
    c.check()
    c.close()


def test_refusals_launch_nothing():
    for c in (Bf16(512, 16, 1, [1, 1], [10, 20], [(2, 4)], seed=2).build(),
              Q8(512, 16, 1, [1, 1], [10, 20], [(2, 4)], seed=2).build()):
        torch.cuda.synchronize()
        before = pg.pg_launch_count()
        q8 = isinstance(c, Q8Case)
        f, pool = (pg.pg_attn_paged_shared_q8, c.q8) if q8 else (pg.pg_attn_paged_shared, c.desc)

        def call(want, plan=c.plan, pool=pool, layer=0, q=c.q, out=c.out, lse=c.lse, scale=1.0, ws=c.ws,
                 n=c.ws_bytes, stream=None):
            assert f(plan, pool, layer, q, out, lse, scale, ws, n, stream) == want

        call(pg.PG_ERR_ARG, plan=None)
        call(pg.PG_ERR_ARG, pool=None)
        call(pg.PG_ERR_ARG, q=None)
        call(pg.PG_ERR_ARG, out=None)
        call(pg.PG_ERR_LAYER, layer=3)
        call(pg.PG_ERR_NONFINITE, scale=float("inf"))
        call(pg.PG_ERR_WORKSPACE, ws=None)
        call(pg.PG_ERR_WORKSPACE, n=c.ws_bytes - 1)
        call(pg.PG_ERR_ALIGN, ws=c.ws.data_ptr() + 8)
        call(pg.PG_ERR_ALIGN, out=c.out.data_ptr() + 16)
        call(pg.PG_ERR_ALIGN, lse=c.lse.data_ptr() + 1)
        call(pg.PG_ERR_STREAM, stream=torch.cuda.Stream())
        assert pg.pg_launch_count() == before
        assert torch.isnan(c.out).all()
        ok()
        c.close()


def test_empty_batch():
    rc, plan = pg.pg_plan_paged_shared(None, 0, [0], [0], [], [], [], 0, [0], [], 16, 1, 512, 16)
    pg.check(rc)
    c = Bf16(512, 16, 1, [1], [0], [(1, 0)]).build()
    before = pg.pg_launch_count()
    assert pg.pg_shared_workspace_bytes(plan) == 0
    pg.check(pg.pg_attn_paged_shared(plan, c.desc, 0, None, None, None, 1.0))
    assert pg.pg_launch_count() == before
    plan.close()
    c.close()


# ------------------------------------------------------------------ a run together
@pytest.mark.parametrize("D", [256, 512])
def test_requests_fork_from_a_prompt_on_an_8_bit_cache(D):
    """A document is read once into an 8-bit pool; three requests go on from its pages: their own prompts,
    then tokens, each step written (prep) and attended (shared) on one plan updated in place. At the end
    the cache is read back and the last step's attention repeated on the bf16 pool."""
    from q8_ref import values
    hq, hkv = HEADS[D][0]
    ps, doc, R = 16, 160, 3
    g = np.random.Generator(np.random.PCG64(50 + D))
    P = doc // ps + R * 4
    codes = torch.full((1, P, 2, hkv, ps, D), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, P, 2, hkv, ps), 0xFF, dtype=torch.uint8, device="cuda")
    q8 = pg.q8_descriptor(codes, scales)
    order = g.permutation(P).astype(np.int32)
    prefix, rest = order[:doc // ps], order[doc // ps:]
    f = (1e4 if D == 256 else 1e6) ** (-2.0 * np.arange(D // 2) / D)
    a = np.arange(256)[:, None] * f
    cos, sin = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (np.cos(a), np.sin(a)))
    w = torch.from_numpy((0.2 * (1 + 0.1 * g.standard_normal((2, D)))).astype(np.float32)).to(torch.bfloat16).cuda()
    plan = None

    def step(groups, pre, qo, start, lists):
        nonlocal plan
        qo, start = np.asarray(qo), np.asarray(start)
        n = start + qo
        npg = -(-n // ps)
        ids = np.concatenate([p[:k] for p, k in zip(lists, npg)])
        kw = [len(qo), np.concatenate([[0], np.cumsum(qo)]), np.concatenate([[0], np.cumsum(npg)]), ids,
              n - (npg - 1) * ps, start, len(groups), np.concatenate([[0], np.cumsum(groups)]), pre, hq, hkv, D, ps]
        rc, plan = pg.pg_plan_paged_shared(plan, *kw)
        pg.check(rc, "plan")
        T = int(qo.sum())
        cols = (hq + (2 if D == 256 else 1) * hkv) * D
        raw = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).to(torch.bfloat16).cuda()
        q = torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        pg.check(pg.pg_prep_paged_q8(plan, q8, 0, raw, cols, raw[:, hq * D:], cols,
                                     raw[:, (hq + hkv) * D:] if D == 256 else None, cols, w[0], w[1], 1e-6, cos, sin,
                                     256, q), "prep")
        out = torch.full_like(q, float("nan"))
        lse = torch.full((T, hq), float("nan"), device="cuda")
        ws = torch.full((pg.pg_shared_q8_workspace_bytes(plan),), 0xFF, dtype=torch.uint8, device="cuda")
        pg.check(pg.pg_attn_paged_shared_q8(plan, q8, 0, q, out, lse, 1.0, ws, ws.numel()), "attention")
        ok()
        rows = values(codes.cpu()[0], scales.cpu()[0]).numpy()  # [P, kv, head, slot, D]
        check(q, out, lse, qo, start, lists, rows)
        return q, out, lse, qo, start, rows

    def check(q, out, lse, qo, start, lists, rows):
        qd, got, gl = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
        t = 0
        for r in range(len(qo)):
            n = int(start[r] + qo[r])
            kv = rows[np.asarray(lists[r])].transpose(0, 3, 1, 2, 4).reshape(-1, 2, hkv, D)[:n]
            for i in range(int(qo[r])):
                m = int(start[r]) + i + 1
                for h in range(hq):
                    k, v = kv[:m, 0, h * hkv // hq], kv[:m, 1, h * hkv // hq]
                    z = k @ qd[t, h]
                    top = z.max()
                    p = np.exp(z - top)
                    ref, mag = p @ v / p.sum(), p @ np.abs(v) / p.sum()
                    # scores of up to D products of about unit size in all; bounded_ref's rule with the
                    # own keys' rounding and q8_ref's floor of small weights
                    e = 2 * (16 * 2.0 ** -23 * float(np.abs(qd[t, h]) @ np.abs(k).max(0)) + 2.0 ** -21 * 70) + 2.0 ** -20
                    lim = 2.0 ** -8 * (2 * mag + np.abs(ref)) + e * mag + 2.0 ** -21 * m * np.abs(v).max()
                    assert (np.abs(got[t, h] - ref) <= lim).all(), (r, i, h)
                    assert abs(gl[t, h] - (top + np.log(p.sum()))) <= e + 2.0 ** -20, (r, i, h)
                t += 1

    step([1], [0], [doc], [0], [prefix])
    lists = [np.concatenate([prefix, rest[r::R]]) for r in range(R)]
    lens = np.array([doc, doc, doc])
    before = codes[0, torch.from_numpy(prefix).long().cuda()].clone()
    for qo in ([20, 3, 7], [1, 1, 1], [1, 1, 1], [2, 1, 1]):
        last = step([R], [doc], qo, lens, lists)
        lens = lens + np.asarray(qo)
    assert torch.equal(codes[0, torch.from_numpy(prefix).long().cuda()], before)  # no step wrote the document
    q, out, lse, qo, start, rows = last
    bf = torch.zeros((1, P, 2, hkv, ps, D), dtype=torch.bfloat16, device="cuda")
    pg.check(pg.pg_kv_dequantize(plan, q8, pg.pool_descriptor(bf), 0, 1))
    ws = torch.empty(pg.pg_shared_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    pg.check(pg.pg_attn_paged_shared(plan, pg.pool_descriptor(bf), 0, q, out, lse, 1.0, ws, ws.numel()))
    ok()
    check(q, out, lse, qo, start, lists, rows)
    plan.close()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """The parts' kernel withholds an arrival: the call returns, the status word says so, and the context
    stays usable."""
    c = Bf16(512, 16, 1, [1, 1], [10, 20], [(2, 40)], seed=2).build()
    c.attend()
    ok()
    try:
        assert pg.pg_test_bounded_wait(1, 20_000_000) == pg.PG_OK
        c.attend()
        torch.cuda.synchronize()
        assert pg.pg_device_status() == pg.PG_ERR_DEVICE_TIMEOUT
    finally:
        assert pg.pg_test_bounded_wait(0) == pg.PG_OK
    c.out.fill_(float("nan"))
    c.attend()
    ok()
    c.check()
    c.close()


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("qo,own,groups", [
    ([1] * 7, [5, 0, 0, 64, 1, 300, 17], [(1, 9), (3, 1), (2, 33), (1, 0)]),
    ([5, 130, 1, 64], [0, 7, 200, 0], [(3, 25), (1, 4)]),
])
def test_both_forms_and_the_choice(kind, D, qo, own, groups):
    """The plain walk is the entry without prefixes, to the bit; the choice is one of the two forms."""
    hq, hkv = HEADS[D][0]
    got = {}
    for form in (2, 1, 0):
        pg.check(pg.pg_test_shared_form(form))
        c = kind(D, hq, hkv, qo, own, groups, seed=21).build()
        c.attend()
        ok()
        c.check(f"form {form}")
        got[form] = c.out.clone(), c.lse.clone()
        if form == 2:
            q8 = isinstance(c, Q8Case)
            nbytes, f, pool = (pg.pg_q8_workspace_bytes, pg.pg_attn_paged_q8, c.q8) if q8 else \
                (pg.pg_sink_workspace_bytes, pg.pg_attn_paged_sink, c.desc)
            ws = torch.empty(max(16, nbytes(c.plan)), dtype=torch.uint8, device="cuda")
            pg.check(f(c.plan, pool, 0, c.q, c.out, c.lse, -1, 0, 1.0, ws, ws.numel()))
            ok()
            assert torch.equal(c.out, got[2][0]) and torch.equal(c.lse, got[2][1])
        c.close()
    assert any(torch.equal(got[0][0], got[f][0]) and torch.equal(got[0][1], got[f][1]) for f in (1, 2))


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
@pytest.mark.parametrize("qo,own,groups,plain", [
    ([1], [100], [(1, 8)], True),             # nothing to share
    ([1] * 3, [10, 0, 99], [(3, 0)], True),   # no prefix
    ([1] * 64, [20] * 64, [(64, 256)], False),
    ([256] * 8, [0] * 8, [(8, 32)], False),   # (steps of more tokens take the parts)
    ([2] * 32, [64] * 32, [(32, 256)], False),
])
def test_the_plan_chooses_by_size(kind, qo, own, groups, plain):
    """Parts are a kernel of their own (and a read-back, and a join behind prompts): told by the launches."""
    pg.check(pg.pg_test_shared_form(0))
    c = kind(512, 16, 1, qo, own, groups, seed=5).build()

    def launches():
        torch.cuda.synchronize()
        n = pg.pg_launch_count()
        c.attend()
        ok()
        return pg.pg_launch_count() - n

    chosen = launches()
    c.check()
    decode, q8 = max(qo) == 1, isinstance(c, Q8Case)
    assert chosen == (2 if decode else 2 if q8 else 1) + (0 if plain else 1 + q8 + (not decode))
    c.close()


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "q8"])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("D", [256, 512])
def test_a_captured_plain_walk_follows_its_plan(kind, decode, D):
    """Captured in the plain form, replayed under a plan whose own calls would take parts."""
    hq, hkv = HEADS[D][0]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        pg.check(pg.pg_test_shared_form(2))
        qo = [1, 1, 1, 1] if decode else [40, 1, 9, 2]
        a = kind(D, hq, hkv, qo, [0, 15, 40, 8], [(2, 30), (2, 2)], seed=1, stream=stream).build()
        a.attend()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            a.attend()
        pg.check(pg.pg_test_shared_form(1))
        total, own = len(a.ids), [0, 15, 40, 8]
        qb = qo if decode else [2, 9, 1, 40]
        own[0] += 16 * (total - 45 - sum(-(-(o + q) // 16) for o, q in zip(own, qb)))
        b = kind(D, hq, hkv, qb, own, [(1, 3), (3, 14)], seed=2, stream=stream)
        assert len(b.ids) == total and b.P == a.P
        pg.check(b.replan(a.plan)[0])
        a.q.copy_(b.q_cpu)
        if kind is Q8:
            a.codes.copy_(b.codes_cpu)
            a.scales.copy_(b.scales_cpu)
        else:
            a.pool.copy_(b.pool_cpu)
        a.out.fill_(float("nan"))
        a.ws.fill_(0xFF)
        g.replay()
        stream.synchronize()
        assert pg.pg_device_status(stream) == pg.PG_OK
        b.out, b.lse = a.out, a.lse
        b.check()
    a.close()
