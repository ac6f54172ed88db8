"""How the bounded-cache operators are called (GPU): refusals, streams, captured graphs, grown
plans, guarded workspaces, odd alignments, large batches and far offsets, and a serving loop that
scores, evicts and goes on through the page allocator. References and tolerances: bounded_ref.py."""
import numpy as np
import pytest
import torch

from bounded_ref import Case, apply_reference, select_reference
from paged_sliding_window_qkv_gb300 import pg

pytestmark = pytest.mark.gpu
HQ = {256: (16, 8), 512: (16, 1)}


def ok():
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK


def small(D=256, qo=(3, 1), start=(40, 7), **kw):
    return Case(D, *HQ[D], list(qo), list(start), **kw)


# ------------------------------------------------------------------ refusals
def test_attention_refusals():
    c = small(layers=2).build()
    n = pg.pg_workspace_bytes(c.plan)
    launched = pg.pg_launch_count()

    def sink(plan=c.plan, pool=c.desc, layer=0, q=c.q, out=c.out, lse=c.lse, w=5, s=4, scale=1.0,
             ws=c.ws, nb=n, stream=None):
        return pg.pg_attn_paged_sink(plan, pool, layer, q, out, lse, w, s, scale, ws, nb, stream)

    assert sink(w=-2) == pg.PG_ERR_WINDOW
    assert sink(s=-1) == pg.PG_ERR_WINDOW
    assert sink(scale=float("nan")) == pg.PG_ERR_NONFINITE
    assert sink(layer=2) == pg.PG_ERR_LAYER and sink(layer=-1) == pg.PG_ERR_LAYER
    assert sink(q=None) == pg.PG_ERR_ARG and sink(out=None) == pg.PG_ERR_ARG
    assert sink(q=c.q.data_ptr() + 16) == pg.PG_ERR_ALIGN
    assert sink(lse=c.lse.data_ptr() + 2) == pg.PG_ERR_ALIGN
    assert sink(stream=torch.cuda.Stream()) == pg.PG_ERR_STREAM
    assert sink(pool=pg.pool_descriptor(c.pool, num_pages=1)) == pg.PG_ERR_LAYOUT
    assert sink(pool=pg.pool_descriptor(c.pool, head_dim=512)) == pg.PG_ERR_LAYOUT

    def mass(stats=c.stats, lse=c.lse, ws=c.ws, nb=pg.pg_mass_workspace_bytes(c.plan)):
        return pg.pg_attn_paged_mass(c.plan, c.desc, 0, c.q, c.out, lse, stats, -1, 0, 1.0, ws, nb)

    assert mass(stats=None) == pg.PG_ERR_ARG
    assert mass(lse=None) == pg.PG_ERR_ARG
    assert mass(stats=pg.stats_descriptor(c.mass, c.pos, num_pages=3)) == pg.PG_ERR_LAYOUT
    assert mass(stats=pg.stats_descriptor(c.mass, c.pos, capacity=7)) == pg.PG_ERR_LAYOUT
    assert mass(stats=pg.stats_descriptor(c.mass[:1], c.pos[:1])) == pg.PG_ERR_LAYOUT
    assert mass(stats=pg.stats_descriptor(c.mass, c.pos, mass=c.mass.data_ptr() + 1)) == pg.PG_ERR_ALIGN
    assert mass(ws=None) == pg.PG_ERR_WORKSPACE
    assert mass(nb=pg.pg_mass_workspace_bytes(c.plan) - 1) == pg.PG_ERR_WORKSPACE
    assert mass(ws=c.ws.data_ptr() + 4) == pg.PG_ERR_ALIGN
    assert pg.pg_launch_count() == launched
    c.close()
    d = small(512, (1, 1), (40, 7)).build()
    assert pg.pg_attn_paged_sink(d.plan, d.desc, 0, d.q, d.out, d.lse, 5, 1, 1.0, None, 0) == pg.PG_ERR_WORKSPACE
    assert pg.pg_attn_paged_sink(d.plan, d.desc, 0, d.q, d.out, d.lse, 5, 1, 1.0, d.ws,
                                 pg.pg_workspace_bytes(d.plan) - 1) == pg.PG_ERR_WORKSPACE
    d.close()


def test_eviction_refusals():
    c = small(512, (1, 1), (40, 70), layers=2).build()
    src = torch.full((2, 2, 1, 16), -5, dtype=torch.int32, device="cuda")
    launched = pg.pg_launch_count()

    def sel(stats=c.stats, layer=0, n=2, budget=16, sinks=4, recent=8, out=src, stream=None):
        return pg.pg_kv_evict_select(c.plan, stats, layer, n, budget, sinks, recent, out, stream)

    assert sel(budget=0, sinks=0, recent=0) == pg.PG_ERR_ARG
    assert sel(sinks=9) == pg.PG_ERR_ARG and sel(recent=13) == pg.PG_ERR_ARG
    assert sel(sinks=-1) == pg.PG_ERR_ARG and sel(recent=-1) == pg.PG_ERR_ARG
    assert sel(sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == pg.PG_ERR_ARG
    assert sel(layer=1) == pg.PG_ERR_LAYER and sel(layer=-1) == pg.PG_ERR_LAYER
    assert sel(n=0) == pg.PG_ERR_LAYER and sel(n=3) == pg.PG_ERR_LAYER
    assert sel(out=None) == pg.PG_ERR_ARG and sel(out=src.data_ptr() + 2) == pg.PG_ERR_ALIGN
    assert sel(stats=None) == pg.PG_ERR_ARG
    assert sel(stats=pg.stats_descriptor(c.mass, c.pos, page_size=8, capacity=c.mass.numel() // 2)) \
        == pg.PG_ERR_PLAN_MISMATCH
    assert sel(stream=torch.cuda.Stream()) == pg.PG_ERR_STREAM
    few = c.mass[:, :1].contiguous(), c.pos[:, :1].contiguous()
    assert sel(stats=pg.stats_descriptor(*few)) == pg.PG_ERR_PAGE_OOB

    def app(pool=c.desc, stats=c.stats, n=2, budget=16):
        return pg.pg_kv_evict_apply(c.plan, pool, stats, 0, n, budget, src)

    assert app(n=3) == pg.PG_ERR_LAYER and app(budget=0) == pg.PG_ERR_ARG
    assert app(pool=pg.pool_descriptor(c.pool[:1].contiguous())) == pg.PG_ERR_LAYOUT
    assert (src == -5).all() and pg.pg_launch_count() == launched
    c.close()


def test_ring_plans_and_shared_pages_are_refused():
    c = small(256, (1, 1), (100, 100)).build()
    rc, ring = pg.pg_plan_paged_prefill_ring(None, 2, c.qo_indptr, c.pg_indptr, c.ids, c.start, 16, 8,
                                             256, 16, 60)
    pg.check(rc)
    src = torch.zeros((1, 2, 8, 8), dtype=torch.int32, device="cuda")
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    assert pg.pg_attn_paged_sink(ring, c.desc, 0, c.q, c.out, c.lse, 5, 1, 1.0, big, big.numel()) \
        == pg.PG_ERR_PLAN_MISMATCH
    assert pg.pg_attn_paged_mass(ring, c.desc, 0, c.q, c.out, c.lse, c.stats, 5, 1, 1.0, big, big.numel()) \
        == pg.PG_ERR_PLAN_MISMATCH
    assert pg.pg_kv_evict_select(ring, c.stats, 0, 1, 8, 0, 0, src) == pg.PG_ERR_PLAN_MISMATCH
    assert pg.pg_kv_evict_apply(ring, c.desc, c.stats, 0, 1, 8, src) == pg.PG_ERR_PLAN_MISMATCH
    ring.close()
    ids = c.ids.copy()
    ids[-1] = ids[0]  # two requests share a page
    for far in (False, True):  # the check's two forms: page ids dense or far apart
        pages = ids.astype(np.int64) * (40_000_000 if far else 1)
        rc, plan = pg.pg_plan_paged_segment(None, 2, c.qo_indptr, c.pg_indptr, pages.astype(np.int32),
                                            c.last, c.ks, c.start, 16, 8, 256, 16)
        pg.check(rc)
        stats = c.stats if not far else pg.stats_descriptor(
            c.mass, c.pos, num_pages=1 << 30, capacity=(1 << 30) * 8 * 16)
        if not far:  # attention alone may share pages
            pg.check(pg.pg_attn_paged_sink(plan, c.desc, 0, c.q, c.out, c.lse, 5, 1, 1.0, big, big.numel()))
            assert pg.pg_attn_paged_mass(plan, c.desc, 0, c.q, c.out, c.lse, c.stats, 5, 1, 1.0, big,
                                         big.numel()) == pg.PG_ERR_SHARED_PAGE
            assert pg.pg_kv_evict_apply(plan, c.desc, c.stats, 0, 1, 8, src) == pg.PG_ERR_SHARED_PAGE
        assert pg.pg_kv_evict_select(plan, stats, 0, 1, 8, 0, 0, src) == pg.PG_ERR_SHARED_PAGE
        plan.close()
    ok()
    c.close()


def test_an_updated_plan_is_checked_again():
    c = small(512, (1, 1), (100, 100)).build()
    src = torch.zeros((1, 2, 1, 8), dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 1, 8, 0, 0, src))
    ids = c.ids.copy()
    ids[-1] = ids[0]
    rc, _ = pg.pg_plan_paged_segment(c.plan, 2, c.qo_indptr, c.pg_indptr, ids, c.last, c.ks, c.start,
                                     16, 1, 512, 16)
    pg.check(rc)
    assert pg.pg_kv_evict_select(c.plan, c.stats, 0, 1, 8, 0, 0, src) == pg.PG_ERR_SHARED_PAGE
    rc, _ = pg.pg_plan_paged_segment(c.plan, 2, c.qo_indptr, c.pg_indptr, c.ids, c.last, c.ks, c.start,
                                     16, 1, 512, 16)
    pg.check(rc)
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 1, 8, 0, 0, src))
    ok()
    c.close()


def test_empty_plan_launches_nothing():
    c = small().build()
    z = np.zeros(1, np.int64)
    rc, plan = pg.pg_plan_paged_segment(None, 0, z, z, None, None, z, None, 16, 8, 256, 16)
    pg.check(rc)
    n = pg.pg_launch_count()
    assert pg.pg_attn_paged_sink(plan, c.desc, 0, None, None, None, 5, 1, 1.0) == pg.PG_OK
    assert pg.pg_attn_paged_mass(plan, c.desc, 0, None, None, None, c.stats, 5, 1, 1.0) == pg.PG_OK
    assert pg.pg_kv_evict_select(plan, c.stats, 0, 1, 8, 0, 0, None) == pg.PG_OK
    assert pg.pg_kv_evict_apply(plan, c.desc, c.stats, 0, 1, 8, None) == pg.PG_OK
    assert pg.pg_launch_count() == n
    plan.close()
    c.close()


# ------------------------------------------------------------------ memory around the call
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("qo,start", [([200, 3], [0, 300]), ([1] * 5, [0, 130, 700, 2000, 64])])
def test_guarded_buffers(D, qo, start):
    """Nothing is written outside the rows, the workspace's stated size and the statistics."""
    c = Case(D, *HQ[D], qo, start, seed=2).build()
    T = c.q.shape[0]
    out = torch.full((T + 2, c.hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 2, c.hq), 7.0, device="cuda")
    for mass in (False, True):
        n = (pg.pg_mass_workspace_bytes if mass else pg.pg_workspace_bytes)(c.plan)
        ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
        if mass:
            pg.check(pg.pg_attn_paged_mass(c.plan, c.desc, 0, c.q, out[1:], lse[1:], c.stats, 90, 3, 1.0,
                                           ws, n))
        else:
            pg.check(pg.pg_attn_paged_sink(c.plan, c.desc, 0, c.q, out[1:], lse[1:], 90, 3, 1.0, ws, n))
        ok()
        assert (ws[n:] == 0xAB).all()
        c.out, c.lse = out[1:-1], lse[1:-1]
        c.reference(90, 3)
        c.check_attention()
        for x in (out, lse):
            assert (x[0] == 7).all() and (x[-1] == 7).all()
    c.check_mass()
    assert torch.equal(c.pool.cpu(), c.pool_cpu)
    c.close()


@pytest.mark.parametrize("skew", [1, 2, 4])
@pytest.mark.parametrize("n", [50, 1500, 9000])
def test_statistics_at_any_alignment(skew, n):
    c = Case(512, 2, 2, [1, 1], [n - 1, n // 2], seed=n)
    c.pos_cpu[:] = torch.randperm(c.pos_cpu.numel(), dtype=torch.int32).reshape(c.pos_cpu.shape) + 10 * n
    c.build()
    m = torch.zeros(c.mass.numel() + 8, device="cuda")
    p = torch.zeros(c.mass.numel() + 8, dtype=torch.int32, device="cuda")
    mass, pos = (x[skew:skew + c.mass.numel()].view(c.mass.shape) for x in (m, p))
    mass.copy_(c.mass)
    pos.copy_(c.pos)
    b = n * 2 // 3
    src = torch.full((1, 2, 2, b), -9, dtype=torch.int32, device="cuda")
    stats = pg.stats_descriptor(mass, pos)
    pg.check(pg.pg_kv_evict_select(c.plan, stats, 0, 1, b, 0, 0, src))
    ok()
    want = select_reference(c, b, 0, 0, c.mass_cpu.numpy(), c.pos_cpu.numpy(), [0])
    assert (src.cpu().numpy() == want).all()
    pg.check(pg.pg_kv_evict_apply(c.plan, c.desc, stats, 0, 1, b, src))
    ok()
    pool, rm, rp = apply_reference(c, want, [0], c.pool_cpu, c.mass_cpu, c.pos_cpu)
    assert torch.equal(c.pool.cpu(), pool) and torch.equal(mass.cpu(), rm) and torch.equal(pos.cpu(), rp)
    c.upload()
    pg.check(pg.pg_attn_paged_mass(c.plan, c.desc, 0, c.q, c.out, c.lse, stats, -1, 0, 1.0, c.ws,
                                   pg.pg_mass_workspace_bytes(c.plan)))
    ok()
    c.reference(-1, 0, mass=rm, pos=rp)
    c.mass, c.pos = mass, pos
    c.check_attention()
    c.check_mass(old=rm)
    c.close()


# ------------------------------------------------------------------ batches and far offsets
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("R", [33, 150, 300])
def test_many_requests(D, R):
    rng = np.random.Generator(np.random.PCG64(R))
    start = rng.integers(0, 400, R)
    start[:5] = [0, 15, 16, 127, 128]
    c = Case(D, *HQ[D], np.ones(R, int), start, seed=R).build()
    c.weigh(200, 3)
    ok()
    c.reference(200, 3)
    c.check_attention()
    c.check_mass()
    c.close()
    qo = rng.integers(1, 40, R)
    c = Case(D, *HQ[D], qo, start, seed=R + 1).build()
    c.weigh(-1, 0)
    ok()
    c.reference(-1, 0)
    c.check_attention()
    c.check_mass()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_offsets_past_32_bits(D):
    """Pages at the far end of a pool of more than 2^31 elements, in its second layer."""
    per_page = 2 * HQ[D][1] * 16 * D
    P = (1 << 30) // per_page + 5000  # two layers: more than 2^31 elements, more than 2^32 bytes
    for qo, start in (([40, 7], [100, 0]), ([1, 1], [700, 33])):
        c = Case(D, *HQ[D], qo, start, seed=5, layers=1)
        near = c.P
        c.ids = c.ids + (P - near)
        c.plan = None
        pool = torch.empty((2, P, 2, HQ[D][1], 16, D), dtype=torch.bfloat16, device="cuda")
        assert pool.numel() > 2 ** 31
        pool[1, P - near:] = c.pool_cpu[0].cuda()
        mass = torch.zeros((2, P, HQ[D][1], 16), device="cuda")
        pos = torch.full((2, P, HQ[D][1], 16), 10 ** 6, dtype=torch.int32, device="cuda")
        mass[1, P - near:] = c.mass_cpu[0].cuda()
        pos[1, P - near:] = c.pos_cpu[0].cuda()
        rc, plan = pg.pg_plan_paged_segment(None, 2, c.qo_indptr, c.pg_indptr, c.ids, c.last, c.ks, c.start,
                                            c.hq, c.hkv, D, 16)
        pg.check(rc)
        c.plan = plan
        desc, stats = pg.pool_descriptor(pool), pg.stats_descriptor(mass, pos)
        c.upload()
        pg.check(pg.pg_attn_paged_mass(plan, desc, 1, c.q, c.out, c.lse, stats, 90, 3, 1.0, c.ws,
                                       pg.pg_mass_workspace_bytes(plan)))
        ok()
        c.ids = c.ids - (P - near)
        c.reference(90, 3)
        c.check_attention()
        c.mass, c.pos = mass[1:, P - near:].contiguous(), pos[1:, P - near:].contiguous()
        c.check_mass()
        src = torch.empty((1, 2, c.hkv, 20), dtype=torch.int32, device="cuda")
        pg.check(pg.pg_kv_evict_select(plan, stats, 1, 1, 20, 2, 3, src))
        pg.check(pg.pg_kv_evict_apply(plan, desc, stats, 1, 1, 20, src))
        ok()
        m0, p0 = c.mass.cpu(), c.pos.cpu()
        want = select_reference(c, 20, 2, 3, m0.numpy(), p0.numpy(), [0])
        assert (src.cpu().numpy() == want).all()
        wp, wm, wpos = apply_reference(c, want, [0], c.pool_cpu, m0, p0)
        assert torch.equal(pool[1, P - near:].cpu(), wp[0])
        assert torch.equal(mass[1, P - near:].cpu(), wm[0])
        c.close()
        del pool, mass, pos
        torch.cuda.empty_cache()


# ------------------------------------------------------------------ streams and graphs
def test_two_streams_at_once():
    """Two plans on two streams, workspaces of their own, calls in flight together."""
    runs = []
    for i, D in enumerate((256, 512)):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            runs.append(Case(D, *HQ[D], [1] * 20, list(range(100, 2100, 100)), seed=i, stream=s).build())
    torch.cuda.synchronize()
    for _ in range(8):
        for c in runs:
            with torch.cuda.stream(c.stream):
                c.sink(300, 4)
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK
    for c in runs:
        c.reference(300, 4)
        c.check_attention()
        c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_captured_decode_step_follows_the_plan(D):
    """One captured step (weights, choice) replayed while the plan is updated in place under it, to
    more and to fewer keys on the same pages (a captured call holds the plan's layout: as many
    requests, tokens and pages)."""
    s = torch.cuda.Stream()
    start = np.array([130, 40, 300])
    with torch.cuda.stream(s):
        c = Case(D, *HQ[D], [1, 1, 1], start + 40, seed=3, stream=s)
        c.build()
        budget = 30
        src = torch.zeros((1, 3, c.hkv, budget), dtype=torch.int32, device="cuda")

        def call():
            c.weigh(-1, 0)
            pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 1, budget, 2, 5, src, s))

        call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        for extra in (45, 40, 43):
            c.start, c.n = start + extra, start + extra + 1
            npg = (c.n + 15) // 16
            assert (np.diff(c.pg_indptr) == npg).all()
            c.last = (c.n - (npg - 1) * 16).astype(np.int32)
            rc, _ = pg.pg_plan_paged_segment(c.plan, 3, c.qo_indptr, c.pg_indptr, c.ids, c.last, c.ks,
                                             c.start, c.hq, c.hkv, D, 16, s)
            pg.check(rc)
            m0, p0 = c.mass.cpu(), c.pos.cpu()
            c.out.fill_(float("nan"))
            g.replay()
            s.synchronize()
            assert pg.pg_device_status(s) == pg.PG_OK
            c.reference(-1, 0, mass=m0, pos=p0)
            c.check_attention(f"{extra}")
            c.check_mass(f"{extra}", old=m0)
            want = select_reference(c, budget, 2, 5, c.mass.cpu().numpy(), c.pos.cpu().numpy(), [0])
            assert (src.cpu().numpy() == want).all()
    c.close()


def test_captured_prefill():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = small(512, (300, 20), (0, 90), stream=s, seed=4).build()
        c.weigh()
        s.synchronize()
        c.upload()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.weigh()
        g.replay()
        s.synchronize()
    assert pg.pg_device_status() == pg.PG_OK
    c.reference(-1, 0)
    c.check_attention()
    c.check_mass()
    c.close()


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_hidden_keys_add_no_weight(D, bad):
    """Non-finite K rows outside the mask reach neither the sums nor the statistics."""
    for qo, start in (([64], [576]), ([1], [600])):
        c = Case(D, *HQ[D], qo, start, seed=6)
        page, off = c.rows_of(0)
        c.pool_cpu[0, page[64:448], 0, :, off[64:448]] = bad
        c.build()
        c.weigh(127, 64)
        ok()
        c.reference(127, 64)
        c.check_attention()
        c.check_mass()
        c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("gain", [30.0, 200.0])
def test_peaked_scores(D, gain):
    """Scores of hundreds: references move during a row, weights underflow to zero."""
    for qo, start in (([150, 20], [0, 700]), ([1, 1, 1], [900, 400, 31])):
        c = Case(D, *HQ[D], qo, start, seed=7, gain=gain).build()
        c.weigh(300, 4)
        ok()
        c.reference(300, 4)
        c.check_attention()
        c.check_mass()
        c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_growing_scores(D):
    """Each later tile's scores far above the earlier ones': every tile rescales."""
    n = 700
    c = Case(D, *HQ[D], [1, 1], [n - 1, n - 1], seed=8)
    for r in range(2):
        page, off = c.rows_of(r)
        grow = torch.linspace(0.0, 12.0, n).repeat(1)[:, None, None]
        row = torch.ones((n, c.hkv, D)) * grow / D
        if r == 1:
            row = row.flip(0)
        c.pool_cpu[0, page, 0, :, off] = row.to(torch.bfloat16)
    c.q_cpu[:] = 80.0
    c.build()
    c.weigh()
    ok()
    c.reference(-1, 0)
    c.check_attention()
    c.check_mass()
    c.close()


# ------------------------------------------------------------------ together
def test_a_serving_loop_that_evicts():
    """A global layer served under a budget through the page allocator: prompts are scored as they
    are read, every step over the budget evicts, and decoding goes on with segment plans. Each
    step is checked against the reference from the state before it; at the end the keys held are
    those of the recorded positions, bit for bit."""
    D, hq, hkv, ps, budget, L = 512, 16, 1, 16, 40, 2
    P = 64
    rc, srv = pg.pg_kv_server_create(P, P, ps, 1023, 0, 1 << 16)
    pg.check(rc)
    ids = [pg.pg_kv_request_open(srv)[1] for _ in range(3)]
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = 4096
    cos, sin = (torch.empty((rows, D // 2), device="cuda") for _ in range(2))
    pg.check(pg.pg_rope_table(cos, sin, rows, D, 1.0e6))
    wq = torch.full((D,), 2.0 / np.sqrt(D), dtype=torch.bfloat16, device="cuda")
    wk = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((L, P, 2, hkv, ps, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    mass = torch.full((L, P, hkv, ps), float("nan"), device="cuda")
    pos = torch.full((L, P, hkv, ps), -1, dtype=torch.int32, device="cuda")
    desc, stats = pg.pool_descriptor(pool), pg.stats_descriptor(mass, pos)
    written = {}  # (request, layer, position) -> the K row prep stored
    front = dict.fromkeys(ids, 0)
    plan = None
    for step, lens in enumerate([[70, 33, 90], [1, 1, 1], [1, 1, 1], [25, 1, 3], [1, 1, 1], [1, 1, 1]]):
        for rid, n in zip(ids, lens):
            pg.check(pg.pg_kv_admit_step(srv, rid, n))
        rc, ptr, pages, last, first, start = pg.pg_kv_batch_segment_inputs(srv, ids, lens)
        pg.check(rc)
        c = Case(D, hq, hkv, lens, start, ps=ps, evicted=first, layers=L, seed=step)
        assert (c.pg_indptr == ptr).all() and (c.last == last).all()
        c.ids, c.P = pages, P
        rc, plan = pg.pg_plan_paged_segment(plan, 3, c.qo_indptr, ptr, pages, last, first, start, hq, hkv,
                                            D, ps)
        pg.check(rc)
        c.plan = plan
        T = int(c.qo_indptr[-1])
        ws = torch.empty(max(pg.pg_mass_workspace_bytes(plan), 16), dtype=torch.uint8, device="cuda")
        src = torch.empty((L, 3, hkv, budget), dtype=torch.int32, device="cuda")
        for layer in range(L):
            q, k = (torch.randn((T, h, D), device="cuda", generator=g).to(torch.bfloat16) for h in (hq, hkv))
            qo = torch.empty_like(q)
            out, lse = torch.empty_like(q), torch.empty((T, hq), device="cuda")
            pg.check(pg.pg_prep_paged_hd512(plan, desc, layer, q, hq * D, k, hkv * D, wq, wk, 1e-6, cos, sin,
                                            rows, qo))
            m0, p0 = mass.cpu(), pos.cpu()
            pg.check(pg.pg_attn_paged_mass(plan, desc, layer, qo, out, lse, stats, -1, 0, 1.0, ws, ws.numel()))
            ok()
            c.layer, c.pool_cpu, c.q_cpu = layer, pool.cpu(), qo.cpu()
            c.out, c.lse, c.mass, c.pos = out, lse, mass, pos
            c.reference(-1, 0, mass=m0.nan_to_num(0.0), pos=p0)
            c.check_attention(f"step {step}")
            got = mass.cpu()
            c.mass = torch.where(torch.isnan(got) & torch.isnan(m0), torch.zeros_like(got), got)
            c.check_mass(f"step {step}", old=m0.nan_to_num(0.0))
            for i, rid in enumerate(ids):
                page, off = c.rows_of(i)
                for t in range(lens[i]):
                    s = int(c.n[i]) - lens[i] + t
                    written[rid, layer, int(start[i]) + t] = pool[layer, page[s], 0, 0, off[s]].cpu()
        m0, p0, pool0 = mass.cpu(), pos.cpu(), pool.cpu()
        pg.check(pg.pg_kv_evict_select(plan, stats, 0, L, budget, 4, 16, src))
        pg.check(pg.pg_kv_evict_apply(plan, desc, stats, 0, L, budget, src))
        ok()
        want = select_reference(c, budget, 4, 16, m0.numpy(), p0.numpy(), range(L))
        assert (src.cpu().numpy() == want).all()
        wp, wm, wpos = apply_reference(c, want, range(L), pool0, m0, p0)
        assert torch.equal(pool.cpu().view(torch.int16), wp.view(torch.int16))
        assert torch.equal(pos.cpu(), wpos)
        for i, rid in enumerate(ids):
            pg.check(pg.pg_kv_commit_step(srv, rid))
            front[rid] += lens[i]
            if c.n[i] > budget:
                pg.check(pg.pg_kv_request_evict(srv, rid, budget))
    assert pg.pg_kv_free_pages(srv, pg.PG_KV_GLOBAL)[1] == P - 3 * 3  # three pages of 16 hold 40 keys
    for rid in ids:
        pages = pg.pg_kv_request_pages(srv, rid, pg.PG_KV_GLOBAL)[1]
        for layer in range(L):
            seen = set()
            for s in range(min(budget, front[rid])):  # one request stays below the budget
                p = int(pos[layer, pages[s // ps], 0, s % ps])
                seen.add(p)
                assert torch.equal(pool[layer, pages[s // ps], 0, 0, s % ps].cpu(), written[rid, layer, p])
            assert len(seen) == min(budget, front[rid]) and set(range(4)) <= seen
            assert set(range(front[rid] - 16, front[rid])) <= seen
    plan.close()
    pg.pg_kv_server_destroy(srv)


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("ps", [8, 16, 32, 64, 3])
@pytest.mark.parametrize("window,sinks", [(100, 4), (65, 70), (3, 1), (40, 0)])
def test_pages_behind_the_window_may_be_given_away(D, ps, window, sinks):
    """Places of pages that no query sees all name one page that holds NaN and that another request
    owns; the outputs are those of the full page list."""
    for qo, start in (([40, 3, 200], [700, 300, 450]), ([1, 1, 1], [700, 301, 64])):
        c = Case(D, *HQ[D], qo, start, ps=ps, seed=window + ps)
        foreign = int(np.setdiff1d(np.arange(c.P), c.ids)[0])
        c.pool_cpu[0, foreign] = float("nan")
        full = c.ids.copy()
        for r in range(len(qo)):
            for i in range(c.pg_indptr[r + 1] - c.pg_indptr[r]):
                last = (i + 1) * ps - 1  # the page's last key
                if last < start[r] - window and i * ps >= sinks:
                    c.ids[c.pg_indptr[r] + i] = foreign
        assert (c.ids == foreign).sum() > 1
        c.build()
        c.sink(window, sinks)
        ok()
        c.ids = full
        c.reference(window, sinks)
        c.check_attention(f"{qo}")
        c.close()


def test_a_local_layer_served_from_a_few_pages():
    """Window and sinks through the page allocator: two requests run to ten times the window from a
    pool that holds a fifth of their keys, prefill chunks and single tokens; each step against the
    full history. A request under this window and a step of 30 holds up to 1 + 9 + 1 pages, so two
    do not always fit in 20: the second is then refused and served in the batch after."""
    D, hq, hkv, ps, window, sinks = 256, 16, 8, 8, 40, 5
    P = 20  # pages; 2 requests of 400 tokens are 100
    rc, srv = pg.pg_kv_server_create(P, 1000, ps, window, 0, 1 << 16)
    pg.check(rc)
    ids = [pg.pg_kv_request_open(srv)[1] for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(9)
    cos, sin = (torch.empty((1024, D // 2), device="cuda") for _ in range(2))
    pg.check(pg.pg_rope_table(cos, sin, 1024, D, 1.0e4))
    wq = torch.full((D,), 2.0 / np.sqrt(D), dtype=torch.bfloat16, device="cuda")
    wk = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((1, P, 2, hkv, ps, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    desc = pg.pool_descriptor(pool)
    hist = [torch.zeros((0, 2, hkv, D), dtype=torch.bfloat16) for _ in ids]
    plan = None
    steps = [[30, 17]] + [[1, 1]] * 12 + [[25, 1], [3, 30]] + [[1, 1]] * 20 + [[30, 30]] * 8 + [[1, 1]] * 9
    refused = 0
    for step, lens in enumerate(steps):
        todo = [0, 1]
        while todo:
            now = []
            for i in todo:
                free = pg.pg_kv_free_pages(srv, pg.PG_KV_LOCAL)[1]
                rc = pg.pg_kv_admit_step(srv, ids[i], lens[i])
                if rc == pg.PG_KV_OK:
                    now.append(i)
                    continue
                end = len(hist[i]) + lens[i]
                assert rc == pg.PG_KV_ERR_NO_PAGES and -(-end // ps) - -(-len(hist[i]) // ps) > free
                assert pg.pg_kv_free_pages(srv, pg.PG_KV_LOCAL)[1] == free
                refused += 1
            assert now
            todo = [i for i in todo if i not in now]
            rids, n_new = [ids[i] for i in now], [lens[i] for i in now]
            rc, ptr, pages, last, start = pg.pg_kv_batch_plan_inputs(srv, pg.PG_KV_LOCAL, rids, n_new)
            pg.check(rc)
            qo = np.concatenate([[0], np.cumsum(n_new)])
            rc, plan = pg.pg_plan_paged_prefill(plan, len(now), qo, ptr, pages, last, start, hq, hkv, D, ps)
            pg.check(rc)
            T = int(qo[-1])
            q, k, v = (torch.randn((T, h, D), device="cuda", generator=g).to(torch.bfloat16)
                       for h in (hq, hkv, hkv))
            qr, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((T, hq), device="cuda")
            n = pg.pg_workspace_bytes(plan)
            ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
            pg.check(pg.pg_prep_paged_hd256(plan, desc, 0, q, hq * D, k, hkv * D, v, hkv * D, wq, wk, 1e-6,
                                            cos, sin, 1024, qr))
            pg.check(pg.pg_attn_paged_sink(plan, desc, 0, qr, out, lse, window, sinks, 1.0, ws, n))
            ok()
            for j, i in enumerate(now):
                s = np.arange(start[j], start[j] + n_new[j])
                page = torch.from_numpy(pages[ptr[j] + s // ps].astype(np.int64)).cuda()
                new = pool[0].permute(0, 3, 1, 2, 4)[page, torch.from_numpy(s % ps).cuda()].cpu()
                hist[i] = torch.cat([hist[i], new])
            # the same rows over a full page list of the whole history
            c = Case(D, hq, hkv, n_new, start, ps=ps, seed=step)
            for j, i in enumerate(now):
                page, off = c.rows_of(j)
                c.pool_cpu[0].permute(0, 3, 1, 2, 4)[torch.as_tensor(page), torch.as_tensor(off)] = hist[i]
            c.q_cpu, c.out, c.lse = qr.cpu(), out, lse
            c.reference(window, sinks)
            c.check_attention(f"step {step}")
            for rid in rids:
                pg.check(pg.pg_kv_commit_step(srv, rid))
                pg.check(pg.pg_kv_request_trim(srv, rid, sinks)[0])
    assert refused
    assert min(len(h) for h in hist) > 300 and pg.pg_kv_free_pages(srv, pg.PG_KV_LOCAL)[1] > 0
    plan.close()
    pg.pg_kv_server_destroy(srv)


@pytest.mark.parametrize("D,hq,hkv,ps,qo", [(256, 16, 8, 16, 1), (256, 16, 8, 16, 70), (512, 16, 1, 8, 1),
                                            (512, 16, 1, 8, 130), (256, 4, 2, 4, 1), (256, 4, 2, 4, 9)])
def test_the_last_positions(D, hq, hkv, ps, qo):
    """A request whose earlier keys were evicted may sit anywhere in int32, up to the stated end."""
    end = 2 ** 31 - 1 - 1024
    for e, rc in [(end, pg.PG_OK), (end + 1, pg.PG_ERR_I32_OVERFLOW), (2 ** 31 - 1, pg.PG_ERR_I32_OVERFLOW)]:
        start = e - qo
        c = Case(D, hq, hkv, [qo], [start], ps=ps, evicted=start - 150, seed=D + qo).build()
        n = max(pg.pg_workspace_bytes(c.plan), pg.pg_mass_workspace_bytes(c.plan), 16)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        for window, sinks in [(60, start - 140), (2 ** 31 - 1, 2 ** 31 - 1), (-1, 0)]:
            args = (c.plan, c.desc, 0, c.q, c.out, c.lse)
            assert pg.pg_attn_paged_sink(*args, window, sinks, 1.0, ws, n) == rc
            if rc == pg.PG_OK:
                ok()
                c.reference(window, sinks)
                c.check_attention(f"window {window}")
            assert pg.pg_attn_paged_mass(*args, c.stats, window, sinks, 1.0, ws, n) == rc
        ok()
        c.close()


@pytest.mark.parametrize("D,hq,hkv,ps", [(512, 16, 1, 16), (256, 16, 8, 8), (256, 4, 2, 5), (512, 16, 1, 1)])
@pytest.mark.parametrize("qo", [1, 40, 300])
@pytest.mark.parametrize("window,sinks", [(60, 7), (0, 0), (600, 130), (-1, 0)])
def test_statistics_of_unseen_keys_are_not_touched(D, hq, hkv, ps, qo, window, sinks):
    """Their masses are -0 here, which adding nothing would turn into +0."""
    c = Case(D, hq, hkv, [qo, qo], [700, 333], ps=ps, seed=qo + ps)
    c.mass_cpu.fill_(-0.0)
    c.build()
    n = max(pg.pg_mass_workspace_bytes(c.plan), 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pg.check(pg.pg_attn_paged_mass(c.plan, c.desc, 0, c.q, c.out, c.lse, c.stats, window, sinks, 1.0, ws, n))
    ok()
    mass, pos = c.mass.cpu().view(torch.int32).numpy(), c.pos.cpu().numpy()
    held = np.zeros(mass.shape[1::2], bool)  # [page][slot]
    for r in range(2):
        p = c.start[r] + np.arange(qo)
        j = np.arange(c.n[r])
        see = (j[None] <= p[:, None]) & ((window < 0) | (p[:, None] - j[None] <= window) | (j[None] < sinks))
        page, off = c.rows_of(r)
        held[page[see.any(0)], off[see.any(0)]] = True
        new = j >= c.start[r]
        assert (pos[0, page[new], :, off[new]] == j[new][:, None]).all()
        assert (pos[0, page[~new], :, off[~new]] == -7).all()
    assert (mass[0].transpose(0, 2, 1)[~held] == -2 ** 31).all()
    assert (mass[0].transpose(0, 2, 1)[held] >= 0).all()
