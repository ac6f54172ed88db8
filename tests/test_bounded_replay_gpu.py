"""Captured bounded-cache calls replayed under plans that are updated in place (GPU): as many
requests, tokens and pages as the capture had, held by other requests than before. References and
tolerances: bounded_ref.py."""
import numpy as np
import pytest
import torch

from bounded_ref import Case, apply_reference, select_reference
from paged_sliding_window_qkv_gb300 import pg

pytestmark = pytest.mark.gpu


def replan(c, qo, start, seed):
    """The case's plan, updated in place to other lengths and another order of as many pages."""
    tokens, pages, storage = int(c.qo.sum()), len(c.ids), c.plan.info().d_page_ids
    c.qo, c.start = np.asarray(qo, np.int64), np.asarray(start, np.int64)
    c.n = c.start + c.qo - c.ks
    npg = (c.n + c.ps - 1) // c.ps
    assert int(c.qo.sum()) == tokens and int(npg.sum()) == pages
    c.pg_indptr = np.concatenate([[0], np.cumsum(npg)])
    c.qo_indptr = np.concatenate([[0], np.cumsum(c.qo)])
    c.ids = np.random.Generator(np.random.PCG64(seed)).permutation(c.P)[:pages].astype(np.int32)
    c.last = (c.n - (npg - 1) * c.ps).astype(np.int32)
    rc, _ = pg.pg_plan_paged_segment(c.plan, len(c.qo), c.qo_indptr, c.pg_indptr, c.ids, c.last, c.ks,
                                     c.start, c.hq, c.hkv, c.D, c.ps, c.stream)
    pg.check(rc)
    assert c.plan.info().d_page_ids == storage  # in place


def capture(call, stream):
    call()  # eager: configures every kernel once
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        call()
    return g


def refill(c, seed, evicted=0):
    """Distinct positions in any order, and masses with ties, into the case's own statistics."""
    g = np.random.Generator(np.random.PCG64(seed))
    pos, mass = c.pos_cpu.numpy(), c.mass_cpu.numpy()
    for layer in range(c.layers):
        for r in range(len(c.qo)):
            page, off = c.rows_of(r)
            for h in range(c.hkv):
                pos[layer, page, h, off] = g.permutation(int(c.n[r]))
                m = g.exponential(1.0, int(c.n[r])).astype(np.float32)
                m[g.random(len(m)) < 0.2] = 0.5
                mass[layer, page, h, off] = m
    c.mass.copy_(c.mass_cpu)
    c.pos.copy_(c.pos_cpu)


# (head_dim, KV heads, page size, layers, keys captured, keys replayed, budget)
GROWN = [
    (512, 1, 256, 1, [300], [500], 450),             # inside the last page
    (512, 1, 16, 2, [256, 256], [496, 16], 300),     # pages move to one request
    (256, 2, 16, 1, [100, 100], [40, 170], 150),
    (256, 2, 5, 1, [200, 200], [395, 5], 350),       # no power of two
    (512, 1, 3, 1, [9, 9, 9], [21, 3, 3], 20),
    (256, 8, 16, 4, [300] * 20, [2400] + [192] * 18 + [224], 2200),  # next to none move
]


@pytest.mark.parametrize("D,hkv,ps,layers,before,after,budget", GROWN)
def test_captured_apply_moves_every_kept_key(D, hkv, ps, layers, before, after, budget):
    s = torch.cuda.Stream()
    every = list(range(layers))
    with torch.cuda.stream(s):
        c = Case(D, hkv, hkv, [1] * len(before), np.array(before) - 1, ps=ps, layers=layers, seed=budget,
                 stream=s)
        c.build()
        src = torch.full((layers, len(before), hkv, budget), -1, dtype=torch.int32, device="cuda")
        g = capture(lambda: pg.check(pg.pg_kv_evict_apply(c.plan, c.desc, c.stats, 0, layers, budget, src, s)), s)
        for turn, n in enumerate((after, before, after)):
            replan(c, [1] * len(n), np.array(n) - 1, turn)
            refill(c, turn)
            c.pool.copy_(c.pool_cpu)
            want = select_reference(c, budget, 1, 2, c.mass_cpu.numpy(), c.pos_cpu.numpy(), every)
            src.copy_(torch.from_numpy(want))
            g.replay()
            s.synchronize()
            assert pg.pg_device_status(s) == pg.PG_OK
            pool, mass, pos = apply_reference(c, want, every, c.pool_cpu, c.mass_cpu, c.pos_cpu)
            assert torch.equal(c.pool.view(torch.int16).cpu(), pool.view(torch.int16))
            assert torch.equal(c.mass.cpu(), mass) and torch.equal(c.pos.cpu(), pos)
    c.close()


def replayed_weights(D, hq, hkv, ps, shapes, window, sinks):
    """Weights captured at the first of shapes [(tokens, keys) of each request, ...] and replayed at
    all of them in turn, each against 64 bits."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        (qo, n), rest = shapes[0], shapes[1:]
        c = Case(D, hq, hkv, qo, np.array(n) - qo, ps=ps, seed=ps, stream=s).build()
        g = capture(lambda: c.weigh(window, sinks), s)
        for turn, (qo, n) in enumerate([*rest, shapes[0], *rest]):
            replan(c, qo, np.array(n) - qo, turn)
            c.mass.copy_(c.mass_cpu)
            c.pos.copy_(c.pos_cpu)
            c.out.fill_(float("nan"))
            c.lse.fill_(float("nan"))
            c.ws.fill_(0xFF)
            g.replay()
            s.synchronize()
            assert pg.pg_device_status(s) == pg.PG_OK
            c.reference(window, sinks)
            c.check_attention(f"{n}")
            c.check_mass(f"{n}")
    c.close()


@pytest.mark.parametrize("D,hq,hkv", [(256, 4, 2), (512, 4, 1)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (90, 5)])
@pytest.mark.parametrize("ps,qo,before,after", [
    (5, [20], [62], [65]),                     # inside the last page, past a block of 64 keys
    (3, [10, 10], [150, 150], [288, 10]),      # pages move to one request
    (1, [7, 30, 5], [100, 40, 60], [8, 187, 5]),
    (16, [10, 33], [150, 160], [16, 300]),
    (64, [40, 200], [250, 260], [40, 500]),
])
def test_captured_prompt_weights_follow_the_plan(D, hq, hkv, window, sinks, ps, qo, before, after):
    replayed_weights(D, hq, hkv, ps, [(qo, before), (qo, after)], window, sinks)


# (head_dim, KV heads, page size, layers, keys captured, keys replayed, budget): the replayed segments
# are longer than the registers that the captured choice holds its keys in
@pytest.mark.parametrize("D,hkv,ps,layers,before,after,budget", [
    (256, 2, 16, 1, [400, 400], [784, 16], 300),
    (256, 2, 5, 2, [400, 400], [795, 5], 500),
    (512, 1, 16, 1, [1000, 1000], [2000, 16], 1500),
    (512, 1, 3, 1, [2000, 2000], [3999, 3], 100),
    (256, 1, 16, 1, [20000, 17000], [36992, 16], 20000),                 # a cluster's
    (256, 8, 16, 2, [1100] * 20, [16] * 19 + [21776], 5000),
])
def test_captured_choice_of_grown_requests(D, hkv, ps, layers, before, after, budget):
    s = torch.cuda.Stream()
    every = list(range(layers))
    with torch.cuda.stream(s):
        c = Case(D, hkv, hkv, [1] * len(before), np.array(before) - 1, ps=ps, layers=layers, seed=budget,
                 stream=s)
        c.build()
        src = torch.full((layers, len(before), hkv, budget), -1, dtype=torch.int32, device="cuda")

        def call():
            pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, layers, budget, 3, 40, src, s))
            pg.check(pg.pg_kv_evict_apply(c.plan, c.desc, c.stats, 0, layers, budget, src, s))

        g = capture(call, s)
        for turn, n in enumerate((after, before)):
            replan(c, [1] * len(n), np.array(n) - 1, turn)
            refill(c, turn)
            c.pool.copy_(c.pool_cpu)
            src.fill_(-99)
            g.replay()
            s.synchronize()
            assert pg.pg_device_status(s) == pg.PG_OK
            want = select_reference(c, budget, 3, 40, c.mass_cpu.numpy(), c.pos_cpu.numpy(), every)
            assert (src.cpu().numpy() == want).all()
            pool, mass, pos = apply_reference(c, want, every, c.pool_cpu, c.mass_cpu, c.pos_cpu)
            assert torch.equal(c.pool.view(torch.int16).cpu(), pool.view(torch.int16))
            assert torch.equal(c.mass.cpu(), mass) and torch.equal(c.pos.cpu(), pos)
    c.close()


@pytest.mark.parametrize("D,hq,hkv", [(256, 4, 2), (256, 16, 8), (512, 4, 1), (512, 16, 1)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (900, 70)])
@pytest.mark.parametrize("ps,before,after", [
    (5, [600, 600], [1195, 5]),                # more chunks than the launch has
    (1, [40, 300, 20], [2, 355, 3]),
    (3, [30, 30, 30], [33, 27, 30]),
    (16, [600, 600], [1200, 16]),
    (256, [200, 300], [256, 500]),
])
def test_captured_token_weights_follow_the_plan(D, hq, hkv, window, sinks, ps, before, after):
    one = [1] * len(before)
    replayed_weights(D, hq, hkv, ps, [(one, before), (one, after)], window, sinks)


def replayed_windowed(D, hq, hkv, ps, shapes, window):
    """replayed_weights, with the entries that have neither sinks nor weights."""
    fn = pg.pg_attn_paged_prefill_lse if D == 256 else pg.pg_attn_paged_prefill_hd512_lse
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        qo, n = shapes[0]
        c = Case(D, hq, hkv, qo, np.array(n) - qo, ps=ps, seed=ps, stream=s).build()
        nb = pg.pg_workspace_bytes(c.plan)

        def call():
            pg.check(fn(c.plan, c.desc, 0, c.q, c.out, c.lse, window, 1.0, c.ws, nb, s))

        g = capture(call, s)
        for turn, (qo, n) in enumerate([*shapes[1:], *shapes]):
            replan(c, qo, np.array(n) - qo, turn)
            c.out.fill_(float("nan"))
            c.lse.fill_(float("nan"))
            c.ws.fill_(0xFF)
            g.replay()
            s.synchronize()
            assert pg.pg_device_status(s) == pg.PG_OK
            out, lse, _, _, wabs = c.reference(window, 0)
            # (these entries sum the rounded weights: each within half a step of its own, so the sum
            # is, and with it lse, which is off by at most 2^-8 more than bounded_ref.py says)
            got = c.out.double().cpu().numpy()
            assert (np.abs(got - out) <= 2.0 ** -8 * (2 * wabs + np.abs(out)) + c.e * wabs + 1e-30).all()
            got = c.lse.double().cpu().numpy()
            assert (np.abs(got - lse) <= 2.0 ** -8 + c.e + 2.0 ** -22 * np.abs(lse)).all()
    c.close()


@pytest.mark.parametrize("D,hq,hkv", [(256, 4, 2), (512, 4, 1)])
@pytest.mark.parametrize("window", [-1, 900])
@pytest.mark.parametrize("ps,before,after", [(5, [600, 600], [1195, 5]), (1, [40, 300, 20], [2, 355, 3]),
                                             (16, [600, 600], [1200, 16])])
def test_captured_windowed_decode_follows_the_plan(D, hq, hkv, window, ps, before, after):
    """The decode form of other page sizes than the tensor cores' has the same chunks."""
    one = [1] * len(before)
    replayed_windowed(D, hq, hkv, ps, [(one, before), (one, after)], window)


# ([tokens], [keys]) captured and replayed: other requests hold the prompt's tokens, so it has more or
# fewer query tiles
SPREAD = [
    (16, ([256, 256], [300, 300]), ([511, 1], [520, 70])),
    (16, ([1, 1, 200], [16, 16, 208]), ([66, 68, 68], [80, 70, 75])),
    (16, ([130, 2], [140, 300]), ([2, 130], [300, 130])),
    (64, ([300] + [1] * 9, [700] + [60] * 9), ([30] * 9 + [39], [64] * 9 + [690])),
    (5, ([33, 33, 33], [40, 40, 40]), ([97, 1, 1], [110, 5, 3])),
    (1, ([120, 1], [200, 1]), ([60, 61], [100, 101])),
]


@pytest.mark.parametrize("D,hq,hkv", [(256, 16, 8), (256, 4, 1), (512, 16, 1), (512, 2, 2)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (90, 5)])
@pytest.mark.parametrize("ps,before,after", SPREAD)
def test_captured_prompt_weights_of_other_lengths(D, hq, hkv, window, sinks, ps, before, after):
    replayed_weights(D, hq, hkv, ps, [before, after], window, sinks)
    replayed_weights(D, hq, hkv, ps, [after, before], window, sinks)


@pytest.mark.parametrize("D,hq,hkv", [(256, 16, 8), (512, 16, 1)])
@pytest.mark.parametrize("ps,before,after", SPREAD)
def test_captured_windowed_prompts_of_other_lengths(D, hq, hkv, ps, before, after):
    replayed_windowed(D, hq, hkv, ps, [before, after], 90)
    replayed_windowed(D, hq, hkv, ps, [after, before], -1)


def test_a_plan_of_as_many_tokens_keeps_its_layout():
    """Whatever the spread of 600 tokens over 7 requests, page sizes of both kernel families."""
    g = np.random.Generator(np.random.PCG64(1))
    for D, hq, hkv, ps in ((256, 16, 8, 16), (512, 16, 1, 8), (256, 4, 2, 5), (512, 2, 1, 1)):
        sizes = set()
        plan = None
        for turn in range(40):
            cut = np.sort(g.choice(np.arange(1, 600), 6, replace=False))
            qo = np.concatenate([[0], cut, [600]])
            n = np.diff(qo)
            npg = -(-n // ps)
            spare = 640 - int(npg.sum())
            # (as many pages too: the first request's earlier keys fill them)
            npg[0] += spare
            start = np.zeros(7, np.int64)
            start[0] = spare * ps
            last = (n + start - (npg - 1) * ps).astype(np.int32)
            indptr = np.concatenate([[0], np.cumsum(npg)])
            rc, plan = pg.pg_plan_paged_prefill(plan, 7, qo, indptr, np.arange(640, dtype=np.int32), last, start,
                                                hq, hkv, D, ps)
            pg.check(rc)
            info = plan.info()
            sizes.add((info.metadata_bytes, info.d_page_ids))
            tile = info.cta_tile_q
            assert info.num_work == sum(-(-int(x) // tile) for x in n)
        assert len(sizes) == 1
        plan.close()


@pytest.mark.parametrize("D,hq,hkv,ps", [(256, 16, 8, 16), (256, 4, 2, 5), (512, 16, 1, 16), (512, 4, 1, 3)])
@pytest.mark.parametrize("shapes", [([200, 3, 60], [2, 250, 11]), ([1, 1, 261], [88, 88, 87])])
def test_captured_ring_prompts_of_other_lengths(D, hq, hkv, ps, shapes):
    """A ring plan's tables have the same room: the replay equals the eager call under the updated plan."""
    window, s = 100, torch.cuda.Stream()
    g = np.random.Generator(np.random.PCG64(D + ps))
    held = -(-(window + 261) // ps)  # pages a ring
    with torch.cuda.stream(s):
        pool = torch.randn((1, 3 * held, 2, hkv, ps, D), device="cuda", dtype=torch.bfloat16)
        q = torch.randn((sum(shapes[0]), hq, D), device="cuda", dtype=torch.bfloat16) / D ** 0.5
        outs = [torch.empty_like(q) for _ in range(2)]
        desc, plan, graph = pg.pool_descriptor(pool), None, None
        fn = pg.pg_attn_paged_prefill if D == 256 else pg.pg_attn_paged_prefill_hd512
        for turn, qo in enumerate([*shapes, *shapes]):
            rc, plan = pg.pg_plan_paged_prefill_ring(
                plan, 3, np.concatenate([[0], np.cumsum(qo)]), np.arange(4) * held,
                g.permutation(3 * held).astype(np.int32), g.integers(0, 5000, 3), hq, hkv, D, ps, window, s)
            pg.check(rc)

            def call(out):
                pg.check(fn(plan, desc, 0, q, out, window, 1.0, None, 0, s))

            outs[0].fill_(float("nan"))
            call(outs[0])
            if graph is None:
                s.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    call(outs[1])
            outs[1].fill_(float("nan"))
            graph.replay()
            s.synchronize()
            assert pg.pg_device_status(s) == pg.PG_OK
            assert torch.isfinite(outs[0].float()).all()
            assert torch.equal(outs[0], outs[1])
        plan.close()
