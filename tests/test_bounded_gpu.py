"""Bounded-cache operators against a plain 64-bit reference (GPU): attention with sink tokens,
accumulated attention weights, eviction. The tolerances are derived in bounded_ref.py."""
import numpy as np
import pytest
import torch

from bounded_ref import Case, apply_reference, select_reference
from paged_sliding_window_qkv_gb300 import pg

pytestmark = pytest.mark.gpu

HEADS = {256: [(16, 8), (8, 8), (16, 1), (8, 2)], 512: [(16, 1), (8, 1), (4, 2), (2, 2)]}


def ok():
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK


# ------------------------------------------------------------------ sinks
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 1), (5, 4), (63, 64), (100, 3), (100, 700),
                                          (-1, 9), (2000, 4)])
def test_sink_prefill(D, window, sinks):
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    c = Case(D, hq, hkv, [1, 2, 333, 64, 130], [0, 700, 0, 511, 90], seed=window + sinks).build()
    c.sink(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("ps", [1, 3, 4, 8, 32, 64, 128])
def test_sink_prefill_page_sizes(D, ps):
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    c = Case(D, hq, hkv, [77, 200], [300, 0], ps=ps, seed=ps).build()
    c.sink(50, 20)
    ok()
    c.reference(50, 20)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D,hq,hkv", [(d, *h) for d in (256, 512) for h in HEADS[d]])
def test_sink_head_groups(D, hq, hkv):
    for qo in ([70, 41], [1, 1, 1]):
        start = [210, 0] if len(qo) == 2 else [210, 0, 33]
        c = Case(D, hq, hkv, qo, start, seed=hq + hkv, layers=2, layer=1).build()
        c.sink(60, 5)
        ok()
        c.reference(60, 5)
        c.check_attention(f"{D} {hq}/{hkv} {qo}")
        c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 2), (15, 16), (100, 5), (1023, 4), (-1, 0),
                                          (300, 5000)])
def test_sink_decode(D, window, sinks):
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    start = [0, 1, 15, 16, 31, 32, 100, 511, 1500, 2222]
    c = Case(D, hq, hkv, [1] * len(start), start, seed=window + 2 * sinks + 1).build()
    c.sink(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("ps", [1, 2, 5, 8, 64])
def test_sink_decode_page_sizes(D, ps):
    hq, hkv = (16, 8) if D == 256 else (8, 1)
    c = Case(D, hq, hkv, [1] * 4, [0, 40, 333, 700], ps=ps, seed=ps).build()
    c.sink(50, 20)
    ok()
    c.reference(50, 20)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_sink_segments_and_empty_rows(D):
    """Sinks are absolute positions: a segment past them has none, and rows may see nothing."""
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    for qo, start in (([40, 3], [200, 90]), ([1, 1], [200, 90])):
        held = [60, 50]  # positions [0, 60) and [30, 80): before most windows
        c = Case(D, hq, hkv, qo, start, evicted=[0, 30], held=held, seed=4).build()
        for window, sinks in ((20, 8), (20, 33), (145, 0), (3, 0)):
            c.upload()
            c.sink(window, sinks)
            ok()
            c.reference(window, sinks)
            c.check_attention(f"{qo} {window} {sinks}")
        c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("scale", [0.0, -1.0, 0.25])
def test_sink_scales(D, scale):
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    for qo, start in (([90], [100]), ([1, 1], [100, 44])):
        c = Case(D, hq, hkv, qo, start, seed=3).build()
        c.sink(40, 6, scale)
        ok()
        c.reference(40, 6, scale)
        c.check_attention()
        c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sink_hidden_keys_may_hold_anything(D, bad):
    """Keys between the sinks and the window, and slots behind the last key, are not read (or act
    as zero): decode to the key, prefill to the tile."""
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    c = Case(D, hq, hkv, [1, 1], [500, 77], seed=8)
    for r, (a, b) in enumerate(((4, 500 - 100), (4, 77 - 60))):
        page, off = c.rows_of(r)
        c.pool_cpu[0, page[a:b], :, :, off[a:b]] = bad
    for r in range(2):  # behind the last key of the last page
        last = c.ids[c.pg_indptr[r + 1] - 1]
        c.pool_cpu[0, last, :, :, c.last[r]:] = bad
    c.build()
    for window in (60,):
        c.sink(window, 4)
        ok()
        c.reference(window, 4)
        c.check_attention()
    c.close()
    # prefill: the hidden keys fill whole tiles of 64
    c = Case(D, hq, hkv, [30], [640], seed=9)
    page, off = c.rows_of(0)
    c.pool_cpu[0, page[64:512], :, :, off[64:512]] = bad
    c.pool_cpu[0, c.ids[-1], :, :, c.last[0]:] = bad
    c.build()
    c.sink(640 - 512, 64)
    ok()
    c.reference(640 - 512, 64)
    c.check_attention()
    c.close()


def test_sink_matches_the_windowed_entry():
    c = Case(256, 16, 8, [300, 20], [0, 900], seed=5).build()
    c.sink(100, 0)
    a = c.out.clone()
    pg.check(pg.pg_attn_paged_prefill(c.plan, c.desc, 0, c.q, c.out, 100, 1.0))
    ok()
    assert (a.float() - c.out.float()).abs().max() <= 2.0 ** -6  # two bf16 roundings of |out| < 4
    c.close()


# ------------------------------------------------------------------ accumulated weights
@pytest.mark.parametrize("D,hq,hkv", [(256, 16, 8), (256, 8, 1), (512, 16, 1), (512, 4, 2)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 4), (0, 0)])
def test_mass_prefill(D, hq, hkv, window, sinks):
    c = Case(D, hq, hkv, [1, 333, 64, 130, 5], [0, 0, 511, 90, 1000], seed=window + hq).build()
    c.weigh(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.check_mass()
    # the weights of a row sum to one: a head's mass gained is the rows that see something
    c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("ps", [1, 3, 8, 32, 64, 256])
def test_mass_page_sizes(D, ps):
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    for qo, start in (([77, 200], [300, 0]), ([1, 1, 1], [300, 0, 63])):
        c = Case(D, hq, hkv, qo, start, ps=ps, seed=ps, layers=2, layer=1).build()
        c.weigh()
        ok()
        c.reference(-1, 0)
        c.check_attention()
        c.check_mass(f"{qo}")
        c.close()


@pytest.mark.parametrize("D,hq,hkv", [(256, 16, 8), (256, 16, 1), (512, 16, 1), (512, 2, 2)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 4)])
def test_mass_decode(D, hq, hkv, window, sinks):
    start = [0, 1, 15, 16, 255, 256, 700, 1500, 2222]
    c = Case(D, hq, hkv, [1] * len(start), start, seed=hq + window).build()
    c.weigh(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.check_mass()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_mass_long_prefill(D):
    """Enough query rows that their range is cut, a ragged batch beside them."""
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    c = Case(D, hq, hkv, [1400, 3, 700], [100, 2000, 0], seed=6).build()
    c.weigh()
    ok()
    c.reference(-1, 0)
    c.check_attention()
    c.check_mass()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_mass_repeats_bit_for_bit(D):
    hq, hkv = (16, 8) if D == 256 else (16, 1)
    for qo, start in (([600, 3], [0, 100]), ([1] * 5, [9, 2000, 77, 1024, 5])):
        c = Case(D, hq, hkv, qo, start, seed=7).build()
        got = []
        for _ in range(2):
            c.upload()
            c.weigh()
            ok()
            got.append((c.out.clone(), c.lse.clone(), c.mass.clone()))
        for a, b in zip(*got):
            assert torch.equal(a, b)
        c.close()


# ------------------------------------------------------------------ eviction
def _scramble(c, seed, evicted=0):
    """Positions as earlier evictions leave them, and masses with ties, zeros and odd values."""
    g = np.random.Generator(np.random.PCG64(seed))
    pos, mass = c.pos_cpu.numpy(), c.mass_cpu.numpy()
    for layer in range(c.layers):
        for r in range(len(c.qo)):
            page, off = c.rows_of(r)
            end = int(c.start[r] + c.qo[r])
            for h in range(c.hkv):
                p = g.permutation(g.choice(end, size=int(c.n[r]), replace=False))
                pos[layer, page, h, off] = p
                m = g.exponential(1.0, int(c.n[r])).astype(np.float32)
                m[g.random(len(m)) < 0.2] = 0.0
                m[g.random(len(m)) < 0.2] = 0.5
                m[g.random(len(m)) < 0.02] = np.nan
                m[g.random(len(m)) < 0.02] = np.inf
                m[g.random(len(m)) < 0.02] = -0.0
                m[g.random(len(m)) < 0.02] = -1.0
                mass[layer, page, h, off] = m


@pytest.mark.parametrize("D,hkv,ps", [(512, 1, 16), (256, 8, 16), (512, 2, 1), (256, 2, 5), (256, 1, 64)])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (7, 2, 3), (64, 4, 60), (300, 4, 100),
                                                 (1023, 0, 0), (1024, 4, 16), (2100, 4, 8)])
def test_evict(D, hkv, ps, budget, sinks, recent):
    n = [1, 2, 63, 64, 301, 1025, 2099]
    start = [x + 40 - 1 for x in n]
    c = Case(D, hkv, hkv, [1] * len(n), start, ps=ps, evicted=40, layers=3, seed=budget)
    _scramble(c, budget)
    c.build()
    layers = [1, 2]
    src = torch.full((2, len(n), hkv, budget), -99, dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 1, 2, budget, sinks, recent, src))
    ok()
    want = select_reference(c, budget, sinks, recent, c.mass_cpu.numpy(), c.pos_cpu.numpy(), layers)
    got = src.cpu().numpy()
    assert (got == want).all(), np.argwhere(got != want)[:5].tolist()
    assert torch.equal(c.mass.view(torch.int32).cpu(), c.mass_cpu.view(torch.int32))
    pool, mass, pos = apply_reference(c, want, layers, c.pool_cpu, c.mass_cpu, c.pos_cpu)
    for _ in range(2):  # a repeated call changes nothing
        pg.check(pg.pg_kv_evict_apply(c.plan, c.desc, c.stats, 1, 2, budget, src))
        ok()
        assert torch.equal(c.pool.view(torch.int16).cpu(), pool.view(torch.int16))
        assert torch.equal(c.mass.view(torch.int32).cpu(), mass.view(torch.int32))
        assert torch.equal(c.pos.cpu(), pos)
    c.close()


@pytest.mark.parametrize("n,budget", [(20000, 12345), (40000, 39999), (70000, 100), (9000, 8999), (140000, 70000)])
def test_evict_long(n, budget):
    c = Case(256, 1, 1, [1, 1], [n - 1, n - 700], seed=n)
    _scramble(c, n)
    c.build()
    src = torch.full((1, 2, 1, budget), -99, dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 1, budget, 4, 90, src))
    ok()
    want = select_reference(c, budget, 4, 90, c.mass_cpu.numpy(), c.pos_cpu.numpy(), [0])
    assert (src.cpu().numpy() == want).all()
    c.close()


@pytest.mark.parametrize("n,keep", [(2048, 1000), (5000, 1), (8192, 4096), (8193, 8192), (16384, 5000), (16384, 9),
                                    (30000, 20000)])
@pytest.mark.parametrize("masses", ["distinct", "rising", "falling", "two", "zeros", "wide", "first of four low",
                                    "first of four high", "recent"])
def test_evict_orders(n, keep, masses):
    """Masses whose order follows the slots, ties at the cut, and some whose fourth slots tell nothing of
    the others."""
    R = 2
    c = Case(256, 1, 1, [1] * R, [n - 1, n - 10], seed=n + keep)
    g = np.random.Generator(np.random.PCG64(keep))
    mass, pos = c.mass_cpu.numpy(), c.pos_cpu.numpy()
    for r in range(R):
        page, off = c.rows_of(r)
        k, s = int(c.n[r]), np.arange(int(c.n[r]))
        m = g.exponential(1.0, k)
        if masses in ("rising", "falling"):
            m = np.sort(m) if masses == "rising" else np.sort(m)[::-1]
        elif masses == "two":
            m = np.where(g.random(k) < 0.5, 1.0, np.nextafter(np.float32(1), np.float32(2)))
        elif masses == "zeros":
            m = np.where(g.random(k) < 0.1, m, 0.0)
        elif masses == "wide":
            m = np.exp2(g.uniform(-120, 120, k))
        elif masses.startswith("first"):
            m = np.where(s % 4 == 0, m * (1e-3 if masses.endswith("low") else 1e3), m)
        mass[0, page, 0, off] = m.astype(np.float32)
        pos[0, page, 0, off] = g.permutation(k)
    c.build()
    recent = keep if masses == "recent" else 0
    src = torch.full((1, R, 1, keep), -99, dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 1, keep, 0, recent, src))
    ok()
    want = select_reference(c, keep, 0, recent, mass, pos, [0])
    assert (src.cpu().numpy() == want).all()
    c.close()


@pytest.mark.parametrize("n,budget", [(2048, 700), (2049, 2000), (4100, 4096), (8192, 33), (9000, 4000)])
def test_evict_many_segments(n, budget):
    R, hkv = 20, 2
    c = Case(256, hkv, hkv, [1] * R, [max(1, n - 97 * r) - 1 for r in range(R)], layers=9, ps=64, seed=n)
    _scramble(c, n)
    c.build()
    src = torch.full((9, R, hkv, budget), -99, dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 9, budget, 3, 20, src))
    ok()
    want = select_reference(c, budget, 3, 20, c.mass_cpu.numpy(), c.pos_cpu.numpy(), list(range(9)))
    assert (src.cpu().numpy() == want).all()
    c.close()


def test_evict_apply_many_segments():
    R, layers, n, budget = 61, 20, 1100, 1030
    c = Case(256, 1, 1, [1] * R, [n - 1 - r for r in range(R)], layers=layers, ps=64, seed=61)
    _scramble(c, 61)
    c.build()
    src = torch.full((layers, R, 1, budget), -99, dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, layers, budget, 4, 20, src))
    pg.check(pg.pg_kv_evict_apply(c.plan, c.desc, c.stats, 0, layers, budget, src))
    ok()
    every = list(range(layers))
    want = select_reference(c, budget, 4, 20, c.mass_cpu.numpy(), c.pos_cpu.numpy(), every)
    assert (src.cpu().numpy() == want).all()
    pool, mass, pos = apply_reference(c, want, every, c.pool_cpu, c.mass_cpu, c.pos_cpu)
    assert torch.equal(c.pool.view(torch.int16).cpu(), pool.view(torch.int16))
    assert torch.equal(c.mass.view(torch.int32).cpu(), mass.view(torch.int32))
    assert torch.equal(c.pos.cpu(), pos)
    c.close()


@pytest.mark.parametrize("D,n,budget", [(256, 1055, 1030), (512, 2304, 2299), (512, 2600, 2520)])
def test_evict_apply_few_moves(D, n, budget):
    """Next to none of the kept keys move, in more segments than a wave of small blocks."""
    R, layers = 41, 4
    c = Case(D, 1, 1, [1] * R, [n - 1 - r for r in range(R)], layers=layers, ps=32, seed=n)
    _scramble(c, n)
    c.build()
    src = torch.full((layers, R, 1, budget), -99, dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, layers, budget, 4, 20, src))
    pg.check(pg.pg_kv_evict_apply(c.plan, c.desc, c.stats, 0, layers, budget, src))
    ok()
    every = list(range(layers))
    want = select_reference(c, budget, 4, 20, c.mass_cpu.numpy(), c.pos_cpu.numpy(), every)
    assert (src.cpu().numpy() == want).all()
    pool, mass, pos = apply_reference(c, want, every, c.pool_cpu, c.mass_cpu, c.pos_cpu)
    assert torch.equal(c.pool.view(torch.int16).cpu(), pool.view(torch.int16))
    assert torch.equal(c.mass.view(torch.int32).cpu(), mass.view(torch.int32))
    assert torch.equal(c.pos.cpu(), pos)
    c.close()


@pytest.mark.parametrize("n", [4, 129, 512, 513, 1024])
@pytest.mark.parametrize("part", [0.02, 0.5, 0.98])
@pytest.mark.parametrize("ps", [3, 16])
def test_evict_short(n, part, ps):
    lens = sorted({1, 2, n // 3 + 1, n - 1, n})
    keep = max(1, int(n * part))
    c = Case(256, 2, 2, [1] * len(lens), [x - 1 for x in lens], ps=ps, layers=2, seed=n)
    _scramble(c, n + keep)
    c.build()
    src = torch.full((2, len(lens), 2, keep), -99, dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 2, keep, 0, keep // 3, src))
    ok()
    want = select_reference(c, keep, 0, keep // 3, c.mass_cpu.numpy(), c.pos_cpu.numpy(), [0, 1])
    assert (src.cpu().numpy() == want).all()
    c.close()


def test_evict_all_equal_masses():
    """Every key ties: the lower slots stay."""
    c = Case(512, 1, 1, [1], [999], seed=1)
    c.mass_cpu.fill_(0.25)
    c.pos_cpu[0, c.rows_of(0)[0], 0, c.rows_of(0)[1]] = torch.arange(1000, dtype=torch.int32)
    c.build()
    src = torch.empty((1, 1, 1, 500), dtype=torch.int32, device="cuda")
    pg.check(pg.pg_kv_evict_select(c.plan, c.stats, 0, 1, 500, 0, 10, src))
    ok()
    want = np.arange(500)
    want[490:] = np.arange(990, 1000)
    assert (src.cpu().numpy().ravel() == want).all()
    c.close()


def test_evict_apply_skips_what_select_does_not_give():
    c = Case(256, 2, 2, [1], [99], seed=2).build()
    src = torch.arange(50, dtype=torch.int32, device="cuda").repeat(1, 1, 2, 1)
    src[0, 0, 0, 3], src[0, 0, 0, 4], src[0, 0, 1, 5] = 7, 100, 1 << 30
    pg.check(pg.pg_kv_evict_apply(c.plan, c.desc, c.stats, 0, 1, 50, src))
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_ERR_DEVICE_BOUNDS
    assert torch.equal(c.pool.cpu(), c.pool_cpu) and torch.equal(c.mass.cpu(), c.mass_cpu)
    c.close()
