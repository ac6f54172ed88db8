"""Workspaces of the decode entries (GPU): the sizes that the entries without sinks ask for, and
pg_attn_paged_sink within them. References and tolerances: bounded_ref.py."""
import numpy as np
import pytest
import torch

from bounded_ref import Case
from paged_sliding_window_qkv_gb300 import pg

pytestmark = pytest.mark.gpu


def decode_plan(D, hq, hkv, ps, R, n):
    npg = -(-n // ps)
    at = np.arange(R + 1, dtype=np.int64)
    rc, plan = pg.pg_plan_paged_prefill(None, R, at, at * npg, np.arange(R * npg, dtype=np.int32),
                                        np.full(R, n - (npg - 1) * ps, np.int32), np.full(R, n - 1, np.int64),
                                        hq, hkv, D, ps)
    pg.check(rc)
    return plan


@pytest.mark.parametrize("ps", [2, 4, 8, 16, 256])
def test_hd256_sizes_do_not_grow_with_the_keys(ps):
    """The streaming kernel's records are counted by its CTAs: one size serves a request of any length."""
    sizes = set()
    for n in (3, 700, 16384):
        plan = decode_plan(256, 16, 8, ps, 4, n)
        sizes.add(pg.pg_workspace_bytes(plan))
        plan.close()
    assert len(sizes) == 1


@pytest.mark.parametrize("D,hq,hkv,ps", [(512, 16, 1, 16), (512, 8, 2, 256), (512, 4, 4, 5), (256, 16, 8, 5),
                                         (256, 8, 1, 1)])
def test_chunked_sizes_are_the_chunks(D, hq, hkv, ps):
    """A partial of D floats, its maximum and its sum for every row and chunk of 512 (256) keys."""
    for R, n in ((1, 8000), (64, 100), (64, 500), (3, 3001)):
        plan = decode_plan(D, hq, hkv, ps, R, n)
        chunks = -(-n // (512 if D == 512 else 256))
        assert pg.pg_workspace_bytes(plan) == R * hq * chunks * (D + 2) * 4
        plan.close()


@pytest.mark.parametrize("D,hq,hkv,ps", [(512, 16, 1, 16), (512, 16, 1, 5), (512, 4, 2, 64), (256, 16, 8, 4),
                                         (256, 4, 4, 2), (256, 16, 8, 16)])
def test_a_decode_loop_keeps_its_buffer(D, hq, hkv, ps):
    """A workspace sized at 100 keys a request serves 500 (a chunk of head_dim 512; head_dim 256: any
    number), with and without sinks."""
    R = 9
    size = None
    fn = pg.pg_attn_paged_prefill if D == 256 else pg.pg_attn_paged_prefill_hd512
    for n in (100, 500):
        c = Case(D, hq, hkv, [1] * R, [n - 1 - 7 * r for r in range(R)], ps=ps, seed=n).build()
        if size is None:
            size = pg.pg_workspace_bytes(c.plan)
            ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        pg.check(fn(c.plan, c.desc, 0, c.q, c.out, 90, 1.0, ws, size))
        out, _, _, _, wabs = c.reference(90, 0)
        got = c.out.double().cpu().numpy()
        assert (np.abs(got - out) <= 2.0 ** -8 * (2 * wabs + np.abs(out)) + c.e * wabs + 1e-30).all()
        c.out.fill_(float("nan"))
        for window, sinks in ((90, 3), (-1, 0)):
            c.out.fill_(float("nan"))
            pg.check(pg.pg_attn_paged_sink(c.plan, c.desc, 0, c.q, c.out, c.lse, window, sinks, 1.0, ws, size))
            torch.cuda.synchronize()
            assert pg.pg_device_status() == pg.PG_OK
            c.reference(window, sinks)
            c.check_attention(f"{n} {window}")
        c.close()
    assert (ws[size:] == 0xFF).all()


@pytest.mark.parametrize("D,hq,hkv,ps,R,top", [(512, 16, 1, 16, 3, 3001), (512, 2, 2, 64, 1, 700), (512, 8, 1, 8, 30, 500),
                                               (256, 4, 4, 2, 160, 900), (256, 8, 8, 4, 80, 900)])
def test_sink_decode_within_either_size(D, hq, hkv, ps, R, top):
    """pg_workspace_bytes and the entry's own, larger size (head_dim 512: another kernel may run), and what
    is between them."""
    g = np.random.Generator(np.random.PCG64(R))
    n = g.integers(1, top, R)
    n[-1] = top
    c = Case(D, hq, hkv, [1] * R, n - 1, ps=ps, seed=R).build()
    least = pg.pg_workspace_bytes(c.plan)
    full = pg.pg_sink_workspace_bytes(c.plan)
    assert least <= full <= max(least, pg.pg_mass_workspace_bytes(c.plan))
    assert full == least if D == 256 else full > least
    for size in sorted({least, (least + full) // 2, (least + 7 * full) // 8, full}):
        for window, sinks in ((600, 5), (-1, 0)):
            ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
            c.out.fill_(float("nan"))
            c.lse.fill_(float("nan"))
            pg.check(pg.pg_attn_paged_sink(c.plan, c.desc, 0, c.q, c.out, c.lse, window, sinks, 1.0, ws, size))
            torch.cuda.synchronize()
            assert pg.pg_device_status() == pg.PG_OK
            c.reference(window, sinks)
            c.check_attention(f"{window}")
            assert (ws[size:] == 0xFF).all()
    c.close()
