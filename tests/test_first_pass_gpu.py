"""First passes on new tensors (GPU): caches swept in between, so that code, page tables and data come
from memory and warps run far apart. Each call leaves no error, and its second pass gives the same bits."""
import numpy as np
import pytest
import torch

from bounded_ref import Case
from paged_sliding_window_qkv_gb300 import pg

pytestmark = pytest.mark.gpu


def sweep():
    torch.empty(96 << 20, dtype=torch.float32, device="cuda").normal_()  # three times the L2
    torch.cuda.empty_cache()
    torch.cuda.synchronize()


def codes(shape, g):
    """Random finite e4m3 codes, scales of about one."""
    c = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
    c[(c & 0x7F) == 0x7F] = 0
    return c, torch.randint(117, 122, shape[:-1], dtype=torch.uint8, device="cuda", generator=g)


def twice(call, outs):
    call()
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK
    first = [x.clone() for x in outs]
    call()
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(first, outs))


@pytest.mark.parametrize("D,hq,hkv", [(512, 16, 1), (256, 16, 8)])
@pytest.mark.parametrize("round_", range(4))
def test_ragged_prompts(D, hq, hkv, round_):
    r = np.random.RandomState(round_ + D)
    c = Case(D, hq, hkv, r.randint(100, 513, 4), r.randint(0, 3001, 4), seed=round_).build()
    sweep()
    twice(lambda: c.sink(-1, 0), [c.out, c.lse])
    sweep()
    twice(lambda: c.sink(700, 4), [c.out, c.lse])
    c.close()


@pytest.mark.parametrize("round_", range(4))
def test_chunks_over_8_bit_caches(round_):
    r = np.random.RandomState(round_)
    g = torch.Generator(device="cuda").manual_seed(round_)
    D, hq, ps = 512, 16, 16
    qo, start = r.randint(100, 513, 4), r.randint(0, 8001, 4)
    n = start + qo
    npg = -(-n // ps)
    ind, qi = (np.concatenate([[0], np.cumsum(x)]) for x in (npg, qo))
    ids = r.permutation(int(ind[-1])).astype(np.int32)
    rc, plan = pg.pg_plan_paged_prefill(None, 4, qi, ind, ids, (n - (npg - 1) * ps).astype(np.int32), start, hq, 1, D, ps)
    pg.check(rc)
    c, s = codes((1, int(ind[-1]), 2, 1, ps, D), g)
    pool = pg.q8_descriptor(c, s)
    T = int(qi[-1])
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda").normal_(0, 0.001, generator=g)
    out, lse = torch.zeros_like(q), torch.zeros((T, hq), device="cuda")
    ws = torch.empty(pg.pg_q8_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    sweep()
    twice(lambda: pg.check(pg.pg_attn_paged_q8(plan, pool, 0, q, out, lse, -1, 0, 1.0, ws, ws.numel())), [out, lse])
    plan.close()
