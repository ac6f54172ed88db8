"""The form that a shared plan takes for decode steps over 8-bit pools (GPU), told by its launches: where either
form takes more than 1.3 times the other's time, on pages that the decode on codes takes and on others."""
import numpy as np
import pytest
import torch

from paged_sliding_window_qkv_gb300 import pg

pytestmark = pytest.mark.gpu

# launches: the read-back of the prefixes, their parts, decode and its join; pages of 8 slots: own keys over a
# read-back of theirs, and a join of their own. The plain walk: decode and its join, there behind a read-back.
PARTS, PLAIN = {8: 6, 16: 4, 64: 4}, {8: 3, 16: 2, 64: 2}


@pytest.mark.parametrize("D,hq,hkv,R,prefix,own,ps,parts", [
    (256, 16, 8, 16, 2048, 100, 8, True),     # 48 us against 113: the plain walk reads 16 prefixes back
    (256, 16, 8, 64, 512, 100, 8, True),
    (512, 16, 1, 16, 8192, 1000, 8, True),
    (512, 16, 1, 4, 2048, 100, 8, False),     # 46 against 21
    (256, 16, 8, 64, 2048, 100, 16, True),    # 30 against 51
    (512, 16, 1, 64, 8192, 1000, 64, True),   # 65 against 83
    (512, 16, 1, 16, 8192, 1000, 64, False),  # 43 against 32: a page of 64 slots is a long read-back
    (512, 8, 1, 1, 8192, 1000, 64, False),
])
def test_form(D, hq, hkv, R, prefix, own, ps, parts):
    n = np.full(R, prefix + own)
    npg = -(-n // ps)
    ind = np.concatenate([[0], np.cumsum(npg)])
    ids = np.random.RandomState(R).permutation(int(ind[-1])).astype(np.int32)
    for r in range(1, R):
        ids[ind[r]:ind[r] + prefix // ps] = ids[:prefix // ps]
    rc, plan = pg.pg_plan_paged_shared(None, R, np.arange(R + 1), ind, ids, n - (npg - 1) * ps, n - 1, 1, [0, R],
                                       [prefix], hq, hkv, D, ps)
    pg.check(rc)
    g = torch.Generator(device="cuda").manual_seed(R)
    c = torch.randint(0, 120, (1, int(ind[-1]), 2, hkv, ps, D), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.full(c.shape[:-1], 119, dtype=torch.uint8, device="cuda")
    q = torch.empty((R, hq, D), dtype=torch.bfloat16, device="cuda").normal_(0, 0.02, generator=g)
    outs, lses = [], []
    pool = pg.q8_descriptor(c, s)
    size = max(pg.pg_shared_q8_workspace_bytes(plan), pg.pg_q8_workspace_bytes(plan))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for shared in (True, False):
        outs.append(torch.full_like(q, float("nan")))
        lses.append(torch.full((R, hq), float("nan"), device="cuda"))
        before = pg.pg_launch_count()
        if shared:
            pg.check(pg.pg_attn_paged_shared_q8(plan, pool, 0, q, outs[-1], lses[-1], 1.0, ws, size))
            assert pg.pg_launch_count() - before == (PARTS if parts else PLAIN)[ps]
        else:
            pg.check(pg.pg_attn_paged_q8(plan, pool, 0, q, outs[-1], lses[-1], -1, 0, 1.0, ws, size))
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK
    # codes below 120 are positive, at most 240 * 2^-8: a weight's and an output's bf16 rounding, twice
    top = 240 * 2.0 ** -8
    assert (outs[0].float() - outs[1].float()).abs().max() <= 4 * 2.0 ** -8 * top
    assert (lses[0] - lses[1]).abs().max() <= 2.0 ** -12 * lses[1].abs().max()
    plan.close()
