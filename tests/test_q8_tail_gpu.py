"""8-bit decode of one dominant key before thousands of equal ones 2^-20 to 2^-25 of it (GPU): the small
weights count together.

Tolerance (derived before the first run). A weight times its V row's scale is the sum of four e4m3 terms under a
reference that puts the row's largest at 2^4 or above: within 2^-16 of itself, or within 2^-26 of that largest. An
element is at most 448 * 2^e with e the row's exponent, so with V rows of ones (e = -8) a key is off by at most
1.75 * 2^-26. n of them: n * 1.75 * 2^-26 + 2^-16 * T, T their weight together; scores round 2^-20 * T; the output
rounds to bf16, 2^-8 of it.
"""
import math

import numpy as np
import pytest
import torch

from paged_sliding_window_qkv_gb300 import pg
from q8_ref import quantise

pytestmark = pytest.mark.gpu


# requests: as many as fill the SMs with one segment each, so that a segment stays whole
@pytest.mark.parametrize("D,hq,R", [(512, 16, 152), (512, 8, 152), (256, 16, 152), (256, 2, 304)])
@pytest.mark.parametrize("n", [16384, 131072])
@pytest.mark.parametrize("octaves", [20.3, 22.7, 24.4])
def test_small_weights_count_together(D, hq, R, n, octaves):
    ps = 128
    y = torch.zeros((1, 2, 2, 1, ps, D))  # page 0: the dominant key first; page 1: small ones alone
    y[0, :, 1, 0, :, 1::2] = 1
    y[0, 0, 0, 0, 0, 0] = 1
    y[0, 0, 1, 0, 0] = 0
    y[0, 0, 1, 0, 0, 0::2] = 1
    codes, scales = (x.cuda() for x in quantise(y))
    pages = n // ps
    ids = np.ones((R, pages), np.int32)
    ids[:, 0] = 0
    rc, plan = pg.pg_plan_paged_prefill(None, R, np.arange(R + 1), np.arange(R + 1) * pages, ids.ravel(),
                                        np.full(R, ps, np.int32), np.full(R, n - 1), hq, 1, D, ps)
    pg.check(rc)
    q = torch.zeros((R, hq, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1
    out = torch.full_like(q, float("nan"))
    lse = torch.full((R, hq), float("nan"), device="cuda")
    ws = torch.empty(pg.pg_q8_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    scale = float(np.float32(octaves * math.log(2)))
    pg.check(pg.pg_attn_paged_q8(plan, pg.q8_descriptor(codes, scales), 0, q, out, lse, -1, 0, scale, ws, ws.numel()))
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK
    T = (n - 1) * math.exp(-scale)
    want = torch.tensor([1.0, T], dtype=torch.float64).repeat(D // 2) / (1 + T)
    tol = 1.75 * n * 2.0 ** -26 + (2.0 ** -16 + 2.0 ** -20) * T + 2.0 ** -8 * want
    err = (out.cpu().double() - want).abs()
    assert (err <= tol).all(), (float(err[..., 0].max()), float(err[..., 1].max()), float(tol[1]))
    assert (lse.cpu().double() - (scale + math.log1p(T))).abs().max() <= 2.0 ** -18 * (1 + scale)
    plan.close()
