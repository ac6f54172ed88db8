"""Rows that see a key whose score is not a number: out and lse say so, in every kernel, and rows that
do not see it are untouched (GPU). References and tolerances: bounded_ref.py."""
import numpy as np
import pytest
import torch

from bounded_ref import Case
from paged_sliding_window_qkv_gb300 import pg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,hq,hkv,ps", [(256, 16, 8, 16), (256, 4, 2, 5), (512, 16, 1, 16), (512, 4, 1, 3)])
@pytest.mark.parametrize("qo,start,key", [([40, 30], [100, 700], 110), ([200], [0], 0), ([1, 1, 1], [900, 60, 1800], 75)])
@pytest.mark.parametrize("weights", [False, True])
def test_rows_that_see_a_nan_key(D, hq, hkv, ps, qo, start, key, weights):
    window, sinks = 1000, 0
    c = Case(D, hq, hkv, qo, start, ps=ps, seed=key)
    page, off = c.rows_of(0)
    c.pool_cpu[0, page[key], 0, :, off[key]] = float("nan")
    c.build()
    if weights:
        c.weigh(window, sinks)
    else:
        c.sink(window, sinks)
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK
    req = np.repeat(np.arange(len(qo)), qo)
    p = np.concatenate([s + np.arange(t) for s, t in zip(start, qo)])
    sees = (req == 0) & (p >= key) & (p - key <= window)
    assert sees.any()
    assert np.isnan(c.lse.cpu().numpy()[sees]).all()
    assert np.isnan(c.out.float().cpu().numpy()[sees]).all()
    c.reference(window, sinks)
    c.check_attention(rows=np.flatnonzero(~sees))
    if weights:
        # every key that such a row sees has got a weight that is not a number
        got = c.mass.cpu().numpy()[0]
        j = np.arange(c.n[0])
        row_p = p[sees]
        hit = ((j[None] <= row_p[:, None]) & (row_p[:, None] - j[None] <= window)).any(0)
        assert np.isnan(got[page[hit], :, off[hit]]).all()
        assert np.isfinite(got[page[~hit], :, off[~hit]]).all()
    c.close()
