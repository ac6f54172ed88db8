"""8-bit decode steps whose segments are a tile or two long, with and without hidden keys (GPU): queries of
new segments are converted while earlier tiles' weights are written. References: q8_ref.py."""
import numpy as np
import pytest
import torch

from paged_sliding_window_qkv_gb300 import pg
from q8_ref import Q8Case

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK


# keys: whole tiles of 128 (nothing hidden) and ragged ones, in turn
@pytest.mark.parametrize("D,hq,hkv", [(512, 16, 1), (512, 8, 1), (512, 4, 1), (256, 16, 1), (256, 16, 2), (256, 4, 1), (256, 4, 2)])
@pytest.mark.parametrize("keys", [[128], [128, 256, 128, 130], [128, 128, 128, 128, 128, 100], [384, 1, 128]])
def test_short_segments(D, hq, hkv, keys):
    R = 320 // hkv
    n = np.array((keys * R)[:R])
    c = Q8Case(D, hq, hkv, [1] * R, n - 1, ps=128, seed=len(keys)).build()
    junk = torch.empty(64 << 20, dtype=torch.float32, device="cuda")
    c.attend()
    ok()
    first, lse = c.out.clone(), c.lse.clone()
    c.reference()
    c.check_attention()
    for k in range(12):
        if k % 3 == 0:
            junk.zero_()  # the next step's queries come from memory
        c.attend()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)
    ok()
    c.close()
