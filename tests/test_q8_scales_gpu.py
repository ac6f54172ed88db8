"""Scale bytes that prep does not write (GPU): 0 is 2^-127, 255 NaN, in the read-back and in attention."""
import numpy as np
import pytest
import torch

from paged_sliding_window_qkv_gb300 import pg
from q8_ref import Q8Case, values

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK


@pytest.mark.parametrize("D", [256, 512])
def test_read_back(D):
    """All codes: the element in 64 bits, rounded once."""
    c = Q8Case(D, 2, 1, [1], [63], seed=1)
    c.codes_cpu[:] = torch.arange(D, dtype=torch.int32).remainder(256).to(torch.uint8)
    b = torch.tensor([0, 1, 2, 3, 16, 17, 247, 248, 253, 254, 255], dtype=torch.uint8)
    c.scales_cpu[:] = b[torch.arange(c.scales_cpu.numel()) % len(b)].reshape(c.scales_cpu.shape)
    c.build()
    dst = torch.zeros(c.pool.shape, dtype=torch.bfloat16, device="cuda")
    pg.check(pg.pg_kv_dequantize(c.plan, c.q8, pg.pool_descriptor(dst), 0, 1))
    ok()
    page, off = (torch.from_numpy(x) for x in c.rows_of(0))
    v = values(c.codes_cpu, c.scales_cpu)
    v[c.scales_cpu == 255] = torch.nan
    want, got = v.to(torch.bfloat16)[0][page, :, :, off].float(), dst[0].cpu()[page, :, :, off].float()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, 0.0, 1e39, -1e39), torch.nan_to_num(want, 0.0, 1e39, -1e39))
    c.close()


@pytest.mark.parametrize("D,hq,hkv", [(256, 16, 8), (256, 16, 1), (512, 16, 1), (512, 4, 1)])
@pytest.mark.parametrize("ps", [8, 16])
@pytest.mark.parametrize("qo", [1, 20])
@pytest.mark.parametrize("kv", [0, 1])
def test_rows_that_see_a_byte_of_255(D, hq, hkv, ps, qo, kv):
    c = Q8Case(D, hq, hkv, [qo, qo], [300, 200], ps=ps, seed=D + ps)
    page, off = c.rows_of(0)
    key = 77
    c.scales_cpu[0, page[key], kv, :, off[key]] = 255
    c.build()
    c.attend()
    ok()
    assert torch.isnan(c.out[:qo]).all()
    assert torch.isnan(c.lse[:qo]).all() if kv == 0 else torch.isfinite(c.lse[:qo]).all()
    c.reference()
    c.check_attention(rows=np.arange(qo, 2 * qo))
    c.close()


@pytest.mark.parametrize("D,hq,hkv", [(256, 16, 8), (512, 16, 1)])
def test_bytes_of_zero_in_attention(D, hq, hkv):
    """Rows of some 2^-120: scores of zero, and V rows that add nothing beside others."""
    c = Q8Case(D, hq, hkv, [1, 1], [300, 0], seed=D)
    page, off = c.rows_of(0)
    c.scales_cpu[0, page[40:90], :, :, off[40:90]] = 0
    page1, off1 = c.rows_of(1)
    c.scales_cpu[0, page1[0], 1, :, off1[0]] = 0  # the only V row of the second request
    c.pool_cpu = values(c.codes_cpu, c.scales_cpu).to(torch.bfloat16)
    c.build()
    c.attend()
    ok()
    c.reference()
    c.check_attention(rows=np.arange(1))
    want = c.pool_cpu[0, page1[0], 1, :, off1[0]].double().repeat_interleave(hq // hkv, 0)
    assert (c.out[1].cpu().double() - want).abs().max() <= 2.0 ** -130  # (a step of bf16 there is 2^-133)
    assert want.abs().max() > 2.0 ** -121
    c.close()
