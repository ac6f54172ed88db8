"""Prompts of bounded caches at head_dim 512 (GPU): windows and sinks over head groups, page sizes,
segments and captured calls, and long ragged prompts. References and tolerances: bounded_ref.py."""
import pytest
import torch

from bounded_ref import Case
from paged_sliding_window_qkv_gb300 import pg
from test_bounded_replay_gpu import replayed_weights

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK


# groups of 1 to 16; one token, a tile of the plan, one more, and odd ends
@pytest.mark.parametrize("hq,hkv", [(16, 1), (8, 1), (8, 2), (4, 2), (2, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 1), (70, 5), (300, 64), (5000, 3), (70, 0), (-1, 7)])
def test_window_and_sinks_over_head_groups(hq, hkv, window, sinks):
    tile = 128 // (hq // hkv)
    c = Case(512, hq, hkv, [1, tile, tile + 1, 45], [333, 0, 90, 700], seed=hq + window).build()
    c.sink(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("ps", [8, 16, 64, 256])
@pytest.mark.parametrize("window,sinks", [(100, 9), (100, 0), (-1, 0)])
def test_weights_over_page_sizes(ps, window, sinks):
    c = Case(512, 16, 1, [1, 9, 130], [500, 700, 33], ps=ps, seed=ps + sinks).build()
    c.weigh(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.check_mass()
    c.close()


# positions before the first query's window, up to inside its first tile of 64
@pytest.mark.parametrize("ps", [8, 16, 32])
@pytest.mark.parametrize("start", [640, 700, 721])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_pages_before_the_window_may_hold_anything(ps, start, bad):
    window = 100
    c = Case(512, 16, 1, [21], [start], ps=ps, seed=start)
    hidden = (start - window) // ps  # pages none of whose keys any row sees
    c.pool_cpu[0, c.ids[:hidden]] = bad
    c.build()
    c.sink(window, 0)
    ok()
    c.reference(window, 0)
    c.check_attention()
    c.close()


def test_long_ragged_prompts():
    """Prompts of odd lengths behind thousands of keys, as a second chunk has them."""
    for window, sinks in ((-1, 0), (2047, 0)):
        c = Case(512, 16, 1, [257, 13, 101, 3], [3001, 4000, 0, 2222], seed=1).build()
        c.sink(window, sinks)
        ok()
        c.reference(window, sinks)
        c.check_attention()
        c.close()


def test_segments_with_sinks_and_empty_rows():
    held = [60, 50]  # positions [0, 60) and [30, 80)
    c = Case(512, 8, 1, [40, 19], [200, 75], evicted=[0, 30], held=held, seed=4).build()
    for window, sinks in ((20, 8), (20, 33), (145, 0), (3, 0), (3, 1)):
        c.upload()
        c.sink(window, sinks)
        ok()
        c.reference(window, sinks)
        c.check_attention(f"{window} {sinks}")
    c.close()


def test_no_request_and_no_lse():
    c = Case(512, 16, 1, [33], [100], seed=2).build()
    c.sink(40, 6)
    want = c.out.clone()
    c.out.fill_(float("nan"))
    c.sink(40, 6, lse=False)
    ok()
    assert torch.equal(want, c.out)
    c.close()


# a captured call with a window and sinks: its grid holds any spread of as many tokens
@pytest.mark.parametrize("hq,hkv,ps,shapes", [
    (16, 1, 16, [([40, 40], [160, 160]), ([40, 40], [256, 64])]),
    (16, 1, 16, [([9, 70], [80, 80]), ([70, 9], [144, 16])]),
    (4, 1, 8, [([40, 40], [80, 80]), ([1, 79], [8, 152])]),
])
def test_captured_sinks_follow_the_plan(hq, hkv, ps, shapes):
    replayed_weights(512, hq, hkv, ps, shapes, 90, 5)
