"""Page accounting of evicted requests (include/pg_kv.h), on CPU: the global family's pages after
an eviction, the segment plan inputs, and the refusals; and the refusals of the bounded-cache
entries that need no plan."""
import numpy as np
import pytest

from paged_sliding_window_qkv_gb300 import pg

L, G = pg.PG_KV_LOCAL, pg.PG_KV_GLOBAL


def server(ps=16, pages=64, ring=False):
    if ring:
        rc, s = pg.pg_kv_server_create_ring(pages, pages, ps, 100, 32, 1 << 20)
    else:
        rc, s = pg.pg_kv_server_create(pages, pages, ps, 1023, 0, 1 << 20)
    assert rc == pg.PG_KV_OK
    return s


def step(s, rid, n):
    assert pg.pg_kv_admit_step(s, rid, n) == pg.PG_KV_OK
    assert pg.pg_kv_commit_step(s, rid) == pg.PG_KV_OK


@pytest.mark.parametrize("ring", [False, True])
@pytest.mark.parametrize("ps", [1, 5, 16])
def test_random_steps_and_evictions_keep_the_account(ps, ring):
    rng = np.random.Generator(np.random.PCG64(ps))
    s = server(ps, pages=400, ring=ring)
    ids = [pg.pg_kv_request_open(s)[1] for _ in range(4)]
    front, gone = dict.fromkeys(ids, 0), dict.fromkeys(ids, 0)
    for _ in range(300):
        rid = ids[rng.integers(4)]
        held = front[rid] - gone[rid]
        if rng.random() < 0.4 and held > 0:
            keep = int(rng.integers(0, held + 1))
            assert pg.pg_kv_request_evict(s, rid, keep) == pg.PG_KV_OK
            gone[rid] += held - keep
        elif front[rid] < 250:
            n = int(rng.integers(1, 9))
            rc = pg.pg_kv_admit_step(s, rid, n)
            if rc == pg.PG_KV_ERR_NO_PAGES:
                continue
            assert rc == pg.PG_KV_OK
            rc, ptr, pages, last, first, start = pg.pg_kv_batch_segment_inputs(s, [rid], [n])
            assert rc == pg.PG_KV_OK
            now = front[rid] + n - gone[rid]          # keys held after the step
            assert first[0] == gone[rid] and start[0] == front[rid]
            assert ptr.tolist() == [0, -(-now // ps)] and len(pages) == ptr[1]
            assert (ptr[1] - 1) * ps + last[0] == now
            rc = pg.pg_kv_batch_plan_inputs(s, G, [rid], [n])[0]
            assert rc == (pg.PG_KV_ERR_EVICTED if gone[rid] else pg.PG_KV_OK)
            assert pg.pg_kv_batch_plan_inputs(s, L, [rid], [n])[0] == pg.PG_KV_OK
            if rng.random() < 0.3:
                assert pg.pg_kv_abort_step(s, rid) == pg.PG_KV_OK
            else:
                assert pg.pg_kv_commit_step(s, rid) == pg.PG_KV_OK
                front[rid] += n
        every = []
        for x in ids:
            pages = pg.pg_kv_request_pages(s, x, G)[1]
            assert len(pages) == -(-(front[x] - gone[x]) // ps)
            assert pg.pg_kv_request_info(s, x)[1] == front[x]
            every += pages.tolist()
        assert len(set(every)) == len(every)
        assert pg.pg_kv_free_pages(s, G)[1] == 400 - len(every)
    for x in ids:
        assert pg.pg_kv_request_close(s, x) == pg.PG_KV_OK
    assert pg.pg_kv_free_pages(s, G)[1] == 400 and pg.pg_kv_free_pages(s, L)[1] == 400
    pg.pg_kv_server_destroy(s)


def test_evict_refusals_change_nothing():
    s = server()
    rid = pg.pg_kv_request_open(s)[1]
    step(s, rid, 40)
    before = (pg.pg_kv_request_info(s, rid), pg.pg_kv_request_pages(s, rid, G)[1].tolist())
    assert pg.pg_kv_request_evict(s, rid, 41) == pg.PG_KV_ERR_ARG
    assert pg.pg_kv_request_evict(s, rid, -1) == pg.PG_KV_ERR_ARG
    assert pg.pg_kv_request_evict(s, rid + 9, 3) == pg.PG_KV_ERR_FOREIGN
    assert pg.pg_kv_request_evict(None, rid, 3) == pg.PG_KV_ERR_ARG
    assert pg.pg_kv_admit_step(s, rid, 1) == pg.PG_KV_OK
    assert pg.pg_kv_request_evict(s, rid, 3) == pg.PG_KV_ERR_PENDING
    assert pg.pg_kv_abort_step(s, rid) == pg.PG_KV_OK
    assert before == (pg.pg_kv_request_info(s, rid), pg.pg_kv_request_pages(s, rid, G)[1].tolist())
    assert pg.pg_kv_batch_segment_inputs(s, [rid], [1])[0] == pg.PG_KV_ERR_PENDING
    assert pg.pg_kv_batch_segment_inputs(s, [rid + 9], [1])[0] == pg.PG_KV_ERR_FOREIGN
    assert pg.pg_kv_batch_segment_inputs(s, [], [])[0] == pg.PG_KV_OK
    assert pg.pg_kv_request_evict(s, rid, 40) == pg.PG_KV_OK      # keeps all
    assert before == (pg.pg_kv_request_info(s, rid), pg.pg_kv_request_pages(s, rid, G)[1].tolist())
    assert pg.pg_kv_request_evict(s, rid, 0) == pg.PG_KV_OK       # keeps none
    assert len(pg.pg_kv_request_pages(s, rid, G)[1]) == 0
    step(s, rid, 1)
    assert len(pg.pg_kv_request_pages(s, rid, G)[1]) == 1
    pg.pg_kv_server_destroy(s)


@pytest.mark.parametrize("ps", [1, 4, 16])
@pytest.mark.parametrize("sinks", [0, 3, 20])
def test_trim_keeps_what_a_later_query_sees(ps, sinks):
    rng = np.random.Generator(np.random.PCG64(ps + sinks))
    window, total = 30, 400
    rc, s = pg.pg_kv_server_create(total, total, ps, window, 0, 1 << 20)
    assert rc == pg.PG_KV_OK
    ids = [pg.pg_kv_request_open(s)[1] for _ in range(2)]
    front = dict.fromkeys(ids, 0)
    for _ in range(60):
        rid = ids[rng.integers(2)]
        n = int(rng.integers(1, 6))
        assert pg.pg_kv_admit_step(s, rid, n) == pg.PG_KV_OK
        rc, ptr, pages, last, start = pg.pg_kv_batch_plan_inputs(s, L, [rid], [n])
        assert rc == pg.PG_KV_OK and (pages >= 0).all()
        held = pg.pg_kv_request_pages(s, rid, L)[1]
        assert len(held) == len(pages) == -(-(front[rid] + n) // ps)
        lo = front[rid] - window  # the step's first query's window
        for k, (h, p) in enumerate(zip(held, pages)):
            need = (k + 1) * ps > lo or k * ps < sinks
            assert (h >= 0 or not need) and p == (h if h >= 0 else held[-1])
        assert pg.pg_kv_request_trim(s, rid, sinks)[0] == pg.PG_KV_ERR_PENDING
        assert pg.pg_kv_commit_step(s, rid) == pg.PG_KV_OK
        front[rid] += n
        before = pg.pg_kv_free_pages(s, L)[1]
        rc, freed = pg.pg_kv_request_trim(s, rid, sinks)
        assert rc == pg.PG_KV_OK and pg.pg_kv_free_pages(s, L)[1] == before + freed
        assert pg.pg_kv_request_trim(s, rid, sinks) == (pg.PG_KV_OK, 0)
        assert (pg.pg_kv_request_pages(s, rid, L)[1] >= 0).sum() <= -(-sinks // ps) + -(-(window + 5) // ps) + 1
        assert (pg.pg_kv_request_pages(s, rid, G)[1] >= 0).all()
    mine = [p for x in ids for p in pg.pg_kv_request_pages(s, x, L)[1] if p >= 0]
    assert len(set(mine)) == len(mine) == total - pg.pg_kv_free_pages(s, L)[1]
    for x in ids:
        assert pg.pg_kv_request_close(s, x) == pg.PG_KV_OK
    assert pg.pg_kv_free_pages(s, L)[1] == total
    assert pg.pg_kv_request_trim(s, ids[0], sinks)[0] == pg.PG_KV_ERR_FOREIGN
    pg.pg_kv_server_destroy(s)
    s = server(ring=True)
    rid = pg.pg_kv_request_open(s)[1]
    assert pg.pg_kv_request_trim(s, rid, 0)[0] == pg.PG_KV_ERR_WINDOW
    assert pg.pg_kv_request_trim(s, rid, -1)[0] == pg.PG_KV_ERR_ARG
    pg.pg_kv_server_destroy(s)


def test_a_null_plan_is_refused():
    pool, stats = pg.pg_pool_t(), pg.pg_kv_stats_t()
    before = pg.pg_launch_count()
    assert pg.pg_attn_paged_sink(None, pool, 0, 0, 0, 0, 1, 1, 1.0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_attn_paged_mass(None, pool, 0, 0, 0, 0, stats, 1, 1, 1.0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_kv_evict_select(None, stats, 0, 1, 4, 0, 0, 0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_kv_evict_select(None, stats, 0, 1, 4, 2, 3, 0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_kv_evict_apply(None, pool, stats, 0, 1, 4, 0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_mass_workspace_bytes(None) == 0
    assert pg.pg_launch_count() == before
