"""Refusals of pg_plan_paged_shared that need no GPU: every one comes before any CUDA call."""
import numpy as np
import pytest

from paged_sliding_window_qkv_gb300 import pg


def args(**kw):
    # two groups: requests 0 and 1 share two pages, request 2 shares nothing
    a = dict(num_req=3, qo_indptr=[0, 1, 2, 3], kv_page_indptr=[0, 3, 6, 7],
             page_ids=[4, 5, 6, 4, 5, 7, 8], last_page_len=[3, 16, 1], start_pos=[34, 47, 0],
             num_groups=2, group_indptr=[0, 2, 3], prefix_len=[32, 0], num_qo_heads=16,
             num_kv_heads=1, head_dim=512, page_size=16)
    a.update(kw)
    return a


CASES = {
    "no groups": (dict(num_groups=0), "PG_ERR_ARG"),
    "negative groups": (dict(num_groups=-1), "PG_ERR_ARG"),
    "null indptr": (dict(group_indptr=None), "PG_ERR_ARG"),
    "null prefix": (dict(prefix_len=None), "PG_ERR_ARG"),
    "indptr starts late": (dict(group_indptr=[1, 2, 3]), "PG_ERR_ARG"),
    "indptr ends early": (dict(group_indptr=[0, 1, 2]), "PG_ERR_ARG"),
    "an empty group": (dict(num_groups=3, group_indptr=[0, 2, 2, 3], prefix_len=[32, 0, 0]), "PG_ERR_ARG"),
    "indptr runs past": (dict(num_groups=3, group_indptr=[0, 4, 2, 3], prefix_len=[32, 0, 0]), "PG_ERR_ARG"),
    "negative prefix": (dict(prefix_len=[-16, 0]), "PG_ERR_ARG"),
    "half a page": (dict(prefix_len=[24, 0]), "PG_ERR_COVERAGE"),
    "past the first new token": (dict(prefix_len=[48, 0]), "PG_ERR_COVERAGE"),
    "a prefix past int32": (dict(prefix_len=[2 ** 40, 0]), "PG_ERR_COVERAGE"),
    "other pages": (dict(page_ids=[4, 5, 6, 4, 9, 7, 8]), "PG_ERR_COVERAGE"),
    "odd pages": (dict(page_size=12, last_page_len=[11, 24 - 12, 1], start_pos=[34, 35, 0],
                       prefix_len=[24, 0]), "PG_ERR_PLAN_MISMATCH"),
    "pages of four": (dict(num_req=1, qo_indptr=[0, 1], kv_page_indptr=[0, 2], page_ids=[0, 1],
                           last_page_len=[1], start_pos=[4], num_groups=1, group_indptr=[0, 1],
                           prefix_len=[4], page_size=4), "PG_ERR_PLAN_MISMATCH"),
    "head_dim": (dict(head_dim=128), "PG_ERR_PLAN_MISMATCH"),
    "a group of heads of three": (dict(num_qo_heads=3), "PG_ERR_PLAN_MISMATCH"),
    "a group of heads of 32": (dict(num_qo_heads=32), "PG_ERR_PLAN_MISMATCH"),
    "zero kv heads first": (dict(num_kv_heads=0, num_groups=-1), "PG_ERR_ZERO_KV_HEADS"),
    "the plain plan's checks": (dict(last_page_len=[17, 16, 1]), "PG_ERR_LAST_PAGE_LEN"),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_refused(name):
    change, want = CASES[name]
    rc, plan = pg.pg_plan_paged_shared(None, stream=0, **args(**change))
    assert rc == getattr(pg, want), (name, pg.pg_status_string(rc))
    assert plan is None


def test_null_plan_pointer_and_sizes():
    assert pg._plan_shared(None, 0, None, None, None, None, None, 0, None, None, 16, 1, 512, 16, None) == pg.PG_ERR_ARG
    for f in (pg.pg_shared_workspace_bytes, pg.pg_shared_q8_workspace_bytes, pg.pg_q8_workspace_bytes):
        assert f(None) == 0


def test_form_hook_refuses_other_numbers():
    for form in (-1, 3):
        assert pg.pg_test_shared_form(form) == pg.PG_ERR_ARG
    assert pg.pg_test_shared_form(0) == pg.PG_OK


def test_null_plan_calls():
    z = pg.pg_q8_pool_t()
    p = pg.pg_pool_t()
    assert pg.pg_attn_paged_shared(None, p, 0, None, None, None, 1.0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_attn_paged_shared_q8(None, z, 0, None, None, None, 1.0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_attn_paged_q8(None, z, 0, None, None, None, -1, 0, 1.0, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_kv_dequantize(None, z, p, 0, 1, stream=0) == pg.PG_ERR_ARG
    assert pg.pg_prep_paged_q8(None, z, 0, None, 0, None, 0, None, 0, None, None, 1e-6, None, None, 1, None,
                               stream=0) == pg.PG_ERR_ARG
