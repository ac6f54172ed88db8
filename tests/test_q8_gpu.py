"""8-bit caches on the GPU: prep that quantises as it writes, the read-back, and attention, against
plain 64-bit references (tolerances derived in q8_ref.py and bounded_ref.py)."""
import numpy as np
import pytest
import torch

from paged_sliding_window_qkv_gb300 import pg
from q8_ref import LEAST, MOST, Q8Case, exponents, quantise, values

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_OK


# ------------------------------------------------------------------ prep
class Prep:
    """One prep call into a sentinel-filled 8-bit pool."""

    def __init__(self, D, hq, hkv, qo, start, ps=16, seed=0, layers=1, layer=0, evicted=0, edit=None):
        g = np.random.Generator(np.random.PCG64(seed))
        self.c = Q8Case(D, hq, hkv, qo, start, ps=ps, evicted=evicted, layers=layers, layer=layer, seed=seed)
        c = self.c
        c.codes_cpu.fill_(0x7F)
        c.scales_cpu.fill_(0xFF)
        c.build()
        T = int(c.qo_indptr[-1])
        nv = 2 if D == 256 else 1
        cols = (hq + nv * hkv) * D + 8  # (a stride of its own)
        raw = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).to(torch.bfloat16)
        if edit is not None:
            edit(raw)
        self.raw = raw.cuda()
        self.w = torch.from_numpy((1 + 0.1 * g.standard_normal((2, D))).astype(np.float32)).to(torch.bfloat16).cuda()
        rows = int((c.start + c.qo).max())
        f = (1e4 if D == 256 else 1e6) ** (-2.0 * np.arange(D // 2) / D)
        a = np.arange(rows)[:, None] * f
        self.cos = torch.from_numpy(np.cos(a).astype(np.float32)).cuda()
        self.sin = torch.from_numpy(np.sin(a).astype(np.float32)).cuda()
        self.q = torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.D, self.hq, self.hkv, self.cols, self.T = D, hq, hkv, cols, T

    def parts(self):
        D, hq, hkv = self.D, self.hq, self.hkv
        cut = lambda x, n: x[:, :n * D].reshape(-1, n, D)  # noqa: E731
        q, k = cut(self.raw, hq), cut(self.raw[:, hq * D:], hkv)
        return q, k, cut(self.raw[:, (hq + hkv) * D:], hkv) if D == 256 else None

    def run(self, plan=None, stream=None):
        D, hq, hkv = self.D, self.hq, self.hkv
        at = lambda n: self.raw[:, n * D:]  # noqa: E731
        pg.check(pg.pg_prep_paged_q8(
            plan or self.c.plan, self.c.q8, self.c.layer, self.raw, self.cols, at(hq), self.cols,
            at(hq + hkv) if D == 256 else None, self.cols, self.w[0], self.w[1], 1e-6, self.cos, self.sin,
            self.cos.shape[0], self.q, stream), "prep q8")

    def reference(self):
        """q, K, V in 64 bits [T, heads, D] and the magnitudes their sums add."""
        c = self.c
        pos = np.concatenate([s + np.arange(t) for s, t in zip(c.start, c.qo)])
        cs, sn = (x.double().cpu().numpy()[pos][:, None] for x in (self.cos, self.sin))
        norm = lambda x: x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(1e-6)))  # noqa: E731

        def rope(x, w):
            a, b = np.split(x * w, 2, -1)
            y = np.concatenate([a * cs - b * sn, b * cs + a * sn], -1)
            m = np.abs(a) + np.abs(b)
            return y, np.concatenate([m, m], -1)

        q, k, v = (None if x is None else x.double().cpu().numpy() for x in self.parts())
        w = self.w.double().cpu().numpy()
        v = norm(k if v is None else v)
        return rope(norm(q), w[0]), rope(norm(k), w[1]), (v, np.abs(v))

    def check(self):
        c = self.c
        (q, qm), k, v = self.reference()
        got = self.q.double().cpu().numpy()
        assert (np.abs(got - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -19 * qm).all()
        codes, scales = c.codes.cpu(), c.scales.cpu()
        val = values(codes[c.layer], scales[c.layer]).numpy()
        written = np.zeros(scales.shape, bool)
        for r in range(len(c.qo)):
            page, off = c.rows_of(r)
            s = slice(int(c.n[r] - c.qo[r]), int(c.n[r]))
            page, off = page[s], off[s]
            t = slice(int(c.qo_indptr[r]), int(c.qo_indptr[r + 1]))
            for i, (y, m) in enumerate((k, v)):
                y, m = y[t], m[t]
                e = scales[c.layer][page, i, :, off].numpy().astype(np.int64) - 127
                ref, top = exponents(y), np.abs(y).max(-1)
                # the exponent is the reference's unless the largest element stands at its border
                slop = 2.0 ** -18 * m.max(-1)
                near = (exponents((top + slop)[..., None]) == e) | (exponents((np.maximum(top - slop, 0))[..., None]) == e)
                assert ((e == ref) | near).all()
                x = val[page, i, :, off]
                lim = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * np.exp2(e)[..., None]) + 2.0 ** -18 * m
                assert (np.abs(x - y) <= lim).all(), (r, i, float((np.abs(x - y) - lim).max()))
                # the largest element stands in the codes' top octave
                assert (np.abs(x).max(-1) > 223 * np.exp2(e))[e > LEAST].all()
                written[c.layer, page, i, :, off] = True
        assert (codes.numpy()[~written] == 0x7F).all() and (scales.numpy()[~written] == 0xFF).all()


HEADS = {256: [(16, 8), (8, 8), (16, 1), (4, 2)], 512: [(16, 1), (8, 1), (4, 2)]}


@pytest.mark.parametrize("D,hq,hkv", [(d, *h) for d in (256, 512) for h in HEADS[d]])
@pytest.mark.parametrize("ps", [1, 5, 16, 64])
def test_prep_writes_rounded_rows_and_nothing_else(D, hq, hkv, ps):
    p = Prep(D, hq, hkv, [1, 37, 2, 160], [0, 5, 300, 63], ps=ps, seed=ps + hq, layers=2, layer=1)
    p.run()
    ok()
    p.check()
    p.c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_prep_single_tokens_and_evicted_requests(D):
    hq, hkv = HEADS[D][0]
    p = Prep(D, hq, hkv, [1] * 5, [0, 15, 16, 700, 1300], evicted=[0, 3, 16, 650, 1], seed=7)
    p.run()
    ok()
    p.check()
    p.c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_prep_zero_tiny_and_spiky_rows(D):
    hq, hkv = HEADS[D][0]

    def edit(raw):
        raw[0] = 0                                   # a row of zeros: eps keeps it zero
        raw[1] = raw[1] * 2.0 ** -60                 # far below eps
        raw[2] = 0
        raw[2, ::D] = 30.0                           # one element a row
        raw[3] = torch.sign(raw[3])                  # all of one size
        raw[4] = raw[4] * 2.0 ** 40

    p = Prep(D, hq, hkv, [6], [9], seed=3, edit=edit)
    p.run()
    ok()
    p.check()
    zero = p.c.scales.cpu()[0, p.c.ids[0], :, :, 9]
    assert (zero == LEAST + 127).all()
    p.c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_prep_non_finite_elements(D):
    """A NaN makes its own row NaN (its norm is), and no other row or head."""
    hq, hkv = HEADS[D][0]
    hkv = 2
    at = (hq + 1) * D + 5

    def edit(raw):
        raw[2, at] = float("nan")

    p = Prep(D, hq, hkv, [4], [0], seed=5, edit=edit)
    p.run()
    ok()
    v = values(p.c.codes.cpu()[0], p.c.scales.cpu()[0])[p.c.ids[0].astype(int)]  # [kv, head, slot, D]
    bad = torch.isnan(v[:, :, :4]).any(-1)
    want = torch.zeros_like(bad)
    want[0, 1, 2] = True
    if D == 512:
        want[1, 1, 2] = True
    assert torch.equal(bad, want)
    p.c.close()


# ------------------------------------------------------------------ read-back
@pytest.mark.parametrize("D,hkv", [(256, 8), (256, 1), (512, 1), (512, 2)])
@pytest.mark.parametrize("ps", [1, 3, 16, 64])
def test_dequantize_is_exact_and_touches_held_slots_alone(D, hkv, ps):
    c = Q8Case(D, hkv * 2, hkv, [1, 1, 1, 1, 5], [0, 15, 16, 200, 95], evicted=[0, 2, 0, 77, 0], ps=ps,
               layers=3, seed=ps).build()
    dst = torch.full((4, c.P + 2, 2, hkv, ps, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pg.check(pg.pg_kv_dequantize(c.plan, c.q8, pg.pool_descriptor(dst), 1, 2))
    ok()
    want = torch.full(dst.shape, 7.0, dtype=torch.bfloat16)
    for r in range(5):
        page, off = (torch.from_numpy(x) for x in c.rows_of(r))
        want[1:3, page, :, :, off] = c.pool_cpu[1:3, page, :, :, off]
    assert torch.equal(dst.cpu(), want)
    c.close()


def test_dequantize_every_code_and_scale():
    """All 256 codes under the least, the largest and some scales between."""
    c = Q8Case(256, 2, 1, [1], [63], ps=16, seed=1)
    c.codes_cpu[:] = torch.arange(256, dtype=torch.uint8)
    s = torch.tensor([LEAST, -100, -20, -8, -1, 0, 1, 9, 100, MOST], dtype=torch.int32)
    c.scales_cpu[:] = (s[torch.arange(c.scales_cpu.numel()) % len(s)] + 127).to(torch.uint8).reshape(c.scales_cpu.shape)
    c.build()
    dst = torch.zeros(c.pool.shape, dtype=torch.bfloat16, device="cuda")
    pg.check(pg.pg_kv_dequantize(c.plan, c.q8, pg.pool_descriptor(dst), 0, 1))
    ok()
    page, off = (torch.from_numpy(x) for x in c.rows_of(0))
    want = values(c.codes_cpu[0], c.scales_cpu[0])[page, :, :, off]
    got = dst[0].cpu()[page, :, :, off].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    big = want.abs() >= 2.0 ** 128  # (past bf16: no row that prep writes holds such an element)
    assert torch.equal(torch.nan_to_num(got)[~big], torch.nan_to_num(want)[~big])
    c.close()


def test_dequantize_shared_pages():
    c = Q8Case(512, 16, 1, [1, 1], [40, 70], seed=2)
    c.ids[c.pg_indptr[1]:c.pg_indptr[1] + 2] = c.ids[:2]  # both requests list the same first pages
    c.build()
    dst = torch.zeros(c.pool.shape, dtype=torch.bfloat16, device="cuda")
    pg.check(pg.pg_kv_dequantize(c.plan, c.q8, pg.pool_descriptor(dst), 0, 1))
    ok()
    for r in (0, 1):
        page, off = (torch.from_numpy(x) for x in c.rows_of(r))
        assert torch.equal(dst[0].cpu()[page, :, :, off], c.pool_cpu[0][page, :, :, off])
    c.close()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (0, 0), (0, 1), (63, 64), (100, 3), (2000, 4)])
def test_prefill(D, window, sinks):
    hq, hkv = HEADS[D][0]
    c = Q8Case(D, hq, hkv, [1, 2, 333, 64, 130], [0, 700, 0, 511, 90], seed=window + sinks + 1).build()
    c.attend(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("ps", [1, 3, 8, 32, 128])
@pytest.mark.parametrize("qo,start", [([77, 200], [300, 0]), ([1] * 4, [0, 40, 333, 700])])
def test_page_sizes(D, ps, qo, start):
    hq, hkv = HEADS[D][0]
    c = Q8Case(D, hq, hkv, qo, start, ps=ps, seed=ps).build()
    c.attend(50, 20)
    ok()
    c.reference(50, 20)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D,hq,hkv", [(256, 16, 8), (256, 8, 8), (256, 16, 4), (256, 16, 1), (256, 8, 2),
                                      (512, 16, 1), (512, 8, 1), (512, 4, 2), (512, 16, 2), (512, 2, 2)])
def test_decode_head_groups(D, hq, hkv):
    c = Q8Case(D, hq, hkv, [1] * 4, [210, 0, 33, 1000], seed=hq + hkv, layers=2, layer=1).build()
    for window, sinks in ((-1, 0), (60, 5)):
        c.upload()
        c.attend(window, sinks)
        ok()
        c.reference(window, sinks)
        c.check_attention(f"{D} {hq}/{hkv} {window}")
    c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 2), (15, 16), (100, 5), (1023, 4), (-1, 0), (300, 5000)])
def test_decode(D, window, sinks):
    hq, hkv = HEADS[D][0]
    start = [0, 1, 15, 16, 31, 32, 100, 127, 128, 511, 1500, 2222]
    c = Q8Case(D, hq, hkv, [1] * len(start), start, seed=window + 2 * sinks + 1).build()
    c.attend(window, sinks)
    ok()
    c.reference(window, sinks)
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_segments_and_empty_rows(D):
    """Positions are absolute, slots count from kv_start; rows may see nothing."""
    hq, hkv = HEADS[D][0]
    for qo, start in (([40, 3], [200, 90]), ([1, 1], [200, 90])):
        c = Q8Case(D, hq, hkv, qo, start, evicted=[0, 30], held=[60, 50], seed=4).build()
        for window, sinks in ((20, 8), (20, 33), (145, 0), (3, 0), (-1, 0)):
            c.upload()
            c.attend(window, sinks)
            ok()
            c.reference(window, sinks)
            c.check_attention(f"{qo} {window} {sinks}")
        c.close()


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("scale", [0.0, -1.0, 0.25])
def test_scales_of_scores(D, scale):
    hq, hkv = HEADS[D][0]
    for qo, start in (([90], [100]), ([1, 1], [100, 44])):
        c = Q8Case(D, hq, hkv, qo, start, seed=3).build()
        c.attend(-1, 0, scale)
        ok()
        c.reference(-1, 0, scale)
        c.check_attention()
        c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_hidden_codes_may_be_anything(D):
    """NaN codes and scales in slots that no row sees and behind the last key change nothing."""
    hq, hkv = HEADS[D][0]
    for ps in (16, 64):
        c = Q8Case(D, hq, hkv, [1, 1, 1], [500, 77, 3], ps=ps, seed=8)
        live = np.zeros((c.P, ps), bool)
        for r in range(3):
            page, off = c.rows_of(r)
            j = np.arange(c.n[r])
            see = (c.start[r] - j <= 60) | (j < 4)
            live[page[see], off[see]] = True
        dead = torch.from_numpy(~live)
        c.codes_cpu[0].permute(0, 3, 1, 2, 4)[dead] = 0x7F
        c.scales_cpu[0].permute(0, 3, 1, 2)[dead] = 0xFF
        c.build()
        c.attend(60, 4)
        ok()
        c.reference(60, 4)
        c.check_attention()
        c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_a_visible_nan_reaches_its_rows_alone(D):
    hq, hkv = (4, 2)
    for kv in (0, 1):
        c = Q8Case(D, hq, hkv, [1, 1], [300, 100], seed=11)
        page, off = c.rows_of(0)
        c.codes_cpu[0, page[200], kv, 1, off[200], 9] = 0x7F
        c.build()
        c.attend()
        ok()
        c.reference()
        got = torch.isnan(c.out.cpu())
        want = torch.zeros_like(got)
        if kv == 0:
            want[0, 2:] = True
            assert torch.isnan(c.lse[0, 2:]).all()
        else:
            want[0, 2:, 9] = True
        assert torch.equal(got, want)
        c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_rows_of_very_different_sizes(D):
    """V rows whose scales lie 2^60 apart, K rows of zeros, queries with one large element."""
    hq, hkv = HEADS[D][0]

    def gain(y):
        g = torch.ones(y.shape[:-1])
        n = torch.arange(g[:, :, 1].numel()).reshape(g[:, :, 1].shape)
        g[:, :, 1] = torch.where(n % 7 == 0, 2.0 ** 30, torch.where(n % 7 == 1, 2.0 ** -30, 1.0))
        g[:, :, 0] = torch.where(n % 11 == 0, 0.0, 1.0)
        return g[..., None]

    c = Q8Case(D, hq, hkv, [1, 1, 1], [300, 17, 1000], seed=12, row_gain=gain)
    c.q_cpu[:, :, 3] *= 2.0 ** 6
    c.build()
    c.attend()
    ok()
    c.reference()
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_scores_that_grow_along_the_keys(D):
    """Every tile outgrows the last one's largest score: the running reference moves each time."""
    hq, hkv = HEADS[D][0]

    def gain(y):
        return torch.ones(y.shape[:-1] + (1,))

    c = Q8Case(D, hq, hkv, [1, 1], [1500, 900], seed=13, row_gain=gain)
    y = c.pool_cpu.float()
    q = c.q_cpu.float()
    for r in range(2):
        page, off = c.rows_of(r)
        for g in range(hkv):
            d = q[r, g * (hq // hkv)]
            step = torch.linspace(0, 60, len(page))[:, None] * d / (d * d).sum()
            y[0, page, 0, g, off] = step + 0.01 * y[0, page, 0, g, off]
    c.set_rows(y)
    c.build()
    c.attend()
    ok()
    c.reference()
    c.check_attention()
    c.close()


@pytest.mark.parametrize("D,hq,hkv,n,keys", [(256, 16, 8, 38, 385), (256, 16, 8, 60, 401), (256, 16, 8, 20, 485),
                                             (256, 16, 4, 40, 385), (256, 16, 1, 76, 385), (512, 16, 1, 152, 385),
                                             (512, 16, 1, 76, 300), (512, 8, 1, 152, 900), (256, 16, 8, 76, 130)])
def test_segments_that_end_with_their_ctas(D, hq, hkv, n, keys):
    """Many equal requests, whose tiles fall to the SMs in whole segments (on 152 of them): a last tile of
    few keys ends a CTA's work. Repeated, for what depends on timing."""
    c = Q8Case(D, hq, hkv, [1] * n, [keys - 1] * n, seed=n).build()
    c.attend()
    ok()
    first = c.out.clone()
    c.reference()
    c.check_attention()
    for _ in range(20):
        c.out.fill_(float("nan"))
        c.attend()
        ok()
        assert torch.equal(c.out, first)
    c.close()


def test_long_cache():
    """Element offsets past 2^31: a pool of 2.4e9 codes, the request's pages at its end."""
    D, hq, hkv, ps = 512, 16, 1, 16
    P = 150_000
    c = Q8Case(D, hq, hkv, [1], [1200], ps=ps, seed=14).build()
    codes = torch.zeros((1, P, 2, hkv, ps, D), dtype=torch.uint8, device="cuda")
    scales = torch.full((1, P, 2, hkv, ps), 127, dtype=torch.uint8, device="cuda")
    codes[0, P - c.P:] = c.codes[0]
    scales[0, P - c.P:] = c.scales[0]
    ids = (c.ids + (P - c.P)).astype(np.int32)
    rc, plan = pg.pg_plan_paged_segment(None, 1, c.qo_indptr, c.pg_indptr, ids, c.last, c.ks, c.start, hq, hkv, D, ps)
    pg.check(rc)
    pg.check(pg.pg_attn_paged_q8(plan, pg.q8_descriptor(codes, scales), 0, c.q, c.out, c.lse, -1, 0, 1.0, c.ws,
                                 c.ws_bytes))
    ok()
    c.reference()
    c.check_attention()
    plan.close()
    c.close()


# ------------------------------------------------------------------ streams, graphs, runs together
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("decode", [True, False])
def test_captured_step_follows_its_plan(D, decode):
    """Prep, attention and read-back captured once, replayed after the plan moved on."""
    hq, hkv = HEADS[D][0]
    stream = torch.cuda.Stream()
    qo = [1, 1, 1] if decode else [30, 2, 17]
    with torch.cuda.stream(stream):
        a = Q8Case(D, hq, hkv, qo, [200, 90, 31], seed=21, stream=stream).build()
        dst = torch.zeros(a.pool.shape, dtype=torch.bfloat16, device="cuda")
        d = pg.pool_descriptor(dst)

        def step():
            a.attend(150, 3)
            pg.check(pg.pg_kv_dequantize(a.plan, a.q8, d, 0, 1, stream))

        step()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
        # as many requests, tokens and pages, spread otherwise
        b = Q8Case(D, hq, hkv, qo[::-1], [31, 90, 200] if decode else [44, 90, 187], seed=22, stream=stream)
        assert len(b.ids) == len(a.ids) and b.P == a.P
        rc, _ = pg.pg_plan_paged_segment(a.plan, 3, b.qo_indptr, b.pg_indptr, b.ids, b.last, b.ks, b.start, hq, hkv, D,
                                         16, stream)
        pg.check(rc)
        a.codes.copy_(b.codes_cpu)
        a.scales.copy_(b.scales_cpu)
        a.q.copy_(b.q_cpu)
        dst.zero_()
        a.out.fill_(float("nan"))
        g.replay()
        stream.synchronize()
        assert pg.pg_device_status(stream) == pg.PG_OK
    b.out, b.lse = a.out, a.lse
    b.reference(150, 3)
    b.check_attention()
    for r in range(3):
        page, off = (torch.from_numpy(x) for x in b.rows_of(r))
        assert torch.equal(dst[0].cpu()[page, :, :, off], b.pool_cpu[0][page, :, :, off])
    a.close()


@pytest.mark.parametrize("D", [256, 512])
def test_prompt_then_tokens(D):
    """A request's life: its prompt written and attended, then single tokens, all on one cache, the
    last step's attention against a bf16 pool that was read back."""
    hq, hkv = HEADS[D][0]
    lens = [70, 1, 1, 1]
    total = sum(lens)
    last = None
    pool = None
    for i, n in enumerate(lens):
        start = sum(lens[:i])
        p = Prep(D, hq, hkv, [n], [start], seed=30 + i)
        if pool is not None:
            p.c.codes.copy_(pool[0])
            p.c.scales.copy_(pool[1])
        p.c.ids[:] = np.arange(len(p.c.ids))
        rc, _ = pg.pg_plan_paged_segment(p.c.plan, 1, p.c.qo_indptr, p.c.pg_indptr, p.c.ids, p.c.last, p.c.ks,
                                         p.c.start, hq, hkv, D, 16)
        pg.check(rc)
        p.run()
        p.c.q.copy_(p.q)
        p.c.attend(-1, 0, 0.05)
        ok()
        pages = -(-total // 16)
        codes = torch.zeros((1, pages + 3, 2, hkv, 16, D), dtype=torch.uint8, device="cuda")
        scales = torch.full((1, pages + 3, 2, hkv, 16), 127, dtype=torch.uint8, device="cuda")
        k = min(pages + 3, p.c.P)
        codes[:, :k], scales[:, :k] = p.c.codes[:, :k], p.c.scales[:, :k]
        if i + 1 < len(lens):
            nxt = Q8Case(D, hq, hkv, [lens[i + 1]], [start + n])
            pool = codes[:, :nxt.P].contiguous(), scales[:, :nxt.P].contiguous()
        last = p.c
        last.q_cpu = p.q.cpu()
        last.pool_cpu = torch.nan_to_num(values(p.c.codes.cpu(), p.c.scales.cpu())).to(torch.bfloat16)
        last.reference(-1, 0, 0.05)
        last.check_attention(f"step {i}")
    bf = torch.zeros(last.pool.shape, dtype=torch.bfloat16, device="cuda")
    d = pg.pool_descriptor(bf)
    pg.check(pg.pg_kv_dequantize(last.plan, last.q8, d, 0, 1))
    out = torch.empty_like(last.out)
    ws = torch.empty(max(16, pg.pg_sink_workspace_bytes(last.plan)), dtype=torch.uint8, device="cuda")
    pg.check(pg.pg_attn_paged_sink(last.plan, d, 0, last.q, out, None, -1, 0, 0.05, ws, ws.numel()))
    ok()
    last.out = out
    last.check_attention("bf16 over the read-back")
    last.close()


# ------------------------------------------------------------------ refusals
def test_refusals_launch_nothing_and_write_nothing():
    c = Q8Case(512, 16, 1, [1, 1], [100, 30], seed=40).build()
    torch.cuda.synchronize()
    before = pg.pg_launch_count()
    nan = float("nan")
    out0 = c.out.clone()

    def attn(want, plan=c.plan, pool=c.q8, layer=0, q=c.q, out=c.out, lse=c.lse, window=-1, sinks=0, scale=1.0,
             ws=c.ws, n=c.ws_bytes, stream=None):
        assert pg.pg_attn_paged_q8(plan, pool, layer, q, out, lse, window, sinks, scale, ws, n, stream) == want

    attn(pg.PG_ERR_ARG, plan=None)
    attn(pg.PG_ERR_ARG, pool=None)
    attn(pg.PG_ERR_ARG, q=None)
    attn(pg.PG_ERR_ARG, out=None)
    attn(pg.PG_ERR_LAYER, layer=1)
    attn(pg.PG_ERR_LAYER, layer=-1)
    attn(pg.PG_ERR_WINDOW, window=-2)
    attn(pg.PG_ERR_WINDOW, sinks=-1)
    attn(pg.PG_ERR_NONFINITE, scale=nan)
    attn(pg.PG_ERR_WORKSPACE, n=c.ws_bytes - 1)
    attn(pg.PG_ERR_WORKSPACE, ws=None)
    attn(pg.PG_ERR_ALIGN, ws=c.ws.data_ptr() + 4)
    attn(pg.PG_ERR_ALIGN, q=c.q.data_ptr() + 16)
    attn(pg.PG_ERR_ALIGN, lse=c.lse.data_ptr() + 2)
    attn(pg.PG_ERR_STREAM, stream=torch.cuda.Stream())
    d = lambda **kw: pg.q8_descriptor(c.codes, c.scales, **kw)  # noqa: E731
    attn(pg.PG_ERR_ARG, pool=d(codes=None))
    attn(pg.PG_ERR_ARG, pool=d(scales=None))
    attn(pg.PG_ERR_ALIGN, pool=d(codes=c.codes.data_ptr() + 8))
    attn(pg.PG_ERR_LAYOUT, pool=d(capacity=c.scales.numel() - 1))
    attn(pg.PG_ERR_LAYOUT, pool=d(head_dim=256))
    attn(pg.PG_ERR_LAYOUT, pool=d(num_layers=0))
    attn(pg.PG_ERR_PLAN_MISMATCH, pool=d(page_size=8, num_pages=2 * c.P))
    attn(pg.PG_ERR_PAGE_OOB, pool=d(num_pages=int(c.ids.max()), capacity=int(c.ids.max()) * 32))
    attn(pg.PG_ERR_I32_OVERFLOW, pool=d(num_layers=2 ** 31 - 1, num_pages=2 ** 31 - 1, num_kv_heads=2 ** 20))
    bf = torch.zeros(c.pool.shape, dtype=torch.bfloat16, device="cuda")
    desc = pg.pool_descriptor(bf)

    def read(want, plan=c.plan, src=c.q8, dst=desc, layer=0, layers=1, stream=None):
        assert pg.pg_kv_dequantize(plan, src, dst, layer, layers, stream) == want

    read(pg.PG_ERR_ARG, plan=None)
    read(pg.PG_ERR_ARG, src=None)
    read(pg.PG_ERR_ARG, dst=None)
    read(pg.PG_ERR_LAYER, layers=2)
    read(pg.PG_ERR_LAYER, layers=0)
    read(pg.PG_ERR_LAYOUT, dst=pg.pool_descriptor(bf, capacity=1))
    read(pg.PG_ERR_STREAM, stream=torch.cuda.Stream())
    rc, ring = pg.pg_plan_paged_prefill_ring(None, 1, [0, 1], [0, 4], [0, 1, 2, 3], [100], 16, 1, 512, 16, 40)
    pg.check(rc)
    attn(pg.PG_ERR_PLAN_MISMATCH, plan=ring)
    read(pg.PG_ERR_PLAN_MISMATCH, plan=ring)
    p = Prep(512, 16, 1, [2], [3], seed=1)
    prep = [p.c.plan, p.c.q8, 0, p.raw, p.cols, p.raw, p.cols, None, 0, p.w[0], p.w[1], 1e-6, p.cos, p.sin,
            p.cos.shape[0], p.q]

    def refuse(want, i, value):
        assert pg.pg_prep_paged_q8(*[value if k == i else x for k, x in enumerate(prep)]) == want

    torch.cuda.synchronize()
    launches = pg.pg_launch_count()
    refuse(pg.PG_ERR_ARG, 0, None)
    refuse(pg.PG_ERR_PLAN_MISMATCH, 0, ring)
    refuse(pg.PG_ERR_ARG, 1, None)
    refuse(pg.PG_ERR_LAYER, 2, 1)
    refuse(pg.PG_ERR_ARG, 3, None)
    refuse(pg.PG_ERR_ARG, 4, 16 * 512 - 8)
    refuse(pg.PG_ERR_ALIGN, 4, p.cols + 4)
    refuse(pg.PG_ERR_ARG, 7, p.raw)  # head_dim 512 takes no V
    refuse(pg.PG_ERR_NONFINITE, 11, 0.0)
    refuse(pg.PG_ERR_ROPE_RANGE, 14, 4)
    refuse(pg.PG_ERR_ARG, 15, None)
    assert pg.pg_launch_count() == launches == before
    assert torch.equal(torch.nan_to_num(c.out), torch.nan_to_num(out0)) and not bf.any()
    ok()
    ring.close()
    p.c.close()
    c.close()


@pytest.mark.parametrize("D,hq", [(256, 5), (512, 3), (512, 32)])
def test_head_groups_that_do_not_fill_a_tile_are_refused(D, hq):
    c = Q8Case(D, hq, 1, [1] * 4, [210, 0, 33, 1000], seed=hq + 1).build()
    before = pg.pg_launch_count()
    assert pg.pg_attn_paged_q8(c.plan, c.q8, 0, c.q, c.out, c.lse, -1, 0, 1.0, c.ws, c.ws_bytes) == \
        pg.PG_ERR_PLAN_MISMATCH
    assert pg.pg_launch_count() == before
    c.close()


def test_empty_batch():
    rc, plan = pg.pg_plan_paged_prefill(None, 0, [0], [0], [], [], [], 16, 1, 512, 16)
    pg.check(rc)
    c = Q8Case(512, 16, 1, [1], [3]).build()
    before = pg.pg_launch_count()
    assert pg.pg_q8_workspace_bytes(plan) == 0
    pg.check(pg.pg_attn_paged_q8(plan, c.q8, 0, None, None, None, -1, 0, 1.0))
    pg.check(pg.pg_kv_dequantize(plan, c.q8, c.desc, 0, 1))
    assert pg.pg_launch_count() == before
    plan.close()
    c.close()


@pytest.mark.parametrize("decode", [True, False])
def test_a_bad_device_page_is_reported_and_skipped(decode):
    """A page id out of range on the device: nothing is read there, the other requests are right."""
    import ctypes as C
    rt = None
    for name in ("libcudart.so.13", "libcudart.so"):
        try:
            rt = C.CDLL(name)
            break
        except OSError:
            continue
    if rt is None:
        pytest.skip("libcudart not loadable by name")
    qo, start = ([1] * 4, [100, 300, 40, 7]) if decode else ([30, 2, 60, 9], [100, 300, 40, 7])
    c = Q8Case(512, 16, 1, qo, start, seed=60).build()
    torch.cuda.synchronize()
    bad = np.array([c.P + 1000], np.int32)
    rt.cudaMemcpy.argtypes = [C.c_void_p, C.c_void_p, C.c_size_t, C.c_int]
    at = c.plan.info().d_page_ids + 4 * int(c.pg_indptr[1] + 2)
    assert rt.cudaMemcpy(at, bad.ctypes.data, 4, 1) == 0
    c.attend()
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_ERR_DEVICE_BOUNDS
    c.reference()
    rows = np.concatenate([np.arange(c.qo_indptr[r], c.qo_indptr[r + 1]) for r in (0, 2, 3)])
    c.check_attention(rows=rows)
    dst = torch.full(c.pool.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    pg.check(pg.pg_kv_dequantize(c.plan, c.q8, pg.pool_descriptor(dst), 0, 1))
    torch.cuda.synchronize()
    assert pg.pg_device_status() == pg.PG_ERR_DEVICE_BOUNDS
    want = torch.full(dst.shape, 3.0, dtype=torch.bfloat16)
    for r in range(4):
        page, off = (torch.from_numpy(x) for x in c.rows_of(r))
        keep = torch.ones(len(page), dtype=torch.bool)
        if r == 1:
            keep[32:48] = False
        want[0, page[keep], :, :, off[keep]] = c.pool_cpu[0, page[keep], :, :, off[keep]]
    assert torch.equal(dst.cpu(), want)
    c.close()


@pytest.mark.parametrize("D", [256, 512])
def test_query_rows_of_any_size(D):
    """Rows of zeros, of 2^-40 and of 2^20, one with an infinity, one with a NaN: the last two give NaN rows
    and no other."""
    hq, hkv = (4, 2)
    c = Q8Case(D, hq, hkv, [1, 1], [300, 40], seed=61)
    c.q_cpu[0, 0] = 0
    c.q_cpu[0, 1] *= 2.0 ** -40
    c.q_cpu[0, 2, :5] *= 2.0 ** 3
    c.q_cpu[1, 0, 7] = float("inf")
    c.q_cpu[1, 3, 9] = float("nan")
    c.build()
    c.attend()
    ok()
    bad = torch.zeros((2, hq), dtype=torch.bool)
    bad[1, 0] = bad[1, 3] = True
    assert torch.equal(torch.isnan(c.out.cpu()).all(-1), bad)
    assert torch.equal(torch.isnan(c.out.cpu()).any(-1), bad)
    assert torch.equal(torch.isnan(c.lse.cpu()), bad)
    c.q_cpu[bad] = 0
    keep = c.out, c.lse
    c.reference()
    c.out, c.lse = torch.where(bad[..., None].cuda(), 0, keep[0]), torch.where(bad.cuda(), 0, keep[1])
    out, lse, m, p, wabs = c.ref
    out[bad.numpy()] = 0
    lse[bad.numpy()] = 0
    c.check_attention()
    c.close()


def test_two_plans_on_two_streams():
    """Calls of two plans at once, each with its own workspace."""
    D, hq, hkv = 512, 16, 1
    cs = []
    for seed in (70, 71):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            cs.append(Q8Case(D, hq, hkv, [1] * 20, list(range(100, 2100, 100)), seed=seed, stream=s).build())
    torch.cuda.synchronize()
    for _ in range(10):
        for c in cs:
            with torch.cuda.stream(c.stream):
                c.attend()
    ok()
    for c in cs:
        c.reference()
        c.check_attention()
        c.close()


def rows_near_a_border(D, count):
    """Raw rows whose largest element is 14 * (1 + d) in 64 bits with |d| below 2^-24 (14 = 448 / 32): one
    element a, D - 1 others of two values. Closest first, both sides among them."""
    mant = 1 + np.arange(128) / 128.0  # bf16 numbers of one octave
    b1, b2 = mant[:, None], mant[None, :] / 2
    eps = np.float64(np.float32(1e-6))
    found = []
    for a in np.concatenate([mant * 16, mant * 32]):
        s = (a * a / 196 - eps) * D - a * a  # what the others' squares have to add up to
        n = np.clip(np.rint((s - (D - 1) * b2 ** 2) / (b1 ** 2 - b2 ** 2 + (b1 == b2))), 0, D - 1)
        d = a / np.sqrt((a * a + n * b1 ** 2 + (D - 1 - n) * b2 ** 2) / D + eps) / 14 - 1
        for x, y in zip(*np.nonzero((np.abs(d) < 2.0 ** -24) & (np.abs(d) > 1e-12))):
            found.append((abs(d[x, y]), d[x, y] > 0, a, mant[x], mant[y] / 2, int(n[x, y])))
    found.sort()
    rows = np.zeros((count, D))
    for r, (_, _, a, p, q, n) in enumerate(found[:count]):
        rows[r, 0], rows[r, 1:1 + n], rows[r, 1 + n:] = a, p, q
    assert len(found) >= count and {f[1] for f in found[:count]} == {True, False}
    return rows


@pytest.mark.parametrize("D", [256, 512])
def test_a_row_at_the_border_has_the_exponent_of_64_bits(D):
    hq, hkv, T = 2, 2, 48
    rows = rows_near_a_border(D, T * hkv)

    def edit(raw):
        for h in range(hkv):
            at = (hq + h) * D
            raw[:, at:at + D] = torch.from_numpy(rows[h::hkv]).to(raw.dtype)
            if D == 256:
                at = (hq + hkv + h) * D
                raw[:, at:at + D] = torch.from_numpy(rows[::-1][h::hkv].copy()).to(raw.dtype)

    p = Prep(D, hq, hkv, [T], [0], edit=edit)
    p.w[1] = 1
    p.cos.fill_(1.0)
    p.sin.fill_(0.0)
    p.run()
    ok()
    p.check()
    page, off = p.c.rows_of(0)
    _, (k, _), (v, _) = p.reference()
    for i, y in enumerate((k, v)):
        got = p.c.scales.cpu()[0][page, i, :, off].numpy().astype(np.int64) - 127
        assert (got == exponents(y)).all(), (i, int((got != exponents(y)).sum()))
    p.c.close()
