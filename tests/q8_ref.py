"""Plain 64-bit restatement of the 8-bit cache, and the set-up its tests share.

A quantised row stands for exact bf16 numbers, so attention over it is held to bounded_ref's
reference and tolerances on those numbers. Decode of 8-bit pages adds (derived before any run):
  a weight taken as three e4m3 terms is within 2^-12 of itself (twice the half step 2^-4 of three
  roundings, 2^-13, to be safe), which bounded_ref's 2^-8 * A for a bf16 weight already covers, or
  within 2^-21 of the row's largest weight * 2^(v exponent): `floor` below adds
  2^-21 * sum over the visible keys of the largest |v| of the row, times the largest weight (<= 1)
  a query element taken as two terms is within 2^-22 of the row's largest: `qslop` adds
  2 * 2^-22 * max|q| * max_j sum_d |k_jd| * |scale| to the weights' error, as scores do.
Prep: a result in fp32 is within 2^-19 of the sum of the magnitudes it adds (four products and sums,
the reciprocal square root and the rotary factors, each within 2^-22), and its code within half a
step of that: 2^-4 of the value, or 2^-10 * 2^e where codes are subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

from bounded_ref import Case
from paged_sliding_window_qkv_gb300 import pg

LEAST, MOST = -110, 120


def exponents(y):
    """The scale exponent of every row of y (float64, finite)."""
    m, x = np.frexp(np.abs(y).max(-1))
    return np.where(m > 0, np.clip(x - 9 + (m > 0.875), LEAST, MOST), LEAST)


def quantise(y):
    """(codes, scales) of float32 rows: the product with a power of two and torch's e4m3 rounding."""
    y = y.float()
    e = torch.from_numpy(exponents(torch.where(y.isfinite(), y, 0).double().numpy()))
    scaled = torch.ldexp(y.double(), -e[..., None]).float()
    code = torch.where(scaled.isfinite(), scaled, torch.nan).to(torch.float8_e4m3fn).view(torch.uint8)
    return code, (e + 127).to(torch.uint8)


def values(codes, scales):
    """float64 values of codes under scales."""
    return codes.view(torch.float8_e4m3fn).double() * torch.ldexp(
        torch.ones((), dtype=torch.float64), scales.to(torch.int32) - 127)[..., None]


class Q8Case(Case):
    """bounded_ref.Case over an 8-bit pool: pool_cpu holds the rows' values, exact in bf16."""

    def __init__(self, *args, row_gain=None, **kw):
        super().__init__(*args, **kw)
        y = self.pool_cpu.float()
        if row_gain is not None:
            y = y * row_gain(y)
        self.set_rows(y)

    def set_rows(self, y):
        self.codes_cpu, self.scales_cpu = quantise(y)
        v = values(self.codes_cpu, self.scales_cpu)
        self.pool_cpu = v.to(torch.bfloat16)
        assert torch.equal(torch.nan_to_num(self.pool_cpu.double()), torch.nan_to_num(v))

    def upload(self):
        super().upload()
        self.codes, self.scales = self.codes_cpu.cuda(), self.scales_cpu.cuda()
        self.q8 = pg.q8_descriptor(self.codes, self.scales)
        self.ws_bytes = pg.pg_q8_workspace_bytes(self.plan)
        self.ws = torch.full((max(self.ws_bytes, 16),), 0xFF, dtype=torch.uint8, device="cuda")

    def attend(self, window=-1, sinks=0, scale=1.0, lse=True):
        pg.check(pg.pg_attn_paged_q8(self.plan, self.q8, self.layer, self.q, self.out,
                                     self.lse if lse else None, window, sinks, scale, self.ws,
                                     self.ws_bytes, self.stream), "q8")

    def reference(self, window=-1, sinks=0, scale=1.0, **kw):
        ref = super().reference(window, sinks, scale, **kw)
        fin = torch.nan_to_num(self.pool_cpu[self.layer].double(), 0.0, 0.0, 0.0).abs()
        if (self.qo == 1).all():
            ksum = float(fin[:, 0].sum(-1).max())
            self.e += 4 * 2.0 ** -22 * float(self.q_cpu.double().abs().max()) * ksum * abs(scale)
            n = int(self.n.max()) if window < 0 else min(int(self.n.max()), window + 1 + sinks)
            self.floor = 2.0 ** -21 * n * float(fin[:, 1].max())
        else:
            self.floor = 0.0
        return ref

    def check_attention(self, what="", rows=None):
        out, lse, m, p, wabs = self.ref
        # (the floor is an absolute part of the output's error)
        keep = self.ref
        self.ref = (out, lse, m, p, wabs + self.floor * 2.0 ** 8)
        super().check_attention(what, rows)
        self.ref = keep
