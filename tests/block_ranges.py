"""Inputs of the block-scaled attention at the ends of its ranges, with the error bound that the
kernels' arithmetic gives.

With p_i = 2^(s_i - m) the exact weights (largest 1), L = sum p_i, v_i the exact values,
A = sum p_i |v_i| / L and S the largest sum_c |q_c k_c| * scale:
  - a weight enters P.V as fp16: off by half a step, at most 2^-11 of itself, and at most half of
    fp16's smallest step, 2^-25, where the largest weight is brought to 2^15 by the decode and to
    at least 2^7 by the prefill.  So each weight is off by 2^-40 (decode) or 2^-32 (prefill) of the
    largest, together that times sum |v_i| / L;
  - the prefill carries a value scale (a power of two here) in the widened codes from 2^-12 to 2^10 times
    the largest among the first 128 keys; what is beyond is in the weight's exponent, and that step of a
    block grows by the power of two by which its exponent lies below the largest one;
  - a score is a float32 sum of d products, off by at most (d + 4) 2^-24 S, which moves numerator and
    denominator; the hardware exponential is off by 2^-22, the mantissa of a scale by 2^-21 in the
    exponent, and a float32 sum over n weights takes n / 8 + 16 roundings in a row at most, in both;
  - the output is rounded once, by half a step, or 2^-25 where fp16 is subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

from block_cases import HALF_STEP, Batch
from oracle import block_oracle as bo


class Ranges(Batch):
    """A batch whose references carry the bound above; `step`: what one weight is off by at most."""

    step = 2.0 ** -40  # decode

    def _one(self, q, k, v, ks, vs, table, n, h):
        if n == 0:
            return np.zeros_like(q), np.full_like(q, 2.0 ** -30)
        kk, vv = bo.rows(k, ks, table, n, h), bo.rows(v, vs, table, n, h)
        out, A, S = bo.attend(q, kk, vv, self.scale)
        s = (q @ kk.T) * self.scale
        L = np.exp(s - s.max(-1, keepdims=True)).sum(-1, keepdims=True)
        each = np.abs(vv)
        if self.step > 2.0 ** -40:
            e = np.log2(np.maximum(vs[table[: -(-n // self.B)], h].astype(np.float64), 2.0 ** -64))
            all_e = np.log2(np.maximum(vs[table[table >= 0], h].astype(np.float64), 2.0 ** -64))
            ref = all_e[: max(1, 128 // self.B)].max()
            rest = [x - ref - 3 - np.clip(x - ref - 3, -15, 7) for x in (e, all_e)]
            each = each * np.exp2(max(rest[1].max(), 0.0) - np.repeat(rest[0], self.B)[:n, None])
        tiny = self.step * each.sum(0) / L
        sums = 2.0 ** -21 + 2.0 ** -22 + (n / 8 + 16) * 2.0 ** -24
        tol = (2.0 ** -11 * A + HALF_STEP[self.dtype] * np.abs(out) + A * (2 * (self.d + 4) * 2.0 ** -24 * S + 2 * sums) +
               tiny + 2.0 ** -25)
        return out, tol

    def recode(self):
        """The pools from keys16 and values16 again."""
        self.kc, self.ks = self._coded(self.keys16, True, None)
        self.vc, self.vs = self._coded(self.values16, True, None)
        return self

    def prefill(self):
        self.step = 2.0 ** -32
        return self


def one_ahead(n, gap, outlier, at, dtype, heads=2, dim=64, new=None, seed=51):
    """One sequence of n keys of which key `at` is ahead of the others, all alike, by `gap` nats, and
    whose value has one channel of `outlier`; all other values lie between 0.75 and 1.25."""
    b = Ranges([n], heads, 1, dim, 16, dtype, seed, new=new)
    g = torch.Generator().manual_seed(seed)
    b.keys16 = b.keys16.float()
    b.keys16[..., 0] = 0.0
    b.values16 = 1.0 + 0.25 * (2.0 * torch.rand(b.values16.shape, generator=g) - 1.0)
    blk, off = int(b.tables[0, at // 16]), at % 16
    b.keys16[blk, off, 0, 0] = 1.0
    b.values16[blk, off, 0, 5] = outlier
    b.recode()
    b.q = torch.zeros_like(b.q)
    b.q[..., 0] = gap * dim ** 0.5
    return b


def mixed_scales(kind, dim, new=None):
    """bfloat16 sequences whose blocks have value scales of 2^-64 and 2^100 ("two": as many of each, of
    scores that are all alike in half of the heads), or any power of two between 2^-64 and 2^100 ("all")
    or 2^-30 and 2^40 ("wide")."""
    b = Ranges([600, 64, 333], 8, 2, dim, 16, torch.bfloat16, 52, new=new)
    g = torch.Generator().manual_seed(52)
    if kind == "two":
        b.vs[:] = 2.0 ** -64
        for s, n in enumerate(b.lens_list):
            b.vs[b.tables[s, 1:-(-n // 16):2].long()] = 2.0 ** 100
        b.q[:, ::2] = 0
    else:
        lo, hi = (-64, 100) if kind == "all" else (-30, 40)
        b.vs = torch.exp2(torch.randint(lo, hi + 1, b.vs.shape, generator=g).float())
    return b
