"""Inputs, references and tolerances shared by the tests of the per-block operators.

Tolerance of an attention output, from the arithmetic.  With w_i the exact
weights (sum 1), A = sum w_i |v_i| and S = the largest sum_c |q_c k_c| * scale:
  - the weights enter P.V in fp16: each is off by at most 2^-11 of itself (half
    a step), together 2^-11 A; below 2^-14 of the largest the step is absolute,
    2^-25 of the largest product's unit: at most 2^-24 * (sum |v_i| / scale_i)
    times the largest value scale;
  - 16-bit pools of fp16 divide by the sum of the rounded weights: 2^-11 |out|;
  - a score is a float32 sum of d products: off by at most (d + 4) 2^-24 S
    (the exponent's unit is cancelled between score and factor), which moves
    numerator and denominator: 2 (d + 4) 2^-24 S A; the hardware exponential
    is off by 2^-22, and a float32 sum over n weights takes n / 8 + 16 roundings
    in a row at most, in numerator and denominator: 2 (2^-22 + (n / 8 + 16) 2^-24) A;
  - the output is rounded once: half a step, 2^-11 |out| (fp16) or 2^-8 |out| (bf16).
Subnormal outputs add half of fp16's smallest step, 2^-25.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import block_oracle as bo

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def tolerance(dtype, ref, A, S, d, n, tiny):
    sums = 2.0 ** -22 + (n / 8 + 16) * 2.0 ** -24
    return (2.0 ** -11 * (A + np.abs(ref)) + HALF_STEP[dtype] * np.abs(ref) +
            A * (2 * (d + 4) * 2.0 ** -24 * S + 2 * sums) + tiny + 2.0 ** -25)


def to_np(t: torch.Tensor) -> np.ndarray:
    """float64 values of a float tensor, integers as they are."""
    if t.dtype in (torch.float16, torch.bfloat16, torch.float32):
        return t.double().cpu().numpy()
    return t.cpu().numpy()


class Batch:
    """One layer's block-scaled pools and tables, drawn on the CPU from a seed."""

    def __init__(self, lens, heads, kv_heads, dim, block, dtype, seed, slack=1, pow2=True, new=None, wide=False):
        g = torch.Generator().manual_seed(seed)
        self.lens_list = list(lens)
        S, B = len(self.lens_list), block
        counts = [-(-max(n, 0) // B) for n in self.lens_list]
        self.M = max(1, max(counts)) + slack
        N = sum(counts) + 3
        perm = torch.randperm(N, generator=g).int()
        self.tables = torch.full((S, self.M), -1, dtype=torch.int32)
        at = 0
        for s, c in enumerate(counts):
            self.tables[s, :c] = perm[at:at + c]
            at += c
        self.lens = torch.tensor(self.lens_list, dtype=torch.int32)
        self.H, self.Hk, self.d, self.B, self.N, self.dtype = heads, kv_heads, dim, block, N, dtype
        self.G = heads // kv_heads
        shape = (N, B, kv_heads, dim)
        keys = torch.randn(shape, generator=g) * torch.exp(0.5 * torch.randn((kv_heads, dim), generator=g))
        spread = 2.0 if wide else 0.7
        values = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn((N, 1, kv_heads, 1), generator=g))
        self.keys16, self.values16 = keys.to(dtype), values.to(dtype)
        self.kc, self.ks = self._coded(self.keys16, pow2, g)
        self.vc, self.vs = self._coded(self.values16, pow2, g)
        rows = S
        if new is not None:
            self.new = list(new)
            rows = sum(self.new)
            self.starts = torch.tensor([0] + list(np.cumsum(self.new)), dtype=torch.int32)
        self.q = (torch.randn((rows, heads, dim), generator=g)).to(dtype)
        self.scale = float(np.float32(dim ** -0.5))

    def _coded(self, x, pow2, g):
        a = x.double().abs().amax(dim=(1, 3))
        s = torch.exp2(torch.ceil(torch.log2(a / 448.0))).float()
        if not pow2:  # any float is a scale
            s = s * (1.0 + torch.rand(s.shape, generator=g))
        codes = torch.from_numpy(bo.encode((x.double() / s.double()[:, None, :, None]).numpy()))
        return codes, s

    def poison(self, codes=0x7F):
        """NaN in every slot that must not be read, and in the scales of unused blocks."""
        used = torch.zeros((self.N, self.B), dtype=torch.bool)
        for s, n in enumerate(self.lens_list):
            for i in range(-(-max(n, 0) // self.B)):
                used[int(self.tables[s, i]), : min(self.B, n - i * self.B)] = True
        for c in (self.kc, self.vc):
            c[~used] = codes
        for c in (self.keys16, self.values16):
            c[~used] = float("nan")
        for t in (self.ks, self.vs):
            t[~used.any(1)] = float("nan")
        return self

    def dev(self, *names):
        return [getattr(self, n).cuda() for n in names]

    def reference(self, fp8=True, tables=None, lens=None):
        """(out, tolerance) for the decode of every sequence over its own table, or per-head tables."""
        out = np.zeros((len(self.lens_list), self.H, self.d))
        tol = np.zeros_like(out)
        q = to_np(self.q)
        k, v, ks, vs = self.pools(fp8)
        for s in range(len(self.lens_list)):
            for h in range(self.Hk):
                n = int(self.lens[s]) if lens is None else int(lens[s, h])
                table = self.tables[s].numpy() if tables is None else tables[s, h]
                hs = slice(h * self.G, (h + 1) * self.G)
                out[s, hs], tol[s, hs] = self._one(q[s, hs], k, v, ks, vs, table, n, h)
        return out, tol

    def pools(self, fp8):
        if fp8:
            return self.kc.numpy(), self.vc.numpy(), self.ks.numpy(), self.vs.numpy()
        return to_np(self.keys16), to_np(self.values16), None, None

    def _one(self, q, k, v, ks, vs, table, n, h):
        if n == 0:
            return np.zeros_like(q), np.full_like(q, 2.0 ** -30)
        kk, vv = bo.rows(k, ks, table, n, h), bo.rows(v, vs, table, n, h)
        ref, A, S = bo.attend(q, kk, vv, self.scale)
        if vs is None:
            tiny = 2.0 ** -24 * np.abs(vv).sum(0)
        else:
            ids = np.asarray(table[: -(-n // self.B)], np.int64)
            per = np.repeat(vs[ids, h].astype(np.float64), self.B)[:n, None]
            tiny = 2.0 ** -24 * np.abs(np.divide(vv, per, out=np.zeros_like(vv), where=per > 0)).sum(0) * per.max()
        return ref, tolerance(self.dtype, ref, A, S, self.d, n, tiny)

    def prefill_reference(self):
        q = to_np(self.q)
        out, tol = np.zeros_like(q), np.zeros_like(q)
        k, v, ks, vs = self.pools(True)
        for s, n in enumerate(self.lens_list):
            r0 = int(self.starts[s])
            for i in range(self.new[s]):
                for h in range(self.Hk):
                    hs = slice(h * self.G, (h + 1) * self.G)
                    out[r0 + i, hs], tol[r0 + i, hs] = self._one(q[r0 + i, hs], k, v, ks, vs, self.tables[s].numpy(),
                                                                 n - self.new[s] + i + 1, h)
        return out, tol


def assert_close(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray):
    g = to_np(got)
    assert np.isfinite(g).all(), "non-finite output"
    over = np.abs(g - ref) / tol
    assert over.max() <= 1.0, f"error {over.max():.3f} of the tolerance"
