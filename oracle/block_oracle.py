"""Float64 statements of the per-block operators: block-scaled E4M3 caches, key
bounds, block selection and attention over them.

TEST INFRASTRUCTURE, written from the definitions in include/pagedattn.h with
numpy alone: one token, block or head at a time, no sharing with the CUDA
path.  Codes are decoded and encoded from the format's definition.
"""
from __future__ import annotations

import math

import numpy as np

MIN_SCALE_EXP = -64
MIN_BOUND_EXP = -100


def _e4m3_table() -> np.ndarray:
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return t


E4M3 = _e4m3_table()


def encode(x: np.ndarray) -> np.ndarray:
    """The E4M3 code nearest to each float64, ties to the even code, saturating at +-448; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    mag = E4M3[:127]  # 0 .. 448, increasing
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(mag, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mag[lo], mag[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = pick.astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(127) | (np.signbit(x).astype(np.uint8) << 7), code).astype(np.uint8)


def least_exp(amax: float, top: float, floor: int) -> int:
    e = floor
    if amax > 0:
        e = max(floor, math.frexp(amax / top)[1] - 1)
        while math.ldexp(top, e) < amax:
            e += 1
    return e


def _amax(x: np.ndarray) -> float:
    a = np.abs(x[np.isfinite(x)])
    return float(a.max()) if a.size else 0.0


def runs(slots: np.ndarray, num_blocks: int, block: int):
    """(block, [token, ...]) of every block that the mapping names."""
    found = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < num_blocks * block:
            found.setdefault(s // block, []).append(t)
    return found.items()


def write(new: np.ndarray, codes: np.ndarray, scales: np.ndarray, slots: np.ndarray):
    """pa_reshape_and_cache_fp8_block for one pool: (codes, scales) after the write."""
    codes, scales = codes.copy(), scales.astype(np.float32).copy()
    N, B, Hk, _ = codes.shape
    x = new.astype(np.float64)
    for blk, toks in runs(slots, N, B):
        offs = [int(slots[t]) % B for t in toks]
        for h in range(Hk):
            need = math.ldexp(1.0, least_exp(_amax(x[toks, h]), 448.0, MIN_SCALE_EXP))
            old = float(scales[blk, h])
            old = 0.0 if 0 in offs or not (0.0 < old < math.inf) else old
            s = max(old, need)
            if 0.0 < old < s:
                ratio = float(np.float32(old) / np.float32(s))
                # the product is rounded to float32, then to a code
                moved = np.float32(E4M3[codes[blk, :, h]]) * np.float32(ratio)
                codes[blk, :, h] = encode(moved.astype(np.float64))
            q = (np.float32(x[toks, h]) / np.float32(s)).astype(np.float64)  # the float32 quotient
            codes[blk, offs, h] = encode(q)
            scales[blk, h] = s
    return codes, scales


def bounds(keys: np.ndarray, codes: np.ndarray, exps: np.ndarray, slots: np.ndarray, block: int):
    """pa_update_key_bounds: (key_bounds, bound_exps) after the call."""
    codes, exps = codes.copy(), exps.copy()
    N, Hk, _, d = codes.shape
    x = keys.astype(np.float64)
    for blk, toks in runs(slots, N, block):
        starts = any(int(slots[t]) % block == 0 for t in toks)
        for h in range(Hk):
            k = x[toks, h]
            e = least_exp(_amax(k), 127.0, MIN_BOUND_EXP)
            if not starts:
                e = max(e, int(exps[blk, h]))
            u = math.ldexp(1.0, e)
            lo = np.floor(np.where(np.isnan(k), -np.inf, k).min(0) / u)
            hi = np.ceil(np.where(np.isnan(k), np.inf, k).max(0) / u)
            lo, hi = np.maximum(np.minimum(lo, 127), -127), np.minimum(np.maximum(hi, -127), 127)
            if not starts:
                r = math.ldexp(1.0, int(exps[blk, h]) - e)
                lo = np.minimum(lo, np.floor(codes[blk, h, 0] * r))
                hi = np.maximum(hi, np.ceil(codes[blk, h, 1] * r))
            codes[blk, h, 0], codes[blk, h, 1], exps[blk, h] = lo, hi, e
    return codes, exps


def scores(q: np.ndarray, codes: np.ndarray, exps: np.ndarray, ids) -> np.ndarray:
    """Scores of the blocks `ids` for the query heads q [G, d] of one KV head (codes [N, 2, d], exps [N])."""
    N = codes.shape[0]
    out = np.full(len(ids), -np.inf)
    for row in q.astype(np.float64):
        f = least_exp(_amax(row), 255.0, MIN_BOUND_EXP)
        qi = np.clip(np.rint(np.where(np.isnan(row), 0.0, row) / math.ldexp(1.0, f)), -255, 255)
        for i, b in enumerate(ids):
            if not 0 <= b < N:
                out[i] = np.inf
                continue
            dot = (qi * np.where(qi >= 0, codes[b, 1], codes[b, 0])).sum()
            out[i] = max(out[i], math.ldexp(dot, min(max(f + int(exps[b]), -100), 100)))
    return out


def select(q, codes, exps, tables, lens, block, keep, first, last):
    """pa_select_blocks: (sel_tables, sel_lens)."""
    S, M = tables.shape
    N, Hk = exps.shape
    G = q.shape[1] // Hk
    ids_out = np.full((S, Hk, keep), -1, np.int32)
    lens_out = np.empty((S, Hk), np.int32)
    for s in range(S):
        ctx = int(lens[s])
        if ctx < 0 or ctx > M * block:
            lens_out[s] = -1
            continue
        n = -(-ctx // block)
        for h in range(Hk):
            ids = tables[s, :n].tolist()
            if n > keep:
                sc = scores(q[s, h * G:(h + 1) * G], codes[:, h], exps[:, h], ids)
                forced = [i < first or i >= n - last for i in range(n)]
                order = sorted(range(n), key=lambda i: (not forced[i], -sc[i], i))
                ids = [ids[i] for i in sorted(order[:keep])]
            ids_out[s, h, :len(ids)] = ids
            lens_out[s, h] = ctx - (n - len(ids)) * block
    return ids_out, lens_out


def rows(pool, scales, table, n, h):
    """The first n rows along a table for KV head h, float64 [n, d]; scales None for value pools."""
    B = pool.shape[1]
    ids = np.asarray(table[: -(-n // B)], np.int64)
    x = pool[ids, :, h].reshape(-1, pool.shape[3])[:n]
    if scales is None:
        return x.astype(np.float64)
    return E4M3[x] * np.repeat(scales[ids, h].astype(np.float64), B)[:n, None]


def attend(q, k, v, scale):
    """(out, sum of weights times |v|, largest sum of |q k| * scale) of rows q [R, d] over k, v [n, d]."""
    s = (q @ k.T) * scale
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return w @ v, w @ np.abs(v), (np.abs(q) @ np.abs(k).T * scale).max(-1, keepdims=True)
