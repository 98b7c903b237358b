"""Plain statements of packed prompt attention and of the sequences' blocks.

TEST INFRASTRUCTURE, written from the definitions in include/pagedattn.h with numpy
alone, one row, sequence or block at a time, no sharing with the CUDA path.  The
operators on blocks return new arrays and leave their inputs alone.
"""
from __future__ import annotations

import numpy as np


def up(n: int, block: int) -> int:
    return -(-n // block)


def inside(i: int, n: int) -> bool:
    return 0 <= i < n


def attention(q, key, value, starts, scale, max_len=None):
    """(out, A, S) in float64 of q [R, H, d], key and value [R, Hk, d]: out NaN where no row is computed,
    A = sum of weight * |value|, S [R, H] the largest sum |q_c k_c| * |scale| of a row's scores."""
    R, H, d = q.shape
    G = H // key.shape[1]
    out = np.full((R, H, d), np.nan)
    A, S = np.full((R, H, d), np.nan), np.zeros((R, H))
    for a, b in zip(starts[:-1], starts[1:]):
        for t in range(max(0, a), min(R, b)):
            if max_len is not None and t - a >= max_len:
                continue
            k, v = key[max(0, a):t + 1], value[max(0, a):t + 1]
            for h in range(H):
                with np.errstate(all="ignore"):
                    s = k[:, h // G] @ q[t, h] * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[t, h] = w @ v[:, h // G]
                    A[t, h] = w @ np.abs(v[:, h // G])
                    S[t, h] = (np.abs(k[:, h // G]) @ np.abs(q[t, h])).max() * abs(scale)
    return out, A, S


def truncate(tables, lens, counts, new_lens, block):
    tables, lens, counts = tables.copy(), lens.copy(), counts.copy()
    cap = tables.shape[1] * block
    for s, to in enumerate(new_lens.tolist()):
        if not 0 <= to < lens[s] <= cap:
            continue
        for i in range(up(to, block), up(int(lens[s]), block)):
            if inside(tables[s, i], len(counts)):
                counts[tables[s, i]] -= 1
            tables[s, i] = -1
        lens[s] = to
    return tables, lens, counts


def fork(tables, lens, counts, source, block):
    old, had = tables, lens
    tables, lens, counts = tables.copy(), lens.copy(), counts.copy()
    S, M = tables.shape
    for s, f in enumerate(source.tolist()):
        if not inside(f, S) or f == s or source[f] >= 0 or had[s] != 0 or not 0 < had[f] <= M * block:
            continue
        n = up(int(had[f]), block)
        tables[s, :n] = old[f, :n]
        for i in old[f, :n]:
            if inside(i, len(counts)):
                counts[i] += 1
        lens[s] = had[f]
    return tables, lens, counts


def extend(tables, lens, counts, starts, num_tokens, block):
    """tables, lens, counts, slots, copies, left"""
    was = counts
    tables, lens, counts = tables.copy(), lens.copy(), counts.copy()
    S, M = tables.shape
    N = len(counts)
    free = [i for i in range(N) if was[i] == 0]
    slots = np.full(num_tokens, -1, np.int64)
    copies = np.full((S, 2), -1, np.int64)
    refused, dry = 0, False
    for s in range(S):
        a, b, n0 = int(starts[s]), int(starts[s + 1]), int(lens[s])
        n = b - a
        if n == 0:
            continue
        if a < 0 or b < a or b > num_tokens or n0 < 0 or n0 + n > M * block:
            refused += 1
            continue
        had, want = up(n0, block), up(n0 + n, block)
        need, copy = want - had, False
        if n0 % block:
            last = int(tables[s, had - 1])
            if not inside(last, N):
                refused += 1
                continue
            copy = bool(was[last] > 1)
        need += copy
        if need and (dry or need > len(free)):
            dry = True
            refused += 1
            continue
        got, free = free[:need], free[need:]
        if copy:
            copies[s] = last, got[0]
            counts[last] -= 1
        tables[s, had - copy:want] = got
        counts[got] += 1
        lens[s] = n0 + n
        for j in range(n):
            p = n0 + j
            slots[a + j] = int(tables[s, p // block]) * block + p % block
    return tables, lens, counts, slots, copies, np.array([len(free), refused], np.int32)


def compact(tables, lens, counts, limit, block):
    """moves, number of moves, tables, counts"""
    tables, counts = tables.copy(), counts.copy()
    M = tables.shape[1]
    high = [i for i in range(len(counts) - 1, -1, -1) if counts[i] != 0]
    low = [i for i in range(len(counts)) if counts[i] == 0]
    pairs = [(a, b) for a, b in zip(high, low) if b < a][:limit]
    moves = np.full((limit, 2), -1, np.int64)
    to = {}
    for i, (a, b) in enumerate(pairs):
        moves[i] = a, b
        to[a] = b
        counts[b], counts[a] = counts[a], 0
    for s in range(len(lens)):
        for i in range(min(M, max(0, up(int(lens[s]), block)))):
            tables[s, i] = to.get(int(tables[s, i]), tables[s, i])
    return moves, len(pairs), tables, counts


def holders(tables, lens, num_blocks, block):
    """The counts that the tables call for."""
    counts = np.zeros(num_blocks, np.int32)
    for s, n in enumerate(lens.tolist()):
        for i in tables[s, :up(n, block)].tolist():
            counts[i] += 1
    return counts
