"""Packed prefill and the calls on the sequences' blocks: bad arguments are rejected on the
host (no kernel is launched, so no GPU is needed), and the oracle's statements hold together."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import sequence_oracle as so
from paged_kv_cache_173_gb300 import _lib, api

A = 1 << 20  # a fake, 16-byte aligned "device" address: never dereferenced on these paths
INVALID, UNSUPPORTED, OK = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED, _lib.PA_OK


@pytest.fixture(scope="module")
def L():
    from paged_kv_cache_173_gb300.build import build_library
    build_library()
    return _lib.lib()


def call(L, name, defaults, **kw):
    args = dict(defaults)
    for k in kw:
        assert k in args, k
    args.update(kw)
    return getattr(L, name)(*args.values())


PACKED = dict(out=A, q=A, qs=1024, key=A, ks=256, value=A, vs=256, kc=A, vc=A, sm=A, qsl=A, S=2, R=100, maxq=64, H=8, Hk=2,
              d=128, B=16, N=32, scale=0.1, dtype=0, stream=None)
NONE = dict(kc=None, vc=None, sm=None)


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(key=None), INVALID), (dict(value=None), INVALID),
    (dict(qsl=None), INVALID), (dict(qsl=A + 2), INVALID), (dict(out=A + 8), INVALID), (dict(key=A + 2), INVALID),
    (dict(qs=1016), INVALID), (dict(ks=248), INVALID), (dict(vs=0), INVALID), (dict(qs=-1024), INVALID),
    (dict(qs=1028), UNSUPPORTED), (dict(ks=260), UNSUPPORTED), (dict(vs=1 << 39), UNSUPPORTED),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(sm=None), INVALID), (dict(sm=A + 4), INVALID),
    (dict(kc=A + 8), INVALID), (dict(N=0), INVALID), (dict(B=0), INVALID), (dict(R=-1), INVALID), (dict(S=-1), INVALID),
    (dict(maxq=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(H=7), UNSUPPORTED),
    (dict(H=34, qs=34 * 128), UNSUPPORTED), (dict(S=70000), UNSUPPORTED), (dict(R=2 ** 31 - 1), UNSUPPORTED),
    (dict(R=0, q=None, key=None), OK), (dict(S=0, qsl=None), OK), (dict(maxq=0, out=None), OK),
    (dict(R=0, N=0, B=0, **NONE), OK),
])
def test_packed_prefill_checks_arguments(L, kw, status):
    assert call(L, "pa_prefill_packed", PACKED, **kw) == status
    assert (_lib.last_error() == "") == (status == OK)


STATE = dict(bt=A, M=8, cl=A, rc=A)
STATE_ERRORS = [
    (dict(bt=None), INVALID), (dict(cl=None), INVALID), (dict(rc=None), INVALID), (dict(rc=A + 4), INVALID),
    (dict(bt=A + 2), INVALID), (dict(cl=A + 1), INVALID), (dict(M=0), INVALID), (dict(S=-1), INVALID), (dict(N=0), INVALID),
    (dict(B=8), UNSUPPORTED), (dict(B=24), UNSUPPORTED), (dict(B=512), UNSUPPORTED), (dict(S=65536), UNSUPPORTED),
    (dict(N=1 << 27), UNSUPPORTED), (dict(M=2 ** 27 - 1), UNSUPPORTED),
]
TRUNCATE = dict(STATE, nl=A, S=3, N=32, B=16, stream=None)
EXTEND = dict(STATE, qsl=A, sm=A, bc=A, left=A, S=3, T=5, N=32, B=16, ws=A, wsb=(32 + 16) * 4, stream=None)
COMPACT = dict(moves=A, K=4, num=A, bt=A, M=8, cl=A, rc=A, to=A, co=A, S=3, N=32, B=16, ws=A, wsb=(32 + 16) * 4, stream=None)


@pytest.mark.parametrize("name,args", [("pa_truncate_sequences", TRUNCATE), ("pa_fork_sequences", TRUNCATE),
                                       ("pa_extend_sequences", EXTEND), ("pa_compact_blocks", COMPACT)])
@pytest.mark.parametrize("kw,status", STATE_ERRORS)
def test_calls_check_the_sequences_arguments(L, name, args, kw, status):
    assert call(L, name, args, **kw) == status
    assert _lib.last_error() != ""


@pytest.mark.parametrize("name,args,kw,status", [
    ("pa_truncate_sequences", TRUNCATE, dict(nl=None), INVALID), ("pa_truncate_sequences", TRUNCATE, dict(nl=A + 2), INVALID),
    ("pa_truncate_sequences", TRUNCATE, dict(S=0, bt=None, cl=None, nl=None), OK),
    ("pa_fork_sequences", TRUNCATE, dict(nl=None), INVALID), ("pa_fork_sequences", TRUNCATE, dict(S=0, nl=None), OK),
    ("pa_extend_sequences", EXTEND, dict(qsl=None), INVALID), ("pa_extend_sequences", EXTEND, dict(sm=None), INVALID),
    ("pa_extend_sequences", EXTEND, dict(bc=None), INVALID), ("pa_extend_sequences", EXTEND, dict(left=None), INVALID),
    ("pa_extend_sequences", EXTEND, dict(sm=A + 4), INVALID), ("pa_extend_sequences", EXTEND, dict(T=-1), INVALID),
    ("pa_extend_sequences", EXTEND, dict(T=2 ** 31 - 1), UNSUPPORTED), ("pa_extend_sequences", EXTEND, dict(ws=None), INVALID),
    ("pa_extend_sequences", EXTEND, dict(ws=A + 8), INVALID), ("pa_extend_sequences", EXTEND, dict(wsb=48 * 4 - 1), INVALID),
    ("pa_compact_blocks", COMPACT, dict(moves=None), INVALID), ("pa_compact_blocks", COMPACT, dict(K=-1), INVALID),
    ("pa_compact_blocks", COMPACT, dict(num=None), INVALID), ("pa_compact_blocks", COMPACT, dict(to=None), INVALID),
    ("pa_compact_blocks", COMPACT, dict(co=None), INVALID), ("pa_compact_blocks", COMPACT, dict(co=A + 4), INVALID),
    ("pa_compact_blocks", COMPACT, dict(K=2 ** 31 - 1), UNSUPPORTED), ("pa_compact_blocks", COMPACT, dict(ws=None), INVALID),
    ("pa_compact_blocks", COMPACT, dict(wsb=0), INVALID),
])
def test_calls_check_their_own_arguments(L, name, args, kw, status):
    assert call(L, name, args, **kw) == status


COPY = dict(pools=A, stride=32 * 4096, P=4, bytes=4096, bm=A, n=3, N=32, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(pools=None), INVALID), (dict(bm=None), INVALID), (dict(pools=A + 2), INVALID), (dict(bm=A + 4), INVALID),
    (dict(stride=32 * 4096 - 4), INVALID), (dict(stride=32 * 4096 + 2), UNSUPPORTED), (dict(bytes=4094), UNSUPPORTED),
    (dict(bytes=0), INVALID), (dict(bytes=(1 << 30) + 4), UNSUPPORTED), (dict(N=0), INVALID), (dict(P=-1), INVALID),
    (dict(P=65536), UNSUPPORTED), (dict(n=-1), INVALID), (dict(n=0, bm=None), OK), (dict(P=0, pools=None), OK),
])
def test_copy_checks_arguments(L, kw, status):
    assert call(L, "pa_copy_layer_blocks", COPY, **kw) == status


def test_workspace_size(L):
    assert L.pa_sequence_workspace_bytes(1) == 20 * 4
    assert L.pa_sequence_workspace_bytes(4096) == (4096 + 16) * 4
    assert L.pa_sequence_workspace_bytes(0) == 0 and L.pa_sequence_workspace_bytes(-3) == 0


def test_binding_wants_device_tensors():
    t, v = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        api.pa_truncate_sequences(t, v, v, v, 16)
    with pytest.raises(ValueError, match="CUDA"):
        api.pa_prefill_packed(x, x, x, x, v, 3, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        api.pa_copy_layer_blocks(x, torch.zeros(1, 2, dtype=torch.int64))


# ------------------------------------------------------------------ the oracle
def random_walk(seed, steps=60, S=6, M=9, N=40, B=16):
    """States that a server passes through: (tables, lens, counts) after each call, and what the calls gave."""
    rng = np.random.default_rng(seed)
    tables, lens, counts = np.full((S, M), -1, np.int32), np.zeros(S, np.int32), np.zeros(N, np.int32)
    for _ in range(steps):
        op = rng.integers(0, 5)
        if op <= 1:
            new = rng.integers(0, 40, S) * (rng.random(S) < 0.5)
            starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            tables, lens, counts, slots, copies, left = so.extend(tables, lens, counts, starts, int(starts[-1]) + 2, B)
            taken = slots[slots >= 0]
            assert len(set(taken.tolist())) == len(taken) and slots[-2:].tolist() == [-1, -1]
            assert left[0] == (counts == 0).sum() - len({a for a, _ in copies.tolist() if a >= 0 and counts[a] == 0})
            # a block that new tokens are written into has one holder
            assert all(counts[x // B] == 1 for x in taken.tolist())
        elif op == 2:
            to = np.where(rng.random(S) < 0.4, rng.integers(-1, 100, S) * (rng.random(S) < 0.5), -1)
            tables, lens, counts = so.truncate(tables, lens, counts, to, B)
        elif op == 3:
            tables, lens, counts = so.fork(tables, lens, counts, np.where(rng.random(S) < 0.5, rng.integers(0, S, S), -1), B)
        else:
            limit = int(rng.integers(0, N))
            used = int((counts != 0).sum())
            moves, n, tables, counts = so.compact(tables, lens, counts, limit, B)
            if n < limit:
                assert not counts[used:].any() and counts[:used].all()
        assert np.array_equal(counts, so.holders(tables, lens, N, B))
        yield tables, lens, counts


def test_oracle_keeps_counts_and_tables_in_agreement():
    grown = 0
    for seed in range(20):
        for tables, lens, counts in random_walk(seed):
            grown = max(grown, int(counts.max()))
    assert grown > 2  # blocks were shared on the way


def test_oracle_attention_matches_torch():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((12, 6, 16), (12, 2, 16), (12, 2, 16)))
    out, A_, S_ = so.attention(q.numpy(), k.numpy(), v.numpy(), [0, 5, 5, 12], 0.3)
    for a, b in ((0, 5), (5, 12)):
        want = torch.nn.functional.scaled_dot_product_attention(
            q[a:b].transpose(0, 1), k[a:b].repeat_interleave(3, 1).transpose(0, 1), v[a:b].repeat_interleave(3, 1).transpose(0, 1),
            is_causal=True, scale=0.3).transpose(0, 1)
        assert np.allclose(out[a:b], want.numpy(), atol=1e-12)
    assert (np.abs(out) <= A_ + 1e-12).all()
    assert np.isnan(so.attention(q.numpy(), k.numpy(), v.numpy(), [0, 5, 5, 12], 0.3, 3)[0][3]).all()


def test_the_short_way_declines_what_it_does_not_know(L):
    fast = _lib.fast()
    x = torch.zeros(2, 3, 4, dtype=torch.float16)
    for name, n in dict(packed=12, extend=11, truncate=7, fork=7, compact=11, copy_layers=4).items():
        f = getattr(fast, name)
        assert f() is False and f(*[None] * n) is False and f(*[x] * n) is False
        assert f(*[x] * (n - 2), 0, 0) is False                 # host tensors
        assert f(*[x] * (n - 2), -1, 0) is False and f(*[x] * (n - 2), 0, 1 << 70) is False
        assert f(*[object()] * (n - 2), 1 << 70, 0) is False    # numbers past 64 bits
    with pytest.raises(TypeError):
        fast.bind_sequences(1, 2)
    with pytest.raises(ValueError):
        fast.bind_sequences(*[0] * 6)


def test_the_short_way_takes_one_function_for_failed_launches(L):
    fast = _lib.fast()
    for args in ((), (1,), (print, print)):
        with pytest.raises(TypeError):
            fast.bind_check(*args)


@pytest.mark.parametrize("scale,status", [(2.3e38, OK), (-2.3e38, OK), (3e38, UNSUPPORTED), (-2.4e38, UNSUPPORTED), (3.4028234e38, UNSUPPORTED),
                                          (float("nan"), INVALID), (-float("inf"), INVALID)])
def test_packed_prefill_takes_scales_whose_powers_of_two_exist(L, scale, status):
    assert call(L, "pa_prefill_packed", PACKED, scale=scale, R=0) == status  # (no rows: nothing is launched)
