"""The per-block entry points reject bad arguments on the host (no kernel is
launched, so no GPU is needed), and the float64 oracle of their definitions
meets independent statements of them."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
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


WRITE = dict(key=A, value=A, k=A, v=A, ks=A, vs=A, sm=A, T=4, N=8, B=16, Hk=2, d=128, dtype=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(key=None), INVALID), (dict(value=A + 8), INVALID), (dict(k=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=None), INVALID), (dict(vs=A + 2), INVALID), (dict(sm=A + 4), INVALID), (dict(T=-1), INVALID),
    (dict(N=0), INVALID), (dict(B=8), UNSUPPORTED), (dict(B=48), UNSUPPORTED), (dict(B=512), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(Hk=70000), UNSUPPORTED),
    (dict(N=1 << 28), UNSUPPORTED), (dict(T=0, key=None, ks=None), OK),
])
def test_write_checks_arguments(L, kw, status):
    assert call(L, "pa_reshape_and_cache_fp8_block", WRITE, **kw) == status
    assert (_lib.last_error() == "") == (status == OK)


BOUNDS = dict(key=A, b=A, e=A, sm=A, T=4, N=8, B=16, Hk=2, d=128, dtype=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(key=None), INVALID), (dict(b=None), INVALID), (dict(b=A + 4), INVALID), (dict(e=None), INVALID),
    (dict(e=A + 1), INVALID), (dict(sm=None), INVALID), (dict(T=-2), INVALID), (dict(B=20), UNSUPPORTED),
    (dict(d=72), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(T=0, e=None), OK),
])
def test_bounds_check_arguments(L, kw, status):
    assert call(L, "pa_update_key_bounds", BOUNDS, **kw) == status


DECODE = dict(out=A, q=A, k=A, v=A, ks=A, vs=A, bt=A, M=8, cl=A, S=2, H=8, Hk=2, d=128, B=16, N=32, scale=0.1,
              dtype=0)


@pytest.mark.parametrize("splitk", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=A + 2), INVALID), (dict(ks=None), INVALID), (dict(vs=A + 3), INVALID),
    (dict(bt=None), INVALID), (dict(M=0), INVALID), (dict(scale=float("nan")), INVALID), (dict(S=-1), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(B=8), UNSUPPORTED), (dict(H=6, Hk=4), UNSUPPORTED),
    (dict(H=64, Hk=2), UNSUPPORTED), (dict(d=256, H=32, Hk=2), UNSUPPORTED), (dict(S=70000), UNSUPPORTED),
    (dict(S=0, q=None, ks=None), OK), (dict(S=0, dtype=1), OK),
])
def test_decode_checks_arguments(L, splitk, kw, status):
    tail = dict(ps=64, P=2, ws=A, wsb=10 ** 9, stream=None) if splitk else dict(stream=None)
    name = "pa_decode_splitk_fp8_block" if splitk else "pa_decode_fp8_block"
    assert call(L, name, {**DECODE, **tail}, **kw) == status


@pytest.mark.parametrize("kw", [dict(ps=40), dict(ps=0), dict(P=1), dict(ws=None), dict(wsb=100), dict(ws=A + 4)])
def test_splitk_checks_its_workspace(L, kw):
    tail = dict(ps=64, P=2, ws=A, wsb=10 ** 9, stream=None)
    assert call(L, "pa_decode_splitk_fp8_block", {**DECODE, **tail}, **kw) == INVALID


PREFILL = dict(out=A, q=A, k=A, v=A, ks=A, vs=A, bt=A, M=8, cl=A, qsl=A, S=2, R=100, maxq=64, H=8, Hk=2, d=128, B=16,
               N=32, scale=0.1, dtype=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=256), UNSUPPORTED), (dict(H=6, Hk=2), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(qsl=None), INVALID),
    (dict(qsl=A + 2), INVALID), (dict(maxq=-1), INVALID), (dict(R=-1), INVALID), (dict(ks=None), INVALID),
    (dict(vs=A + 2), INVALID), (dict(B=24), UNSUPPORTED), (dict(S=0, qsl=None, ks=None), OK),
    (dict(maxq=0, qsl=None, vs=None), OK), (dict(R=0), OK),
])
def test_prefill_checks_arguments(L, kw, status):
    assert call(L, "pa_prefill_fp8_block", PREFILL, **kw) == status


SELECT = dict(st=A, sl=A, q=A, b=A, e=A, bt=A, M=64, cl=A, S=2, H=8, Hk=2, d=128, B=16, N=32, keep=8, first=1, last=2,
              dtype=0, ws=A, wsb=2 * 2 * 64 * 4, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(st=None), INVALID), (dict(sl=A + 2), INVALID), (dict(q=None), INVALID), (dict(b=A + 8), INVALID),
    (dict(e=None), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 8), INVALID), (dict(wsb=2 * 2 * 64 * 4 - 1), INVALID),
    (dict(first=-1), INVALID), (dict(last=0), INVALID), (dict(first=6, last=3), INVALID), (dict(keep=0), INVALID),
    (dict(first=2 ** 31 - 1), INVALID), (dict(M=0), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(d=80), UNSUPPORTED),
    (dict(B=512), UNSUPPORTED), (dict(keep=2 ** 30), UNSUPPORTED), (dict(S=0, st=None, ws=None), OK),
])
def test_select_checks_arguments(L, kw, status):
    assert call(L, "pa_select_blocks", SELECT, **kw) == status


def test_select_workspace_size(L):
    assert L.pa_select_workspace_bytes(3, 8, 101) == 3 * 8 * 104 * 4
    assert L.pa_select_workspace_bytes(0, 8, 101) == 0
    assert L.pa_select_workspace_bytes(3, 8, -1) == 0


SPARSE = dict(out=A, q=A, k=A, v=A, ks=A, vs=A, st=A, K=8, sl=A, S=2, H=8, Hk=2, d=128, B=16, N=32, scale=0.1, dtype=0,
              kv=2, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(st=None), INVALID), (dict(sl=A + 1), INVALID), (dict(K=0), INVALID),
    (dict(ks=None), INVALID), (dict(kv=1), UNSUPPORTED), (dict(dtype=1, kv=0), UNSUPPORTED), (dict(kv=3), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(S=0, kv=0, ks=None, vs=None), OK), (dict(S=0, q=None, ks=None), OK),
])
def test_sparse_decode_checks_arguments(L, kw, status):
    assert call(L, "pa_decode_sparse", SPARSE, **kw) == status


def test_binding_checks_shapes_and_types():
    # the checks that need no device come before the one for a CUDA tensor
    with pytest.raises(ValueError, match="CUDA"):
        x = torch.zeros(2, 4, 64, dtype=torch.float16)
        api.pa_decode_sparse(x, x, x, x, x, x, 0.1)


# ------------------------------------------------------------------ the oracle
def test_codes_match_torch():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(50000, generator=g) * 100
    x = torch.cat([x, x * 2.0 ** -12, torch.arange(0, 449) / 16.0, torch.arange(0, 200) * 2.0 ** -12])
    x = x[x.abs() <= 448]
    want = x.to(torch.float8_e4m3fn)
    assert np.array_equal(bo.encode(x.double().numpy()), want.view(torch.uint8).numpy())
    every = torch.arange(256).to(torch.uint8)
    assert np.array_equal(bo.E4M3, every.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    assert bo.encode(np.array([1e9, -math.inf, math.nan])).tolist() == [0x7E, 0xFE, 0x7F]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (449, 1), (224, -1), (1.75, -8), (1.76, -7), (0.0, -64),
                                    (2.0 ** -80, -64), (65504, 8)])
def test_scale_exponents(amax, e):
    assert bo.least_exp(amax, 448.0, -64) == e
    if e > -64:
        assert 448.0 * 2.0 ** e >= amax > 448.0 * 2.0 ** (e - 1)


def test_block_write_quantises_within_half_a_step_and_growth_is_nearly_free():
    rng = np.random.default_rng(0)
    codes, scales = np.zeros((2, 16, 1, 64), np.uint8), np.zeros((2, 1), np.float32)
    x = rng.standard_normal((16, 1, 64)) * np.exp(rng.standard_normal((16, 1, 1)))
    for t in range(16):
        codes, scales = bo.write(x[t:t + 1], codes, scales, np.array([16 + t]))
    once = bo.write(x, np.zeros_like(codes), np.zeros_like(scales), np.arange(16, 32))
    assert scales[1, 0] == once[1][1, 0]  # the scale does not depend on the calls
    got = bo.E4M3[codes[1]] * scales[1, 0]
    # half a step: 2^-4 relative, or half of the smallest subnormal step, twice where a code moved
    assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2 * 2.0 ** -10 * scales[1, 0])).all()
    normal = np.abs(x) >= 2.0 ** -6 * scales[1, 0]
    assert np.array_equal(codes[1][normal], once[0][1][normal])
    assert (codes[0] == 0).all()


def test_bounds_hold_every_key_and_scores_bound_every_product():
    rng = np.random.default_rng(1)
    keys = rng.standard_normal((96, 2, 64)) * np.exp(rng.standard_normal((96, 1, 1)))
    codes, exps = np.zeros((6, 2, 2, 64), np.int8), np.zeros((6, 2), np.int32)
    for t in range(96):
        codes, exps = bo.bounds(keys[t:t + 1], codes, exps, np.array([t]), 16)
    once = bo.bounds(keys, np.zeros_like(codes), np.zeros_like(exps), np.arange(96), 16)
    assert np.array_equal(codes, once[0]) and np.array_equal(exps, once[1])
    u = 2.0 ** exps[:, :, None]
    k = keys.reshape(6, 16, 2, 64)
    assert (codes[:, :, 0] * u <= k.min(1)).all() and (codes[:, :, 1] * u >= k.max(1)).all()
    q = rng.integers(-255, 256, (4, 64)).astype(np.float64)
    q[:, 0] = 255  # whole numbers with exponent 0: the score is a bound, not an estimate
    for h in range(2):
        sc = bo.scores(q, codes[:, h], exps[:, h], range(6))
        assert (sc >= np.einsum("gd,btd->bgt", q, k[:, :, h]).max((1, 2))).all()


def test_selection_keeps_the_best_and_the_forced():
    rng = np.random.default_rng(2)
    keys = rng.standard_normal((320, 1, 64))
    codes, exps = bo.bounds(keys, np.zeros((20, 1, 2, 64), np.int8), np.zeros((20, 1), np.int32), np.arange(320), 16)
    tables = rng.permutation(20).astype(np.int32)[None]
    q = rng.standard_normal((1, 2, 64))
    ids, lens = bo.select(q, codes, exps, tables, np.array([310]), 16, 7, 2, 1)
    assert lens[0, 0] == 310 - 13 * 16
    kept = ids[0, 0].tolist()
    assert kept[:2] == tables[0, :2].tolist() and kept[-1] == tables[0, 19]
    sc = bo.scores(q[0], codes[:, 0], exps[:, 0], tables[0].tolist())
    middle = sorted(range(2, 19), key=lambda i: -sc[i])[:4]
    assert kept[2:6] == [tables[0, i] for i in sorted(middle)]
    ids, lens = bo.select(q, codes, exps, tables, np.array([33]), 16, 7, 2, 1)
    assert ids[0, 0].tolist() == tables[0, :3].tolist() + [-1] * 4 and lens[0, 0] == 33


def test_attention_matches_torch():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 32), (50, 32), (50, 32)))
    out, A_, S = bo.attend(q.numpy(), k.numpy(), v.numpy(), 0.3)
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], scale=0.3)[0]
    assert np.allclose(out, want.numpy(), atol=1e-12)
    assert (np.abs(out) <= A_ + 1e-12).all() and S.shape == (3, 1)


def test_the_short_way_declines_what_it_does_not_know(L):
    """_fast answers False, and launches nothing, for anything but contiguous tensors of the current
    device with the call's types; the caller then goes through the checks that have messages."""
    fast = _lib.fast()
    x = torch.zeros(2, 3, 4, dtype=torch.float16)
    arity = dict(write=9, bounds=7, decode=11, splitk=14, prefill=13, select=13, sparse=11)
    for name, n in arity.items():
        f = getattr(fast, name)
        assert f() is False and f(*[None] * n) is False and f(*[x] * n) is False
        assert f(*[x] * (n - 2), 0, 0) is False                 # host tensors
        assert f(*[x] * (n - 2), -1, 0) is False and f(*[x] * (n - 2), 0, 1 << 70) is False
        assert f(*[object()] * (n - 2), 1 << 70, 0) is False    # numbers past 64 bits
    with pytest.raises((TypeError, ValueError)):
        fast.bind(1, 2)
    with pytest.raises(ValueError):
        fast.bind(*[0] * 7)


def test_tables_leave_room_for_rounding_up(L):
    """A capacity within 1024 tokens of 2^31 is refused: contexts are rounded up in 32 bits."""
    M = (2 ** 31 - 1) // 16
    most = (2 ** 31 - 1 - 1024) // 16
    ws = 2 * 2 * (M + 3) * 4
    for name, d, key in (("pa_decode_fp8_block", dict(DECODE, stream=None), "M"), ("pa_prefill_fp8_block", PREFILL, "M"),
                         ("pa_select_blocks", dict(SELECT, wsb=ws), "M"), ("pa_decode_sparse", SPARSE, "K")):
        for m in (M, most + 1):
            assert call(L, name, d, **{key: m}) == UNSUPPORTED and "2^31 - 1025" in _lib.last_error()
        assert call(L, name, d, S=0, **{key: most}) == OK
    split = dict(DECODE, ps=512, P=M // 32 + 1, ws=A, wsb=2 ** 62, stream=None)
    assert call(L, "pa_decode_splitk_fp8_block", split, M=M) == UNSUPPORTED
