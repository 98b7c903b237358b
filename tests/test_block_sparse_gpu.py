"""GPU parity of the block-sparse decode: key bounds, block selection, attention
over the selected blocks, and the steps of a generation that uses them together.

Bounds and selections are whole numbers and must equal the oracle's; attention
is held to the tolerance derived in block_cases.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_cases import Batch, assert_close, to_np
from oracle import block_oracle as bo
from paged_kv_cache_173_gb300 import api

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


class Bounds:
    def __init__(self, N, Hk, d, seed):
        g = torch.Generator().manual_seed(seed)
        self.codes = torch.randint(-127, 128, (N, Hk, 2, d), generator=g, dtype=torch.int32).to(torch.int8)
        self.exps = torch.randint(-9, 3, (N, Hk), generator=g, dtype=torch.int32)

    def check(self, key, slots, block):
        want = bo.bounds(to_np(key), self.codes.numpy(), self.exps.numpy(), slots.numpy(), block)
        codes, exps = self.codes.cuda(), self.exps.cuda()
        api.pa_update_key_bounds(key.cuda(), codes, exps, slots.cuda(), block)
        torch.cuda.synchronize()
        self.codes, self.exps = codes.cpu(), exps.cpu()
        assert np.array_equal(self.exps.numpy(), want[1])
        assert np.array_equal(self.codes.numpy(), want[0])


def keys(T, Hk, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, Hk, d), generator=g) * torch.exp(torch.randn((T, Hk, 1), generator=g)) * size).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Hk,d", [(16, 8, 128), (32, 3, 64), (64, 2, 256), (128, 1, 128), (256, 2, 64)])
def test_bounds_of_prompts_chunks_and_single_tokens(B, Hk, d, dtype):
    p = Bounds(40, Hk, d, seed=B + d)
    blocks = torch.randperm(40, generator=torch.Generator().manual_seed(1))
    slot = lambda pos: int(blocks[pos // B]) * B + pos % B  # noqa: E731
    n1, n2 = 2 * B + 5, B // 2 + 3
    for step, (lo, hi) in enumerate([(0, n1), (n1, n1 + n2), (n1 + n2, n1 + n2 + 1), (n1 + n2 + 1, n1 + n2 + 2)]):
        slots = torch.tensor([slot(x) for x in range(lo, hi)], dtype=torch.int64)
        p.check(keys(hi - lo, Hk, d, dtype, 10 + step, 3.0 ** step), slots, B)


def test_bounds_do_not_depend_on_the_calls():
    x = keys(48, 2, 64, torch.bfloat16, 3)
    slots = torch.arange(16, 64)
    ends = []
    for cuts in ([0, 48], [0, 1, 2, 20, 33, 48], list(range(49))):
        p = Bounds(5, 2, 64, seed=4)
        for a, b in zip(cuts, cuts[1:]):
            p.check(x[a:b].contiguous(), slots[a:b], 16)
        ends.append((p.codes, p.exps))
    for codes, exps in ends[1:]:
        assert torch.equal(codes[1:4], ends[0][0][1:4]) and torch.equal(exps, ends[0][1])


def test_bounds_hold_the_keys_and_skip_padding():
    p = Bounds(9, 4, 128, seed=5)
    slots = torch.tensor([32, 33, 34, -1, 100, 9 * 16, 7])
    x = keys(7, 4, 128, torch.float16, 6)
    x[4, 0, 3] = float("inf")
    x[4, 1, 2] = float("nan")
    x[6] = 0
    p.check(x, slots, 16)
    lo = p.codes[2, :, 0].double() * torch.exp2(p.exps[2].double())[:, None]
    hi = p.codes[2, :, 1].double() * torch.exp2(p.exps[2].double())[:, None]
    assert (lo <= x[:3].double().amin(0)).all() and (hi >= x[:3].double().amax(0)).all()


# ------------------------------------------------------------------ selection
def make_bounds(b):
    """Bounds of a batch's 16-bit keys, whole blocks (unread slots count as zeros)."""
    x = torch.nan_to_num(b.keys16.float(), nan=0.0).to(b.dtype).reshape(-1, b.Hk, b.d)
    codes, exps = bo.bounds(to_np(x), np.zeros((b.N, b.Hk, 2, b.d), np.int8), np.zeros((b.N, b.Hk), np.int32),
                            np.arange(b.N * b.B), b.B)
    return torch.from_numpy(codes), torch.from_numpy(exps)


def run_select(b, codes, exps, keep, first, last):
    S = len(b.lens_list)
    tables = torch.full((S, b.Hk, keep), 77, dtype=torch.int32, device="cuda")
    lens = torch.full((S, b.Hk), 77, dtype=torch.int32, device="cuda")
    ws = api.alloc_select_workspace(S, b.Hk, b.M, "cuda")
    ws.fill_(float("nan"))
    api.pa_select_blocks(tables, lens, b.q.cuda(), codes.cuda(), exps.cuda(), b.tables.cuda(), b.lens.cuda(), b.B, first,
                         last, ws)
    torch.cuda.synchronize()
    return tables, lens


def check_select(b, codes, exps, keep, first, last):
    want = bo.select(to_np(b.q), codes.numpy(), exps.numpy(), b.tables.numpy(), b.lens.numpy(), b.B, keep, first, last)
    tables, lens = run_select(b, codes, exps, keep, first, last)
    assert np.array_equal(lens.cpu().numpy(), want[1])
    assert np.array_equal(tables.cpu().numpy(), want[0])
    return tables, lens


SELECT = {
    "gqa4": (dict(lens=[1, 130, 777, 2048, 15, 1031], heads=32, kv_heads=8, dim=128, block=16), 12, 1, 2),
    "gqa8-b32": (dict(lens=[3001, 64, 0, 512], heads=64, kv_heads=8, dim=128, block=32), 9, 0, 1),
    "mha-d64-b64": (dict(lens=[5, 64, 65, 1700], heads=6, kv_heads=6, dim=64, block=64), 5, 2, 2),
    "gqa16": (dict(lens=[900, 513, 1], heads=32, kv_heads=2, dim=128, block=16), 20, 4, 4),
    "gqa5-d64": (dict(lens=[333, 500], heads=15, kv_heads=3, dim=64, block=16), 3, 1, 2),
    "gqa8-d256": (dict(lens=[17, 1000, 2500], heads=16, kv_heads=2, dim=256, block=16), 31, 1, 1),
    "b256": (dict(lens=[2555, 256, 4000, 1], heads=8, kv_heads=4, dim=64, block=256), 4, 0, 4),
    "long": (dict(lens=[40000, 17000], heads=2, kv_heads=1, dim=64, block=16), 200, 1, 1),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", list(SELECT))
def test_selection_and_sparse_decode_match_oracle(name, dtype):
    kw, keep, first, last = SELECT[name]
    b = Batch(dtype=dtype, seed=31, **kw).poison()
    codes, exps = make_bounds(b)
    tables, lens = check_select(b, codes, exps, keep, first, last)
    nt, nl = tables.cpu().numpy(), lens.cpu().numpy()
    q, kc, vc, ks, vs, k16, v16 = b.dev("q", "kc", "vc", "ks", "vs", "keys16", "values16")
    out = torch.full_like(q, float("nan"))
    api.pa_decode_sparse(out, q, kc, vc, tables, lens, b.scale, ks, vs)
    ref, tol = b.reference(True, nt, nl)
    assert_close(out, ref, tol)
    out = torch.full_like(q, float("nan"))
    api.pa_decode_sparse(out, q, k16, v16, tables, lens, b.scale)
    ref, tol = b.reference(False, nt, nl)
    assert_close(out, ref, tol)


def test_selection_ties_go_to_the_earlier_block():
    b = Batch([16 * 40], 4, 2, 64, 16, torch.float16, 32)
    codes, exps = make_bounds(b)
    codes[:] = codes[0].clone()  # every block the same
    exps[:] = exps[0].clone()
    tables, _ = check_select(b, codes, exps, 10, 1, 2)
    ids = b.tables[0].tolist()
    assert tables[0, 0].tolist() == ids[:8] + ids[38:40]
    two = b.tables[0, 20:23].long()
    exps[two] += 1  # scores double: positive ones win, negative ones lose
    check_select(b, codes, exps, 10, 1, 2)


def test_selection_of_extreme_exponents_and_queries():
    b = Batch([16 * 64, 16 * 64], 8, 2, 64, 16, torch.bfloat16, 33)
    codes, exps = make_bounds(b)
    g = torch.Generator().manual_seed(1)
    exps[:] = torch.randint(-100, 122, exps.shape, generator=g, dtype=torch.int32)
    b.q[0, 0] = 0
    b.q[0, 1] = (b.q[0, 1].float() * 2.0 ** 100).to(torch.bfloat16)
    b.q[0, 2] = (b.q[0, 2].float() * 2.0 ** -100).to(torch.bfloat16)
    b.q[1, 1, 3] = float("inf")
    b.q[1, 2, 3] = float("nan")
    b.q[1, 5, :] = -float("inf")
    check_select(b, codes, exps, 10, 1, 2)
    codes[:] = 127  # the largest sums
    b.q[:] = 255.0
    check_select(b, codes, exps, 10, 0, 1)


def test_selection_device_value_outcomes():
    b = Batch([300, 513, 100, 400], 8, 2, 64, 16, torch.float16, 34)
    codes, exps = make_bounds(b)
    b.lens[0] = 0
    b.lens[1] = b.M * b.B + 1
    b.lens[2] = -3
    b.tables[3, 7] = b.N + 5
    tables, lens = check_select(b, codes, exps, 6, 1, 1)
    assert (lens[1] == -1).all() and (lens[2] == -1).all() and (tables[:3] == -1).all()
    assert (tables[3] == b.N + 5).any(-1).all()
    q, kc, vc, ks, vs = b.dev("q", "kc", "vc", "ks", "vs")
    out = torch.zeros_like(q)
    api.pa_decode_sparse(out, q, kc, vc, tables, lens, b.scale, ks, vs)
    o = to_np(out)
    assert (o[0] == 0).all() and np.isnan(o[1]).all() and np.isnan(o[2]).all() and np.isnan(o[3]).all()


def test_keeping_every_block_is_dense_decode():
    b = Batch([300, 513, 20], 8, 2, 128, 16, torch.float16, 35).poison()
    codes, exps = make_bounds(b)
    tables, lens = check_select(b, codes, exps, b.M + 3, 1, 1)
    q, kc, vc, ks, vs = b.dev("q", "kc", "vc", "ks", "vs")
    out = torch.zeros_like(q)
    api.pa_decode_sparse(out, q, kc, vc, tables, lens, b.scale, ks, vs)
    ref, tol = b.reference()
    assert_close(out, ref, tol)


# ------------------------------------------------------------------ a generation
@pytest.mark.parametrize("dtype", DTYPES)
def test_generation_prompt_then_sparse_steps(dtype):
    """Prompts are written and prefilled, then tokens are appended one by one: each step updates
    the pools and the bounds, selects and attends.  Everything is checked against the oracle."""
    B, Hk, H, d, N, keep, first, last = 16, 2, 8, 64, 64, 6, 1, 2
    g = torch.Generator().manual_seed(41)
    lens = [150, 47]
    M = 14
    tables = torch.randperm(N, generator=g)[: 2 * M].view(2, M).int()
    slot = lambda s, pos: int(tables[s, pos // B]) * B + pos % B  # noqa: E731
    b = Batch(lens, H, Hk, d, B, dtype, 42, new=lens)
    b.N, b.M, b.tables = N, M, tables
    b.kc, b.vc = torch.full((N, B, Hk, d), 0x7F, dtype=torch.uint8), torch.full((N, B, Hk, d), 0x7F, dtype=torch.uint8)
    b.ks, b.vs = torch.full((N, Hk), float("nan")), torch.full((N, Hk), float("nan"))
    codes, exps = torch.zeros((N, Hk, 2, d), dtype=torch.int8), torch.zeros((N, Hk), dtype=torch.int32)
    kc, vc, ks, vs, gcodes, gexps, gt = [x.cuda() for x in (b.kc, b.vc, b.ks, b.vs, codes, exps, tables)]

    def store(key, value, slots):
        api.pa_reshape_and_cache_fp8_block(key.cuda(), value.cuda(), kc, vc, ks, vs, slots.cuda())
        api.pa_update_key_bounds(key.cuda(), gcodes, gexps, slots.cuda(), B)
        torch.cuda.synchronize()
        k2, s2 = bo.write(to_np(key), b.kc.numpy(), b.ks.numpy(), slots.numpy())
        v2, t2 = bo.write(to_np(value), b.vc.numpy(), b.vs.numpy(), slots.numpy())
        b.kc, b.ks, b.vc, b.vs = [torch.from_numpy(x) for x in (k2, s2, v2, t2)]
        for mine, theirs in ((kc, k2), (vc, v2), (ks, s2), (vs, t2)):
            assert np.array_equal(mine.cpu().numpy(), theirs, equal_nan=True)

    slots = torch.tensor([slot(s, p) for s in range(2) for p in range(lens[s])])
    store(keys(sum(lens), Hk, d, dtype, 1), keys(sum(lens), Hk, d, dtype, 2), slots)
    out = torch.empty_like(b.q).cuda()
    api.pa_prefill_fp8_block(out, b.q.cuda(), kc, vc, ks, vs, gt, b.lens.cuda(), b.starts.cuda(), max(lens), b.scale)
    ref, tol = b.prefill_reference()
    assert_close(out, ref, tol)
    for step in range(20):
        lens = [n + 1 for n in lens]
        b.lens_list, b.lens = lens, torch.tensor(lens, dtype=torch.int32)
        slots = torch.tensor([slot(s, lens[s] - 1) for s in range(2)])
        store(keys(2, Hk, d, dtype, 100 + step, 1.1 ** step), keys(2, Hk, d, dtype, 200 + step), slots)
        b.q = torch.randn((2, H, d), generator=g).to(dtype)
        want = bo.select(to_np(b.q), gcodes.cpu().numpy(), gexps.cpu().numpy(), tables.numpy(), b.lens.numpy(), B, keep,
                         first, last)
        st, sl = run_select(b, gcodes.cpu(), gexps.cpu(), keep, first, last)
        assert np.array_equal(st.cpu().numpy(), want[0]) and np.array_equal(sl.cpu().numpy(), want[1])
        out = torch.empty_like(b.q).cuda()
        api.pa_decode_sparse(out, b.q.cuda(), kc, vc, st, sl, b.scale, ks, vs)
        ref, tol = b.reference(True, want[0], want[1])
        assert_close(out, ref, tol)
        api.pa_decode_fp8_block(out, b.q.cuda(), kc, vc, ks, vs, gt, b.lens.cuda(), b.scale)
        ref, tol = b.reference()
        assert_close(out, ref, tol)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("keep,first,last", [(130, 1, 2), (9000, 0, 1), (8192, 4000, 4192), (3, 1, 1)])
def test_selection_in_rows_of_many_blocks(keep, first, last, ties):
    """Rows of up to 20000 blocks, more than a CTA holds at once, on both sides of that number; with
    ties, a handful of different blocks, so that equal scores reach over all of it."""
    S, Hk, H, d, B, M = 4, 2, 6, 64, 16, 20000
    g = torch.Generator().manual_seed(41)
    N = 5 if ties else 30000
    codes = torch.randint(-127, 128, (N, Hk, 2, d), generator=g, dtype=torch.int32)
    codes = torch.stack([codes.amin(2), codes.amax(2)], 2).to(torch.int8)
    exps = torch.randint(-9, 3, (N, Hk), generator=g, dtype=torch.int32)
    tables = torch.randint(0, N, (S, M), generator=g, dtype=torch.int32)
    lens = torch.tensor([8192 * B, 8193 * B - 3, M * B - 5, 16384 * B + 1], dtype=torch.int32)
    q = torch.randn((S, H, d), generator=g).to(torch.float16)
    want = bo.select(to_np(q), codes.numpy(), exps.numpy(), tables.numpy(), lens.numpy(), B, keep, first, last)
    st = torch.full((S, Hk, keep), 77, dtype=torch.int32, device="cuda")
    sl = torch.full((S, Hk), 77, dtype=torch.int32, device="cuda")
    ws = api.alloc_select_workspace(S, Hk, M, "cuda")
    ws.fill_(float("nan"))
    api.pa_select_blocks(st, sl, q.cuda(), codes.cuda(), exps.cuda(), tables.cuda(), lens.cuda(), B, first, last, ws)
    torch.cuda.synchronize()
    assert np.array_equal(sl.cpu().numpy(), want[1])
    assert np.array_equal(st.cpu().numpy(), want[0])
