"""GPU parity of the block-scaled E4M3 cache: write, decode, split-K decode, prefill.

The write is integer work (a code per element, an exponent per block) and
must match the float64 oracle bit for bit; attention is held to the tolerance
derived in block_cases.
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


# ------------------------------------------------------------------ write
class Pools:
    def __init__(self, N, B, Hk, d, seed):
        g = torch.Generator().manual_seed(seed)
        self.kc = torch.randint(0, 256, (N, B, Hk, d), generator=g, dtype=torch.int32).to(torch.uint8)
        self.vc = torch.randint(0, 256, (N, B, Hk, d), generator=g, dtype=torch.int32).to(torch.uint8)
        self.ks = torch.exp2(torch.randint(-12, 0, (N, Hk), generator=g).float())
        self.vs = torch.exp2(torch.randint(-12, 0, (N, Hk), generator=g).float())

    def check_write(self, key, value, slots):
        want = [bo.write(to_np(new), c.numpy(), s.numpy(), slots.numpy())
                for new, c, s in ((key, self.kc, self.ks), (value, self.vc, self.vs))]
        dev = [t.cuda() for t in (self.kc, self.vc, self.ks, self.vs)]
        api.pa_reshape_and_cache_fp8_block(key.cuda(), value.cuda(), *dev, slots.cuda())
        torch.cuda.synchronize()
        for (codes, scales), c, s in zip(want, dev[:2], dev[2:]):
            assert np.array_equal(s.cpu().numpy(), scales, equal_nan=True)
            got = c.cpu().numpy()
            nan = (codes & 127) == 127  # a NaN code's sign is not kept
            assert np.array_equal(got[~nan], codes[~nan])
            assert ((got[nan] & 127) == 127).all()
        self.kc, self.vc, self.ks, self.vs = [t.cpu() for t in dev]


def tokens(T, Hk, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hk, d), generator=g) * torch.exp(torch.randn((T, Hk, 1), generator=g)) * size
    return x.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Hk,d", [(16, 8, 128), (32, 3, 64), (64, 2, 256), (128, 1, 128), (256, 2, 64)])
def test_write_of_prompts_chunks_and_single_tokens(B, Hk, d, dtype):
    p = Pools(40, B, Hk, d, seed=B + d)
    blocks = torch.randperm(40, generator=torch.Generator().manual_seed(1))
    # a sequence in blocks[0:4]: a prompt that ends inside a block, a chunk that goes on, then tokens one by one
    slot = lambda pos: int(blocks[pos // B]) * B + pos % B  # noqa: E731
    n1, n2 = 2 * B + 5, B // 2 + 3
    step = 0
    for lo, hi in [(0, n1), (n1, n1 + n2), (n1 + n2, n1 + n2 + 1), (n1 + n2 + 1, n1 + n2 + 2)]:
        slots = torch.tensor([slot(x) for x in range(lo, hi)], dtype=torch.int64)
        k = tokens(hi - lo, Hk, d, dtype, seed=10 + step, size=3.0 ** step)  # each larger: scales grow
        p.check_write(k, tokens(hi - lo, Hk, d, dtype, seed=20 + step, size=0.01 * 5.0 ** step), slots)
        step += 1


@pytest.mark.parametrize("dtype", DTYPES)
def test_write_of_one_token_each_to_many_blocks(dtype):
    p = Pools(70, 16, 8, 128, seed=5)
    g = torch.Generator().manual_seed(2)
    slots = torch.randperm(70, generator=g)[:61] * 16 + torch.randint(0, 16, (61,), generator=g)
    slots[7] = -1
    slots[20] = -5
    slots[33] = 70 * 16 + 3  # outside the pool
    for size in (1e-3, 1.0, 1e3):
        p.check_write(tokens(61, 8, 128, dtype, 3, size), tokens(61, 8, 128, dtype, 4, size), slots)


def test_write_of_special_values():
    p = Pools(6, 16, 2, 64, seed=6)
    key = torch.zeros((20, 2, 64), dtype=torch.float16)
    key[0, 0, 0] = float("inf")
    key[0, 0, 1] = -float("inf")
    key[0, 0, 2] = float("nan")
    key[1, 0] = 448.0
    key[1, 1] = 449.0  # just past a power-of-two scale's range
    key[2, 1, 5] = 65504.0
    key[3] = 2.0 ** -24
    value = torch.zeros_like(key)  # a block of zeros: the smallest scale
    value[5, 1, 3] = -2.0 ** -24
    p.check_write(key, value, torch.arange(16, 36))
    p.ks[3] = torch.tensor([0.0, float("nan")])  # no scale: read as none
    p.vs[3] = torch.tensor([-1.0, float("inf")])
    p.check_write(key[3:4] + 1, value[3:4] + 2, torch.tensor([3 * 16 + 7]))
    p.ks[4] = torch.tensor([0.3, 0.011])  # scales that are no powers of two
    p.check_write(tokens(1, 2, 64, torch.float16, 8), tokens(1, 2, 64, torch.float16, 9, 100.0), torch.tensor([4 * 16 + 2]))


def test_write_is_repeatable_and_leaves_other_blocks_alone():
    p = Pools(30, 32, 4, 128, seed=7)
    slots = torch.tensor([40, 41, 42, 200, 201, 700])
    k, v = tokens(6, 4, 128, torch.bfloat16, 1, 50.0), tokens(6, 4, 128, torch.bfloat16, 2, 50.0)
    p.check_write(k, v, slots)
    before = [t.clone() for t in (p.kc, p.vc, p.ks, p.vs)]
    p.check_write(k, v, slots)
    for a, b in zip(before, (p.kc, p.vc, p.ks, p.vs)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ decode
DECODE = {
    "gqa4": dict(lens=[1, 130, 777, 2048, 15, 1031], heads=32, kv_heads=8, dim=128, block=16),
    "gqa8-b32": dict(lens=[3001, 64, 0], heads=64, kv_heads=8, dim=128, block=32),
    "mha-d64-b64": dict(lens=[5, 64, 65, 700], heads=6, kv_heads=6, dim=64, block=64),
    "gqa16": dict(lens=[300, 513, 1], heads=32, kv_heads=2, dim=128, block=16),
    "gqa16-d64": dict(lens=[16, 17, 1200], heads=16, kv_heads=1, dim=64, block=128),
    "gqa5-d64": dict(lens=[33, 500], heads=15, kv_heads=3, dim=64, block=16),
    "d256": dict(lens=[17, 1000, 2500], heads=16, kv_heads=4, dim=256, block=16),
    "gqa8-d256-b128": dict(lens=[333, 4096], heads=16, kv_heads=2, dim=256, block=128),
    "gqa2-d64-b256": dict(lens=[255, 256, 257, 1], heads=8, kv_heads=4, dim=64, block=256),
    # more (sequence, KV head) pairs than resident CTAs, one of them long: ranked launch, several table windows
    "ranked": dict(lens=[9000] + [40 + 3 * i for i in range(69)], heads=8, kv_heads=8, dim=128, block=16),
    "many": dict(lens=[1 + 7 * (i % 13) for i in range(300)], heads=4, kv_heads=4, dim=64, block=16),
}


def run_decode(b, part=0):
    out = torch.full_like(b.q, float("nan")).cuda()
    q, kc, vc, ks, vs, bt, cl = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens")
    if part:
        P = api.max_num_partitions_for(b.M, b.B, part)
        ws = api.alloc_splitk_workspace(len(b.lens_list), b.H, b.d, P, "cuda")
        ws.fill_(float("nan"))
        api.pa_decode_splitk_fp8_block(out, q, kc, vc, ks, vs, bt, cl, b.scale, part, ws, P)
        api.pa_splitk_reduce(out, ws, cl, b.M, b.B, part, P)
    else:
        api.pa_decode_fp8_block(out, q, kc, vc, ks, vs, bt, cl, b.scale)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", list(DECODE))
def test_decode_matches_oracle(name, dtype):
    b = Batch(dtype=dtype, seed=11, **DECODE[name]).poison()
    ref, tol = b.reference()
    assert_close(run_decode(b), ref, tol)
    for part in (b.B, 4 * b.B, 512):
        assert_close(run_decode(b, part), ref, tol)


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_with_any_scales(dtype):
    # scales that are no powers of two, and blocks whose values differ by e^(+-6)
    b = Batch([700, 1500, 90], 16, 4, 128, 16, dtype, 12, pow2=False, wide=True).poison()
    ref, tol = b.reference()
    assert_close(run_decode(b), ref, tol)
    assert_close(run_decode(b, 256), ref, tol)


def test_decode_bfloat16_queries_of_any_size():
    for size in (2.0 ** -100, 2.0 ** -20, 2.0 ** 60):
        b = Batch([300], 8, 2, 128, 16, torch.bfloat16, 13)
        b.q = (b.q.float() * size).to(torch.bfloat16)
        b.scale = float(np.float32(b.scale / size))
        ref, tol = b.reference()
        assert_close(run_decode(b), ref, tol)


def test_decode_zero_scales_and_zero_queries():
    b = Batch([100, 40], 8, 2, 64, 16, torch.float16, 14)
    b.vs[b.tables[0, 2].long()] = 0.0
    b.ks[b.tables[0, 3].long()] = 0.0
    b.vs[b.tables[1, :3].long()] = 2.0 ** -70  # reads as zero
    b.q[0, 0] = 0
    out = run_decode(b)
    ref, tol = b.reference()
    assert_close(out, ref, tol)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("part", [0, 64])
def test_decode_device_value_outcomes(part):
    b = Batch([300, 513, 100, 80, 90, 200, 64], 32, 2, 128, 16, torch.float16, 15)
    b.lens[0] = 0
    b.lens[2] = b.M * b.B + 1
    b.lens[3] = -1
    b.tables[1, 3] = b.N + 7
    b.ks[b.tables[4, 1].long(), 1] = -1.0
    b.vs[b.tables[5, 0].long(), 0] = float("inf")
    b.kc[b.tables[6, 1].long(), 2, 0, 5] = 0x7F
    o = to_np(run_decode(b, part))
    assert (o[0] == 0).all()
    for s in (1, 2, 3):
        assert np.isnan(o[s]).all()
    assert np.isnan(o[4, 16:]).all() and np.isfinite(o[4, :16]).all()
    assert np.isnan(o[5, :16]).all() and np.isfinite(o[5, 16:]).all()
    assert np.isnan(o[6, :16]).all() and np.isfinite(o[6, 16:]).all()


def test_decode_takes_float8_tensors_and_a_stream():
    b = Batch([77, 300], 8, 2, 64, 16, torch.float16, 16)
    ref, tol = b.reference()
    q, kc, vc, ks, vs, bt, cl = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens")
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    api.pa_decode_fp8_block(out, q, kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs, bt, cl, b.scale,
                            stream=side)
    side.synchronize()
    assert_close(out, ref, tol)


# ------------------------------------------------------------------ prefill
PREFILL = {
    "prompts": dict(lens=[70, 17, 100, 1], new=[70, 17, 100, 1], heads=8, kv_heads=2, dim=128, block=16),
    "chunks": dict(lens=[300, 17, 129, 640], new=[40, 1, 129, 130], heads=8, kv_heads=2, dim=128, block=64),
    "gqa16-d64": dict(lens=[200, 35], new=[150, 3], heads=16, kv_heads=1, dim=64, block=32),
    "mha-d64-b256": dict(lens=[300, 257], new=[300, 1], heads=3, kv_heads=3, dim=64, block=256),
    "mha-b128": dict(lens=[400], new=[260], heads=2, kv_heads=2, dim=128, block=128),
}


def run_prefill(b):
    q, kc, vc, ks, vs, bt, cl, qs = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens", "starts")
    out = torch.full_like(q, float("nan"))
    api.pa_prefill_fp8_block(out, q, kc, vc, ks, vs, bt, cl, qs, max(b.new), b.scale)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", list(PREFILL))
def test_prefill_matches_oracle(name, dtype):
    b = Batch(dtype=dtype, seed=21, **PREFILL[name]).poison()
    ref, tol = b.prefill_reference()
    assert_close(run_prefill(b), ref, tol)


@pytest.mark.parametrize("dtype", DTYPES)
def test_prefill_with_any_scales(dtype):
    b = Batch([300, 150], 8, 2, 128, 16, dtype, 22, pow2=False, wide=True, new=[140, 150]).poison()
    ref, tol = b.prefill_reference()
    assert_close(run_prefill(b), ref, tol)


def test_prefill_device_value_outcomes():
    b = Batch([300, 200, 100, 90, 64], 8, 2, 64, 16, torch.float16, 23, new=[20, 30, 10, 90, 0])
    b.lens[2] = 5            # shorter than its new tokens
    b.tables[0, 3] = b.N     # read by every row of sequence 0
    b.ks[b.tables[1, 1].long(), 0] = float("nan")
    o = to_np(run_prefill(b))
    r = b.starts.tolist()
    assert np.isnan(o[r[0]:r[1]]).all()
    assert np.isnan(o[r[1]:r[2], :4]).all() and np.isfinite(o[r[1]:r[2], 4:]).all()
    assert np.isnan(o[r[2]:r[3]]).all()
    assert np.isfinite(o[r[3]:r[4]]).all()


def test_prefill_rows_behind_the_last_sequence_are_left_alone():
    b = Batch([60, 33], 4, 2, 64, 16, torch.float16, 24, new=[60, 33])
    b.q = torch.cat([b.q, b.q[:7]])
    q, kc, vc, ks, vs, bt, cl, qs = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens", "starts")
    out = torch.full_like(q, 3.0)
    api.pa_prefill_fp8_block(out, q, kc, vc, ks, vs, bt, cl, qs, 60, b.scale)
    torch.cuda.synchronize()
    assert (out[93:] == 3.0).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_prefill_with_more_work_than_the_gpu_holds(dtype):
    """768 (sequence, KV head, pair of tiles): most CTAs compute several, of all lengths, among them
    sequences without new tokens and with a context length that cannot be."""
    g = np.random.default_rng(31)
    lens = [int(x) for x in g.integers(1, 400, 48)]
    new = [min(n, int(x)) for n, x in zip(lens, g.integers(0, 256, 48))]
    new[3], lens[3], new[40], lens[40] = 256, 700, 1, 900
    b = Batch(lens, 16, 4, 64, 16, dtype, 32, new=new).poison()
    ref, tol = b.prefill_reference()
    bad = [i for i in (7, 30) if new[i] > 0]
    b.lens[torch.tensor(bad)] = 0
    o = run_prefill(b)
    r = b.starts.tolist()
    for i in bad:
        assert torch.isnan(o[r[i]:r[i + 1]]).all()
        ref[r[i]:r[i + 1]], o[r[i]:r[i + 1]] = 0, 0
    assert_close(o, ref, tol)
    assert torch.equal(run_prefill(b)[:r[7]], o[:r[7]])  # whichever CTA computes a row, its bits are the same


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_prefill_nan_values_reach_only_the_rows_that_see_them(dtype, dim):
    """A NaN code in a new token's value: the token and those behind it get NaN in that channel of
    that head; the tokens before it, whose weight for it is 0, keep their bits."""
    b = Batch([300, 131, 70], 8, 2, dim, 16, dtype, 33, new=[190, 131, 3])
    at = [(0, 109, 0, 5), (0, 131, 1, 40), (0, 298, 0, 63), (1, 0, 1, 0), (1, 127, 0, dim - 1), (1, 128, 0, 17), (2, 68, 1, 33),
          (0, 20, 0, 9)]
    want = None
    for code in (0, 0x7f, 0xff):
        for s, p, h, c in at:
            b.vc[int(b.tables[s, p // b.B]), p % b.B, h, c] = code
        o = run_prefill(b)
        if want is None:
            want = o
            continue
        exp, r = want.clone(), b.starts.tolist()
        for s, p, h, c in at:
            row = max(r[s], r[s + 1] - b.lens_list[s] + p)  # of the token itself (a cached one: every row)
            exp[row:r[s + 1], 4 * h:4 * h + 4, c] = float("nan")
        assert torch.isnan(exp).any() and torch.equal(torch.isnan(o), torch.isnan(exp))
        assert torch.equal(torch.nan_to_num(o), torch.nan_to_num(exp))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_prefill_of_prompts_beside_single_tokens(dtype, dim):
    """Batches whose sequences bring very different numbers of new tokens: prompts, chunks, single
    tokens, none, and a context length that cannot be."""
    new = [1] * 70
    new[0], new[5], new[33], new[40], new[41], new[64], new[69] = 0, 600, 65, 0, 64, 130, 129
    lens = [n + 37 * (i % 9) for i, n in enumerate(new)]
    b = Batch([max(n, 1) for n in lens], 4, 1, dim, 16, dtype, 34, new=new).poison()
    ref, tol = b.prefill_reference()
    b.lens[64], b.lens[2] = 129, -1
    o = run_prefill(b)
    r = b.starts.tolist()
    for i in (2, 64):
        assert torch.isnan(o[r[i]:r[i + 1]]).all()
        ref[r[i]:r[i + 1]], o[r[i]:r[i + 1]] = 0, 0
    assert_close(o, ref, tol)


def test_prefill_of_single_tokens_in_a_large_batch():
    """1030 sequences, one of them a prompt: more than the list of pairs is searched for."""
    new = [1] * 1030
    new[500] = 300
    b = Batch([max(n, 1 + i % 40) for i, n in enumerate(new)], 4, 4, 64, 16, torch.float16, 35, new=new)
    assert_close(run_prefill(b), *b.prefill_reference())


@pytest.mark.parametrize("exponent", [127, 126, -64])
def test_value_scales_at_both_ends_of_their_range(exponent):
    """Value scales of 2^127 (whose inverse is subnormal) down to 2^-64, codes small enough for the output type."""
    b = Batch([150, 33, 1], 8, 2, 128, 16, torch.bfloat16, 36, new=[40, 33, 1])
    g = torch.Generator().manual_seed(37)
    b.vc = (torch.randint(0, 0x31, b.vc.shape, generator=g) | (torch.randint(0, 2, b.vc.shape, generator=g) << 7)).to(torch.uint8)
    b.vs = torch.full_like(b.vs, 2.0 ** exponent)  # at most 0.5 * 2^exponent
    assert_close(run_prefill(b), *b.prefill_reference())
    q, kc, vc, ks, vs, bt, cl = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens")
    b.q = b.q[(b.starts[1:] - 1).long()]
    q = b.q.cuda()
    out = torch.empty_like(q)
    api.pa_decode_fp8_block(out, q, kc, vc, ks, vs, bt, cl, b.scale)
    torch.cuda.synchronize()
    assert_close(out, *b.reference())
