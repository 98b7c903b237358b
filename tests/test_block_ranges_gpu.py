"""GPU parity of the block-scaled attention at the ends of its ranges: queries, keys and scales of
zero and of any size, value scales that differ within a context, one key far ahead of many."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_cases import HALF_STEP, Batch, assert_close
from oracle import block_oracle as bo
from block_ranges import Ranges, mixed_scales, one_ahead
from paged_kv_cache_173_gb300 import api
from test_block_scaled_gpu import run_decode, run_prefill

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


# ------------------------------------------------------------------ queries, keys and scales of zero and of any size
def _small(kind, dtype, dim):
    b = Batch([300, 131, 20], 8, 2, dim, 16, dtype, 41, new=[140, 131, 20])
    if kind == "zero rows":  # beside keys below 1e-4
        b.q[::3] = 0
        b.q[200:, 1] = 0
        b.ks = b.ks * 2.0 ** -20
    elif kind == "zero rows, zero keys":
        b.q[:] = 0
        b.kc[:] = 0
        b.ks[:] = 2.0 ** -64  # as the writer leaves a block of zeros
    elif kind == "zero scales":
        b.q[::2] = b.q[::2] * 2.0 ** -14
        b.ks[:] = 0.0
    elif kind == "some zero scales":
        b.q[1::2] = b.q[1::2] * 2.0 ** -14
        b.ks[b.tables[:, 0].long()] = 0.0
        b.ks[b.tables[0, 3].long(), 1] = 0.0
    return b


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["zero rows", "zero rows, zero keys", "zero scales", "some zero scales"])
def test_prefill_of_zero_queries_keys_and_scales(kind, dtype, dim):
    b = _small(kind, dtype, dim)
    assert_close(run_prefill(b), *b.prefill_reference())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -100, 2.0 ** -20, 2.0 ** 60])
def test_prefill_bfloat16_queries_of_any_size(size, dim):
    b = Batch([300, 40], 8, 2, dim, 16, torch.bfloat16, 42, new=[150, 40])
    b.q = (b.q.float() * size).to(torch.bfloat16)
    usual = b.scale
    for scale in (usual / size, usual * min(1.0, 1.0 / size)):  # scores of the usual size, or near 0 for small queries
        b.scale = float(np.float32(scale))
        assert_close(run_prefill(b), *b.prefill_reference())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.125, -1e-45])
def test_softmax_scales_of_either_sign(scale, dtype):
    b = Batch([300, 131, 20], 8, 2, 64, 16, dtype, 43, new=[140, 131, 20])
    b.scale = scale
    assert_close(run_prefill(b), *b.prefill_reference())
    b.q = b.q[(b.starts[1:] - 1).long()]
    ref, tol = b.reference()
    assert_close(run_decode(b), ref, tol)
    assert_close(run_decode(b, 64), ref, tol)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_prefill_ids_outside_the_pool_in_the_first_blocks(dtype, dim):
    """The first table entries of sequences of several blocks of keys name no block: NaN in every
    call and every row that reads them, and the other rows keep their bits."""
    b = Batch([700, 400, 300, 513, 40], 8, 2, dim, 16, dtype, 44, new=[300, 400, 3, 200, 40])
    want = run_prefill(b)
    assert torch.isfinite(want).all()
    r = b.starts.tolist()
    b.tables[0, 0], b.tables[1, 0], b.tables[3, 5] = b.N, -1, 2 ** 31 - 1
    b.tables[4, 0] = -(2 ** 31)
    for _ in range(40):
        o = run_prefill(b)
        for s in range(5):
            rows = o[r[s]:r[s + 1]]
            assert torch.equal(rows, want[r[s]:r[s + 1]]) if s == 2 else torch.isnan(rows[-1]).all()
            if s != 2:  # the rows whose causal range holds the entry
                sees = max(0, (80 if s == 3 else 0) - (b.lens_list[s] - b.new[s]))
                assert torch.isnan(rows[sees:]).all()


# ------------------------------------------------------------------ weights far below the largest
AHEAD = [  # keys, nats that one is ahead of the others, the largest element of its value, its place
    (131072, 12.1, 448.0, 0), (65536, 10.7, 1792.0, 40000), (16384, 10.7, 1792.0, 5), (16384, 10.1, 3584.0, 16383),
    (4096, 9.0, 60000.0, 2048),
]


def run_sparse(b):
    """The decode of every sequence over tables per KV head that name all of its blocks."""
    q, kc, vc, ks, vs, bt, cl = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens")
    out = torch.full_like(q, float("nan"))
    api.pa_decode_sparse(out, q, kc, vc, bt[:, None].expand(-1, b.Hk, -1).contiguous(),
                         cl[:, None].expand(-1, b.Hk).contiguous(), b.scale, ks, vs)
    torch.cuda.synchronize()
    return out


def check_decodes(b):
    ref, tol = b.reference()
    for got in (run_decode(b), run_decode(b, 64 if b.M <= 1024 else 512), run_decode(b, 4096), run_sparse(b)):
        assert_close(got, ref, tol)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,gap,outlier,at", AHEAD)
def test_decode_of_one_key_ahead_of_many(n, gap, outlier, at, dtype):
    check_decodes(one_ahead(n, gap, outlier, at, dtype))


@pytest.mark.parametrize("heads,dim", [(16, 64), (16, 128), (4, 128), (4, 256)])
def test_decode_of_one_key_ahead_of_many_in_every_shape(heads, dim):
    check_decodes(one_ahead(16384, 10.7, 1792.0, 9000, torch.bfloat16, heads=heads, dim=dim))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", ["two", "all"])
def test_decode_of_blocks_of_very_different_value_scales(kind, dim):
    check_decodes(mixed_scales(kind, dim))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,gap,outlier,at", AHEAD)
def test_prefill_of_one_key_ahead_of_many(n, gap, outlier, at, dtype):
    b = one_ahead(n, gap, outlier, at, dtype, new=[9]).prefill()
    assert_close(run_prefill(b), *b.prefill_reference())


@pytest.mark.parametrize("heads,dim", [(16, 64), (16, 128), (1, 128)])
def test_prefill_of_one_key_ahead_of_many_in_every_shape(heads, dim):
    b = one_ahead(16384, 10.7, 1792.0, 9000, torch.bfloat16, heads=heads, dim=dim, new=[150 // heads + 2]).prefill()
    assert_close(run_prefill(b), *b.prefill_reference())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind", ["two", "wide"])
def test_prefill_of_blocks_of_very_different_value_scales(kind, dim):
    b = mixed_scales(kind, dim, new=[130, 40, 20]).prefill()
    assert_close(run_prefill(b), *b.prefill_reference())


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_of_value_scales_far_above_the_first_ones(dim):
    """2^46 times the largest of the first 128 keys is taken, 2^47 gives NaN to the rows that read it; values
    of zero in the first 128 keys stand for scales around 2^-8."""
    b = Ranges([600, 400, 300], 4, 2, dim, 16, torch.bfloat16, 55, new=[40, 30, 20]).prefill()
    for s in range(3):
        b.vs[b.tables[s, : -(-b.lens_list[s] // 16)].long()] = 2.0 ** -9
        b.vs[b.tables[s, 12].long(), 1] = 2.0 ** 37
    b.vs[b.tables[1, :8].long()] = 2.0 ** -64
    b.vs[b.tables[1, 12].long(), 1] = 2.0 ** 38
    b.vc[b.tables[1, :8].long()] = 0
    ref = b.prefill_reference()
    assert_close(run_prefill(b), *ref)
    b.vs[b.tables[0, 12].long(), 1] = 2.0 ** 38
    b.vs[b.tables[1, 12].long(), 1] = 2.0 ** 39
    got = run_prefill(b)
    assert torch.isnan(got[:70, 2:]).all()
    assert_close(got[:70, :2], ref[0][:70, :2], ref[1][:70, :2])
    assert_close(got[70:], ref[0][70:], ref[1][70:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_prefill_of_many_pairs_with_value_scales_of_their_own(dtype):
    """More (sequence, KV head, pair of tiles) than the GPU has SMs, each sequence and head with values
    of a size of its own: a CTA takes several, whose largest scales differ."""
    g = np.random.default_rng(53)
    lens = [int(x) for x in g.integers(100, 2600, 24)]
    new = [min(n, int(x)) for n, x in zip(lens, g.integers(1, 24, 24))]
    b = Ranges(lens, 32, 16, 64, 16, dtype, 54, new=new).prefill()
    for s, n in enumerate(lens):
        size = torch.exp2(torch.randint(-9, 4 if dtype == torch.float16 else 40, (1, 16), generator=torch.Generator().manual_seed(s)).float())
        b.vs[b.tables[s, :-(-n // 16)].long()] *= size
    assert_close(run_prefill(b), *b.prefill_reference())


# ------------------------------------------------------------------ scores of any size
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 23, 2.0 ** 24, 1.3 * 2.0 ** 24, 2.0 ** 25, 1.6 * 2.0 ** 25])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_whose_rounding_is_large(size, sign, dtype):
    """The best keys score +-`size` (in units of log 2), all others `size` or half of it less: the output is
    the mean of the best keys' values, whatever a score's last place is worth."""
    b = Ranges([300, 200], 4, 2, 64, 16, dtype, 56, new=[40, 130])
    best = [[3, 200, 255], [0, 1, 66]]
    b.keys16 = torch.zeros_like(b.keys16).float()
    b.keys16[..., 1] = 224.0 if sign > 0 else 448.0
    for s in range(2):
        for p in best[s]:
            b.keys16[int(b.tables[s, p // 16]), p % 16, :, 1] = 448.0 if sign > 0 else 224.0
    b.recode()
    b.q = torch.zeros_like(b.q)
    b.q[..., 1] = sign
    b.scale = size / (448.0 if sign > 0 else 224.0) / 1.4426950408889634
    want, tol = np.zeros((2, 4, 64)), np.zeros((2, 4, 64))
    for s in range(2):
        for h in range(4):
            rows = bo.rows(b.vc.numpy(), b.vs.numpy(), b.tables[s].numpy(), b.lens_list[s], h // 2)[best[s]]
            want[s, h] = rows.mean(0)
            tol[s, h] = 2.0 ** -11 * np.abs(rows).mean(0) + HALF_STEP[dtype] * np.abs(want[s, h]) + 2.0 ** -20 * np.abs(rows).max()
    assert_close(run_prefill(b)[[39, 169]], want, tol)
    b.q = b.q[:2]
    for got in (run_decode(b), run_decode(b, 64)):
        assert_close(got, want, tol)


# ------------------------------------------------------------------ bounds of the largest keys
@pytest.mark.parametrize("dtype,top,exponent", [(torch.float16, 65504.0, 10), (torch.bfloat16, 3.3895313892515355e38, 122)])
def test_bounds_of_the_largest_keys(dtype, top, exponent):
    """A block whose bounds hold the largest elements of the type, then smaller ones."""
    codes, exps = np.zeros((2, 1, 2, 64), np.int8), np.full((2, 1), -100, np.int32)
    dev = torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda()
    for slots, size in (([16, 17], 1.0), ([18], 2.0 ** -8), ([19, 20, 21], 2.0 ** -3)):
        key = (torch.linspace(-1.0, 1.0, 64).repeat(len(slots), 1, 1) * size * top).to(dtype)
        codes, exps = bo.bounds(key.double().numpy(), codes, exps, np.array(slots), 16)
        api.pa_update_key_bounds(key.cuda(), *dev, torch.tensor(slots).cuda(), 16)
        torch.cuda.synchronize()
        assert exps[1, 0] == exponent
        assert np.array_equal(dev[0].cpu().numpy(), codes) and np.array_equal(dev[1].cpu().numpy(), exps)
