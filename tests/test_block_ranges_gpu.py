"""GPU parity of the block-scaled attention at the ends of its ranges: queries, keys and scales of
zero and of any size."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_cases import Batch, assert_close
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
