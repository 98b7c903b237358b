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
