"""Packed prefill against float64, and the whole run of a request: room for a prompt, its
attention with the cache write, samples forked off it, decode steps, compaction.

Tolerance of an output, from the arithmetic.  With w_i the exact weights (sum 1), A =
sum w_i |v_i| and S the largest sum |q_c k_c| * scale:
  - the weights enter P.V in the values' type: half a step of each, 2^-11 A (fp16) or
    2^-8 A (bf16); they are summed unrounded.  fp16: the largest weight is 2^7 or more, a
    weight below 2^-14 is off by 2^-25: 2^-32 of the largest for each of n, times max |v|;
  - scores, the exponential and the float32 sums as for the block operators:
    2 (d + 4) 2^-24 S A + 2 (2^-22 + (n / 8 + 16) 2^-24) A;
  - the output is rounded once: half a step, and half of fp16's smallest step, 2^-25.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_cases import HALF_STEP, to_np
from oracle import sequence_oracle as so
from paged_kv_cache_173_gb300 import api

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


class Prompts:
    """Prompts in packed rows, drawn on the CPU from a seed, with pools and slots."""

    def __init__(self, lens, H, Hk, d, dtype, seed, fused=False, pad=0, block=16, cache=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hk, self.d, self.dtype, self.B = list(lens), H, Hk, d, dtype, block
        self.rows = sum(lens) + pad
        self.starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.q = (torch.randn((self.rows, H, d), generator=g) * 0.8).to(dtype)
        self.k = (torch.randn((self.rows, Hk, d), generator=g) * torch.exp(0.5 * torch.randn((Hk, d), generator=g))).to(dtype)
        self.v = (torch.randn((self.rows, Hk, d), generator=g) * torch.exp(0.7 * torch.randn((self.rows, Hk, 1), generator=g))).to(dtype)
        self.scale = float(np.float32(d ** -0.5))
        self.max_len = max(lens) if len(lens) else 0
        self.fused, self.cache = fused, cache
        self.N = self.rows // block + 3
        self.slots = torch.randperm(self.N * block, generator=g)[:self.rows]

    def start(self):
        if self.fused:  # parts of the rows of one projection
            qkv = torch.cat([self.q, self.k, self.v], 1).cuda()
            self.dq, self.dk, self.dv = qkv[:, :self.H], qkv[:, self.H:self.H + self.Hk], qkv[:, self.H + self.Hk:]
        else:
            self.dq, self.dk, self.dv = self.q.cuda(), self.k.cuda(), self.v.cuda()
        self.out = torch.full((self.rows, self.H, self.d), 7.0, dtype=self.dtype, device="cuda")
        self.dst = torch.from_numpy(self.starts).cuda()
        self.dsl = self.slots.cuda()
        self.kc, self.vc = (torch.full((self.N, self.B, self.Hk, self.d), x, dtype=self.dtype, device="cuda") for x in (3.0, 5.0))
        return self

    def run(self, stream=None):
        extra = (self.kc, self.vc, self.dsl) if self.cache else ()
        api.pa_prefill_packed(self.out, self.dq, self.dk, self.dv, self.dst, self.max_len, self.scale, *extra, stream=stream)
        return self

    def reference(self):
        """(out, tolerance) of every row, NaN where none is computed.  Keys of -inf weigh nothing, nor do they count
        in the scores' sums (their scores are -inf, without an error)."""
        q, k, v = to_np(self.q), to_np(self.k), to_np(self.v)
        with np.errstate(all="ignore"):
            out, A, S = so.attention(q, k, v, self.starts, self.scale, self.max_len)
            if np.isneginf(k).any():
                S = so.attention(q, np.where(np.isneginf(k), 0, k), v, self.starts, self.scale, self.max_len)[2]
            n, top = max(self.lens, default=1), np.abs(np.where(np.isfinite(v), v, 0)).max(initial=0)
            sums = 2.0 ** -22 + (n / 8 + 16) * 2.0 ** -24
            tiny = n * 2.0 ** -32 * top + 2.0 ** -25 if self.dtype == F16 else 2.0 ** -100
            tol = (HALF_STEP[self.dtype] * (A + np.abs(out)) + A * (2 * (self.d + 4) * 2.0 ** -24 * S[..., None] + 2 * sums) + tiny)
        return out, tol

    def check(self):
        torch.cuda.synchronize()
        got = to_np(self.out)
        want, tol = self.reference()
        done = np.zeros(self.rows, bool)
        for a, n in zip(self.starts, self.lens):
            done[a:a + min(n, self.max_len)] = True
        assert (got[~done] == 7.0).all()
        err = np.abs(got[done] - want[done])
        assert np.isfinite(got[done]).all() and (err <= tol[done]).all(), \
            (np.argwhere(~(err <= tol[done]))[:4].tolist(), float(np.nanmax(err / tol[done])))
        self.check_pools(done)

    def check_pools(self, done):
        if not self.cache:
            return
        for pool, new, empty in ((self.kc, self.k, 3.0), (self.vc, self.v, 5.0)):
            want = torch.full_like(pool, empty).cpu().flatten(0, 1)
            ok = torch.from_numpy(done) & (self.slots >= 0) & (self.slots < self.N * self.B)
            want[self.slots[ok]] = new[ok]
            assert torch.equal(pool.cpu().flatten(0, 1).view(torch.int16), want.view(torch.int16))


HEADS = [(1, 1), (4, 4), (8, 2), (6, 2), (7, 1), (10, 2), (16, 1), (12, 1), (22, 2), (13, 1), (32, 8)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", HEADS)
def test_groups(H, Hk, d, dtype):
    Prompts([37, 1, 130, 2, 300], H, Hk, d, dtype, H + d, fused=H % 2 == 0, pad=3).start().run().check()


@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [63, 64, 65], [127, 128, 129], [255, 256, 257], [511, 1, 513],
                                  [1] * 50, [16] * 40, [0, 5, 0, 0, 9, 0], [700, 3, 3, 650]])
@pytest.mark.parametrize("H,Hk,d,dtype", [(4, 1, 128, F16), (8, 8, 128, BF16), (5, 1, 64, F16), (2, 2, 64, BF16)])
def test_lengths(lens, H, Hk, d, dtype):
    Prompts(lens, H, Hk, d, dtype, sum(lens), fused=True, pad=1).start().run().check()


@pytest.mark.parametrize("H,Hk,d,dtype,n", [(2, 1, 128, F16, 2500), (1, 1, 64, BF16, 2100), (3, 1, 128, BF16, 1900)])
def test_long_prompts(H, Hk, d, dtype, n):
    Prompts([n, 300], H, Hk, d, dtype, n).start().run().check()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_more_items_than_the_gpu_has_processors(dtype):
    rng = np.random.default_rng(1)
    Prompts([int(x) for x in rng.integers(1, 200, 60)], 16, 8, 64, dtype, 2).start().run().check()


@pytest.mark.parametrize("lens", [[900] + [1] * 80, [1] * 300 + [600], [257] * 3 + [2] * 70])
def test_one_long_prompt_among_short_ones(lens):
    Prompts(lens, 8, 2, 128, F16, len(lens)).start().run().check()


@pytest.mark.parametrize("block", [1, 5, 16, 48, 256])
def test_pools_of_any_block_size(block):
    Prompts([40, 200], 4, 2, 64, BF16, block, block=block).start().run().check()


def test_slots_that_write_nothing():
    p = Prompts([90, 30], 4, 2, 128, F16, 3)
    p.slots[::7] = -1
    p.slots[3::11] = p.N * p.B + torch.arange(len(p.slots[3::11])) * 2 ** 33
    p.slots[5] = -2 ** 60
    p.start().run().check()
    p = Prompts([90, 30], 4, 2, 128, F16, 3, cache=False).start().run()
    p.check()
    assert bool((p.kc == 3.0).all())


def test_rows_past_the_largest_length_are_left():
    p = Prompts([90, 30, 200], 4, 2, 64, F16, 4)
    p.max_len = 77
    p.start().run().check()


@pytest.mark.parametrize("scale", [0.0, -0.0, -0.11, 3.0, 1e-30, -1e-30])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scales(scale, dtype):
    p = Prompts([150, 20], 8, 2, 64, dtype, 5)
    p.scale = float(np.float32(scale))
    p.start().run().check()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_peaked_and_flat_weights(dtype):
    p = Prompts([400], 4, 1, 128, dtype, 6)
    p.q *= 8  # scores of some hundred
    p.start().run().check()
    p = Prompts([400], 4, 1, 128, dtype, 7)
    p.q.zero_()
    p.start().run().check()
    p = Prompts([300], 2, 1, 64, dtype, 8)  # the maximum grows from key to key
    p.k[:] = (torch.arange(300)[:, None, None] * 0.2).to(dtype)
    p.q.fill_(1.0)
    p.start().run().check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [0.02, 0.2, 1.0])
@pytest.mark.parametrize("first", [0, 31, 40, 64, 65, 100, 127, 128, 150, 192, 257])
def test_a_maximum_that_grows(first, step, d, dtype):
    """Equal scores up to a key, from there each one larger than the one before; in q's second head falling ones."""
    p = Prompts([400], 2, 1, d, dtype, first)
    p.k[:] = ((torch.arange(400) - first).clamp(min=0)[:, None, None] * step).to(dtype)
    p.q.fill_(1.0)
    p.q[:, 1] = -1.0
    p.start().run().check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 5, 63, 64, 100, 127, 128, 200, 256, 383])
@pytest.mark.parametrize("top", [3.0, 30.0])
def test_one_large_score(top, at, d, dtype):
    """One key far above all others: by less and by more than the offset of the block before allows for."""
    p = Prompts([400], 2, 1, d, dtype, at)
    p.k *= 0.1
    p.q.fill_(1.0)
    p.k[at] = top
    p.start().run().check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("a,b", [(0, 1), (0, 64), (0, 128), (0, 129), (0, 200), (0, 300), (64, 128), (100, 300), (128, 256), (3, 399)])
def test_keys_of_minus_infinity(a, b, d, dtype):
    """Scores of -inf weigh nothing; a row that sees only such keys has no answer."""
    p = Prompts([400], 2, 1, d, dtype, a + b)
    p.q = p.q.abs() + 0.01
    p.k[a:b] = -float("inf")
    p.start().run()
    torch.cuda.synchronize()
    got = to_np(p.out)
    want, tol = p.reference()
    empty = np.isnan(want).any(axis=(1, 2))
    assert empty[:b].all() and not empty[b:].any() if a == 0 else not empty.any()
    assert np.isnan(got[empty]).all()
    err = np.abs(got - want)[~empty]
    assert np.isfinite(got[~empty]).all() and (err <= tol[~empty]).all(), np.argwhere(~(err <= tol[~empty]))[:4].tolist()


@pytest.mark.parametrize("lens", [[1] * 600 + [1100] + [3] * 600, [1] * 3000 + [900], [2] * 1500 + [2600], [40] * 127 + [0] * 130 + [2000],
                                  [1, 200] * 130 + [3000, 2900], list(range(300)), list(range(300, 0, -1)) + [2000]])
@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences_beside_long_ones(lens, d):
    Prompts(lens, 4, 2, d, F16, 30).start().run().check()


def test_a_list_of_sequences_in_no_order_stays_inside():
    rng = np.random.default_rng(31)
    for top in (3000, 100):
        p = Prompts([3000], 4, 2, 64, BF16, 31).start()
        p.dst = torch.from_numpy(rng.integers(-100, top + 100, 201).astype(np.int32)).cuda()
        guard = p.kc.clone()
        p.dsl.fill_(-1)
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(p.kc, guard)


def test_large_and_tiny_values():
    p = Prompts([200], 2, 1, 64, BF16, 9)
    p.v = (p.v.float() * 1e30).to(BF16)
    p.start().run().check()
    p.v = (p.v.float() * 1e-50).to(BF16)
    p.start().run().check()
    p = Prompts([200], 2, 1, 64, F16, 10)
    p.v.fill_(65504.0)
    p.start().run().check()


def finite_elsewhere(p, changed):
    """Run p with and without what `changed` does to its inputs: rows that do not see it are the same bits.
    Returns both outputs."""
    p.start().run()
    clean = p.out.clone()
    changed(p)
    p.start().run()
    torch.cuda.synchronize()
    return clean.float().cpu(), p.out.float().cpu()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 1, 63, 64, 100, 127, 128, 200, 259])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_what_is_not_finite_reaches_the_rows_that_see_it(dtype, bad, at, G):
    lens = [260, 150]

    def value(p):
        p.v[at, 0, 5] = bad

    clean, got = finite_elsewhere(Prompts(lens, 2 * G, 2, 64, dtype, at, pad=2), value)
    assert torch.equal(got[:at], clean[:at]) and torch.equal(got[260:], clean[260:])
    seen = got[at:260, :G]
    assert not torch.isfinite(seen[..., 5]).any()
    others = [c for c in range(64) if c != 5]
    assert torch.equal(seen[..., others], clean[at:260, :G][..., others])
    assert torch.equal(got[at:260, G:], clean[at:260, G:])

    def key(p):
        p.k[at, 0, 5] = bad

    clean, got = finite_elsewhere(Prompts(lens, 2 * G, 2, 64, dtype, at, pad=2), key)
    assert torch.equal(got[:at], clean[:at]) and torch.equal(got[260:], clean[260:])
    if bad != bad:
        assert got[at:260, :G].isnan().all()

    def query(p):
        p.q[at, 1] = bad

    clean, got = finite_elsewhere(Prompts(lens, 2 * G, 2, 64, dtype, at, pad=2), query)
    assert got[at, 1].isnan().all()
    mask = torch.ones(got.shape[:2], dtype=torch.bool)
    mask[at, 1] = False
    assert torch.equal(got[mask], clean[mask])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_behind_the_last_sequence_do_not_matter(dtype):
    def spoil(p):
        for t in (p.q, p.k, p.v):
            t[-40:] = float("nan")

    p = Prompts([100, 30], 4, 2, 128, dtype, 11, pad=40)
    clean, got = finite_elsewhere(p, spoil)
    assert torch.equal(clean, got) and bool((got[-40:] == 7.0).all())


def test_many_infinities_in_every_channel():
    def value(p):
        p.v[70:90, 0] = float("inf")
        p.v[80:100, 0, ::2] = -float("inf")

    clean, got = finite_elsewhere(Prompts([220], 4, 1, 128, F16, 12), value)
    assert torch.equal(got[:70], clean[:70]) and not torch.isfinite(got[70:]).any()
    assert (got[75] == float("inf")).all() and got[99, :, ::2].isnan().all()


@pytest.mark.parametrize("starts", [[0, 60, 40, 100], [0, 50, 120, 100], [0, 0, 0, 100], [0, 100, 100, 100]])
def test_starts_that_cannot_be_read_nothing_outside(starts):
    p = Prompts([30, 30, 40], 4, 2, 64, F16, 13).start()
    p.dst = torch.tensor(starts, dtype=torch.int32, device="cuda")
    p.max_len = 120
    p.run()
    torch.cuda.synchronize()
    if starts[1] == 0 or starts[1] == 100:
        p.starts, p.lens = np.array([0, 100]), [100]
        p.check()


def test_a_single_row_of_any_stride():
    for n, H, Hk in ((1, 4, 2), (1, 1, 1), (3, 1, 1)):
        p = Prompts([n], H, Hk, 64, F16, n).start()
        wide = torch.randn((n, 8 * 64), device="cuda").half()
        wide[:, :H * 64] = p.dq.flatten(1)
        p.dq = wide[:, :H * 64].unflatten(1, (H, 64))
        p.run().check()


def test_rows_further_apart_than_32_bits():
    n, wide = 1100, 1 << 21  # 4.6 GB of rows, elements past 2^31
    p = Prompts([n], 4, 2, 64, BF16, 14).start()
    big = torch.zeros((n, wide), dtype=BF16, device="cuda")
    parts = []
    for x, at in ((p.dq, 0), (p.dk, 1 << 20), (p.dv, (1 << 21) - 128)):
        m = x.shape[1] * 64
        big[:, at:at + m] = x.flatten(1)
        parts.append(big[:, at:at + m].unflatten(1, (x.shape[1], 64)))
    p.dq, p.dk, p.dv = parts
    p.run().check()


def test_pools_past_four_gigabytes():
    N, B, Hk, d = 150000, 16, 8, 128
    p = Prompts([50], 8, Hk, d, F16, 15).start()
    p.kc, p.vc = (torch.zeros((N, B, Hk, d), dtype=F16, device="cuda") for _ in range(2))
    slots = torch.arange(50) + N * B - 50
    p.dsl = slots.cuda()
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.kc.flatten(0, 1)[slots.cuda()].cpu(), p.k) and torch.equal(p.vc.flatten(0, 1)[slots.cuda()].cpu(), p.v)
    assert not p.kc[0].any()
    p.cache = False
    p.check()


def test_captured_and_replayed_with_new_contents_and_lengths():
    p = Prompts([150, 70, 90], 8, 2, 128, BF16, 16, pad=10).start()
    p.max_len = 200
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.run()
    for seed, lens in ((17, [10, 200, 100]), (18, [200, 0, 1]), (19, [107, 107, 106])):
        n = Prompts(lens, 8, 2, 128, BF16, seed, pad=320 - sum(lens))
        for a, b in ((p.dq, n.q), (p.dk, n.k), (p.dv, n.v), (p.dsl, n.slots), (p.dst, torch.from_numpy(n.starts))):
            a.copy_(b)
        p.out.fill_(7.0)
        p.kc.fill_(3.0), p.vc.fill_(5.0)
        graph.replay()
        n.out, n.kc, n.vc, n.N = p.out, p.kc, p.vc, p.N
        n.max_len = 200
        n.check()


def test_two_calls_at_once_on_two_streams_and_repeatably():
    a = Prompts([300, 200, 5], 16, 4, 128, F16, 20).start()
    b = Prompts([33] * 30, 12, 4, 64, BF16, 21, fused=True).start()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    first = None
    for _ in range(4):
        a.run(sa), b.run(sb)
        torch.cuda.synchronize()
        if first is not None:
            assert torch.equal(first[0], a.out) and torch.equal(first[1], b.out)
        first = a.out.clone(), b.out.clone()
    a.check(), b.check()


def test_empty_calls_do_nothing():
    p = Prompts([10], 4, 2, 64, F16, 22).start()
    before = p.out.clone(), p.kc.clone()
    p.max_len = 0
    p.run()
    api.pa_prefill_packed(p.out[:0], p.dq[:0], p.dk[:0], p.dv[:0], p.dst, 5, 0.1, p.kc, p.vc, p.dsl[:0])
    api.pa_prefill_packed(p.out, p.dq, p.dk, p.dv, p.dst[:1], 5, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(before[0], p.out) and torch.equal(before[1], p.kc)


def test_binding_refuses_what_it_cannot_take():
    p = Prompts([10, 20], 4, 2, 64, F16, 23).start()
    good = dict(out=p.out, q=p.dq, key=p.dk, value=p.dv, query_start_loc=p.dst, max_query_len=20, scale=0.1, k_cache=p.kc,
                v_cache=p.vc, slot_mapping=p.dsl)
    for error, kw in [(TypeError, dict(q=p.dq.float())), (TypeError, dict(key=p.dk.bfloat16())), (ValueError, dict(key=p.dk[:9])),
                      (ValueError, dict(value=p.dv[:, :1])), (ValueError, dict(out=p.out[:3])), (ValueError, dict(value=p.dv.cpu())),
                      (ValueError, dict(k_cache=None)), (ValueError, dict(slot_mapping=None)), (ValueError, dict(slot_mapping=p.dsl[:4])),
                      (TypeError, dict(slot_mapping=p.dsl.int())), (TypeError, dict(query_start_loc=p.dst.long())),
                      (ValueError, dict(query_start_loc=p.dst[:0])), (ValueError, dict(v_cache=p.vc[:, :, :1])),
                      (TypeError, dict(k_cache=p.kc.bfloat16(), v_cache=p.vc.bfloat16())),
                      (ValueError, dict(q=p.dq.transpose(0, 1).contiguous().transpose(0, 1))),
                      (ValueError, dict(out=torch.zeros((30, 8, 64), dtype=F16, device="cuda")[:, ::2]))]:
        with pytest.raises(error):
            api.pa_prefill_packed(**{**good, **kw})
    odd = torch.zeros((30, 4 * 64 + 4), dtype=F16, device="cuda")[:, :256].unflatten(1, (4, 64))
    with pytest.raises(api.PagedAttnError):  # rows that do not start on 16 bytes
        api.pa_prefill_packed(**{**good, "q": odd})
    with pytest.raises(api.PagedAttnError):  # every row the same
        api.pa_prefill_packed(**{**good, "key": p.dk[:1].expand(30, 2, 64)})
    with pytest.raises(api.PagedAttnError):
        api.pa_prefill_packed(**{**good, "scale": float("nan")})
    torch.cuda.synchronize()
    assert bool((p.out == 7.0).all())


@pytest.mark.parametrize("dtype,H,Hk,d,B", [(F16, 8, 2, 128, 16), (BF16, 6, 2, 64, 32)])
def test_requests_from_prompt_to_compaction(dtype, H, Hk, d, B):
    """Two layers: prompts come in, attend and are written; samples fork off them and grow by a token
    of their own each; decode attends; some leave, the pool is made dense, decode attends again."""
    layers, S, M, N = 2, 8, 12, 60
    rng, g = np.random.default_rng(0), torch.Generator().manual_seed(0)
    scale = float(np.float32(d ** -0.5))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tables, lens = torch.full((S, M), -1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    counts = torch.zeros(N, dtype=torch.int32, device="cuda")
    counts[torch.from_numpy(rng.permutation(N)[:9]).cuda()] = 1  # blocks that somebody else holds
    pools = torch.full((layers, 2, N, B, Hk, d), float("nan"), dtype=dtype, device="cuda")
    flat = pools.view(layers * 2, N, B, Hk, d)
    space = api.alloc_sequence_workspace(N, "cuda")
    copies, left = torch.empty((S, 2), dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    hist = [[[np.zeros((0, Hk, d))] * 2 for _ in range(layers)] for _ in range(S)]  # every sequence's keys and values

    def new_rows(n):
        return [(torch.randn((n, Hk, d), generator=g).to(dtype), torch.randn((n, Hk, d), generator=g).to(dtype)) for _ in range(layers)]

    def grow(new):
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        slots = torch.empty(int(starts[-1]), dtype=torch.int64, device="cuda")
        api.pa_extend_sequences(tables, lens, counts, torch.from_numpy(starts).cuda(), slots, copies, left, B, space)
        api.pa_copy_layer_blocks(flat, copies)
        rows = new_rows(int(starts[-1]))
        for s in range(S):
            for x in range(layers):
                hist[s][x] = [np.concatenate([h, to_np(r[starts[s]:starts[s + 1]])]) for h, r in zip(hist[s][x], rows[x])]
        return starts, slots, rows

    def close(got, q, s, x, upto):
        k, v = (h[:upto] for h in hist[s][x])
        for h in range(H):
            sc = k[:, h // (H // Hk)] @ to_np(q)[h] * scale
            w = np.exp(sc - sc.max())
            w /= w.sum()
            want, A = w @ v[:, h // (H // Hk)], w @ np.abs(v[:, h // (H // Hk)])
            tol = HALF_STEP[dtype] * (A + np.abs(want)) + 1e-4 * A + 2.0 ** -20
            assert (np.abs(to_np(got)[h] - want) <= tol).all()

    # prompts
    new = [50, 33, 0, 0, 0, 0, 0, 0]
    starts, slots, rows = grow(new)
    assert left.tolist()[1] == 0
    for x in range(layers):
        q = torch.randn((sum(new), H, d), generator=g).to(dtype)
        out = torch.empty((sum(new), H, d), dtype=dtype, device="cuda")
        api.pa_prefill_packed(out, q.cuda(), rows[x][0].cuda(), rows[x][1].cuda(), torch.from_numpy(starts).cuda(), 50, scale,
                              pools[x, 0], pools[x, 1], slots)
        for t in (0, 17, 49, 50, 82):
            s = 0 if t < 50 else 1
            close(out[t], q[t], s, x, t - int(starts[s]) + 1)

    def decode_all():
        torch.cuda.synchronize()
        now = lens.tolist()
        assert now == [len(hist[s][0][0]) for s in range(S)]
        want = so.holders(tables.cpu().numpy(), lens.cpu().numpy(), N, B)
        assert (counts.cpu().numpy() - want).sum() == 9
        for x in range(layers):
            q = torch.randn((S, H, d), generator=g).to(dtype)
            out = torch.empty((S, H, d), dtype=dtype, device="cuda")
            api.pa_decode(out, q.cuda(), pools[x, 0], pools[x, 1], tables, lens, scale)
            for s in range(S):
                if now[s]:
                    close(out[s], q[s], s, x, now[s])

    decode_all()
    # samples, each with tokens of its own
    source = [-1, -1, 0, 0, 1, 1, 1, -1]
    api.pa_fork_sequences(tables, lens, counts, i32(*source), B)
    for s, f in enumerate(source):
        if f >= 0:
            hist[s] = [list(h) for h in hist[f]]
    for step in ([1, 0, 1, 1, 1, 1, 0, 0], [2, 1, 1, 0, 3, 20, 1, 0], [1, 1, 1, 1, 1, 1, 1, 1]):
        starts, slots, rows = grow(step)
        for x in range(layers):
            api.pa_reshape_and_cache(rows[x][0].cuda(), rows[x][1].cuda(), pools[x, 0], pools[x, 1], slots)
        decode_all()
    # some leave, one takes tokens back; the rest moves together
    to = [0, -1, 40, -1, -1, 0, -1, -1]
    api.pa_truncate_sequences(tables, lens, counts, i32(*to), B)
    for s, n in enumerate(to):
        if n >= 0:
            hist[s] = [[h[:n] for h in layer] for layer in hist[s]]
    moves, num = torch.empty((N, 2), dtype=torch.int64, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    api.pa_compact_blocks(moves, num, tables, lens, counts, tables, counts, B, space)
    api.pa_copy_layer_blocks(flat, moves)
    flat[:, int((counts != 0).sum()):] = float("nan")  # what was given back
    assert int(num) > 0
    decode_all()


# ------------------------------------------------------------- scores of any size
def exact_scores(p, sizes, key_exp, falling=False):
    """Scores without an error: q is one power of two a row (`sizes`, log 2 of its magnitude; every third row is
    negative), a key one number of 8 significant bits, growing from key to key.  Sums of d products stay below 2^24 of
    their smallest step, so float32 holds them."""
    n = p.rows
    step = torch.arange(n) * 127 // max(1, n - 1)
    k = (128 + (127 - step if falling else step)).double() * 2.0 ** (key_exp - 7)
    p.k[:] = k.to(p.dtype)[:, None, None]
    e = torch.tensor([sizes[i % len(sizes)] for i in range(n)])
    sign = torch.where(torch.arange(n) % 3 == 2, -1.0, 1.0).double()
    p.q[:] = (sign * 2.0 ** e.double()).to(p.dtype)[:, None, None]
    p.q[:, 1::2] *= 0.5  # heads of another size
    assert torch.isfinite(p.q.float()).all() and torch.isfinite(p.k.float()).all()
    return p


def check_exact_scores(p):
    """The tolerance without the scores' own error.  What is left of it: a difference of two scores is exact and is
    multiplied by a factor off by half a step, by an operation off by half a step: 2^-23 of itself, where a weight
    2^-g has g 2^-g <= 0.54; up to |m| = 2^16 (log 2 units) a row's offsets m are rounded, by 2^-24 |m| at most in
    each of three places for every block half at which they move."""
    torch.cuda.synchronize()
    got = to_np(p.out)
    q, k, v = to_np(p.q), to_np(p.k), to_np(p.v)
    with np.errstate(all="ignore"):
        want, A, _ = so.attention(q, k, v, p.starts, p.scale, p.max_len)
        n = max(p.lens)
        sums = 2.0 ** -22 + (n / 8 + 16) * 2.0 ** -24
        m = (np.abs(q[..., 0]) * np.abs(np.where(np.isfinite(k), k, 0)).max() * p.d * abs(p.scale) * 1.4427)[..., None]
        moved = np.minimum(m, 2.0 ** 16) * 3 * 2.0 ** -24 * (n / 64 + 1)
        tiny = n * 2.0 ** -32 * np.abs(v).max() + 2.0 ** -25 if p.dtype == F16 else 2.0 ** -100
        tol = HALF_STEP[p.dtype] * (A + np.abs(want)) + 2 * A * (sums + 2.0 ** -23 + moved) + tiny
        err = np.abs(got - want)
    assert np.isfinite(got).all() and (err <= tol).all(), \
        (np.argwhere(~(err <= tol))[:4].tolist(), float(np.nanmax(err / tol)))
    p.check_pools(np.ones(p.rows, bool))


# log 2 of the largest q and key of each type: products to 2^30 and 2^118, scores to 2^37 and 2^125
LARGEST = {F16: (15, 14), BF16: (59, 58)}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, -1.0, 0.088])
@pytest.mark.parametrize("size", [0, 7, 8, 9, 11, 13, 15, "largest"])
def test_equal_scores_of_any_size(size, scale, d, dtype):
    """A row of equal scores is the mean of its values; with one key, the value itself."""
    p = Prompts([1, 2, 70, 300], 2, 1, d, dtype, 40)
    a, b = LARGEST[dtype] if size == "largest" else (size, min(size, 14))
    p.q.fill_(2.0 ** a), p.k.fill_(2.0 ** b)
    p.scale = float(np.float32(scale))
    p.start().run()
    check_exact_scores(p)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("sizes,key_exp", [([-3], 0), ([3], 4), ([5, 6], 5), ([9], 7), ([12], 10), ([15], 14),
                                           ([-6, 0, 4, 8, 12, 15], 6), ([15, -9, -9, 2], 14), ([-14, 3, 15], 0)])
def test_growing_and_falling_scores_of_any_size(sizes, key_exp, scale, falling, d, dtype):
    """Rows of small and of large scores side by side; maxima that move far at every block, or stay at the first key."""
    p = exact_scores(Prompts([3, 400], 2, 1, d, dtype, 41), sizes, key_exp, falling)
    p.scale = scale
    p.start().run()
    check_exact_scores(p)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, -1.0, 4096.0])  # the last: past float32 when multiplied by log2(e) and the scale
def test_the_largest_scores_of_bfloat16(scale, d):
    for falling in (False, True):
        p = exact_scores(Prompts([2, 300], 4, 2, d, BF16, 42), [59, -30, 59, 40], 58, falling)
        p.scale = scale
        p.start().run()
        check_exact_scores(p)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores_beside_keys_of_minus_infinity(d, dtype):
    p = exact_scores(Prompts([400], 2, 1, d, dtype, 43), [15, 3, 12], 13)
    p.q = p.q.abs()
    p.k[1::5] = -float("inf")
    p.k[130:260] = -float("inf")
    p.start().run()
    check_exact_scores(p)


# ----------------------------------------------------- bad starts, and what is not finite at head_dim 128
def with_margins(x, rows, value):
    """x as a view with `rows` rows of `value` before and behind it, and a function that says whether those stand."""
    room = torch.full((x.shape[0] + 2 * rows,) + tuple(x.shape[1:]), value, dtype=x.dtype, device=x.device)
    view = room[rows:rows + x.shape[0]]
    view.copy_(x)
    return view, lambda: bool((room[:rows] == value).all()) and bool((room[rows + x.shape[0]:] == value).all())


def check_inside(p, starts):
    """Run p with these starts: nothing is written around out and the pools, and what is written is what belongs there."""
    p.start()
    p.dst = torch.as_tensor(starts, dtype=torch.int32).cuda()
    p.out, out_ok = with_margins(p.out, 300, 7.0)
    p.kc, k_ok = with_margins(p.kc, 20, 3.0)
    p.vc, v_ok = with_margins(p.vc, 20, 5.0)
    p.run()
    torch.cuda.synchronize()
    assert out_ok() and k_ok() and v_ok()
    assert bool(torch.isfinite(p.out.float()).all())
    for pool, new, empty in ((p.kc, p.k, 3.0), (p.vc, p.v, 5.0)):
        rows = pool.flatten(0, 1).cpu()
        there = rows[p.slots]
        written = (there == new).flatten(1).all(1)
        assert bool((written | (there == empty).flatten(1).all(1)).all())
        rows[p.slots] = empty
        assert bool((rows == empty).all())
    return p


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top", [3000, 100])  # the list of all pairs, and the grid
def test_starts_in_no_order_write_nothing_outside(top, d):
    rng = np.random.default_rng(32)
    for _ in range(3):
        check_inside(Prompts([3000], 4, 2, d, F16, 31), rng.integers(-100, top + 100, 201))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("starts", [[0, 60, 40, 100], [0, 50, 120, 100], [2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31, 100], [-2 ** 31, 2 ** 31 - 1, 0, 50],
                                    [-300, -200, -100, 0], [100, 200, 300, 400], [0, 0, 0, 1000], [-1000, 100, 100, 100]])
def test_bad_starts_write_nothing_outside(starts, d):
    p = Prompts([30, 30, 40], 4, 2, d, F16, 13)
    p.max_len = 120
    check_inside(p, starts)
    if starts[2:] == [0, 1000] or starts[0] == -1000:  # one prompt of all rows
        p.starts, p.lens = np.array([0, 100]), [100]
        p.check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 63, 64, 127, 128, 200, 259])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_what_is_not_finite_at_head_dim_128(dtype, bad, at, G):
    lens, others = [260, 150], [c for c in range(128) if c != 77]
    prompts = lambda: Prompts(lens, 2 * G, 2, 128, dtype, at, pad=2)  # noqa: E731

    def value(p):
        p.v[at, 0, 77] = bad

    clean, got = finite_elsewhere(prompts(), value)
    assert torch.equal(got[:at], clean[:at]) and torch.equal(got[260:], clean[260:])
    assert torch.equal(got[at:260, G:], clean[at:260, G:])
    seen = got[at:260, :G]
    assert not torch.isfinite(seen[..., 77]).any()
    assert torch.equal(seen[..., others], clean[at:260, :G][..., others])

    def key(p):
        p.k[at, 0, 77] = bad

    p = prompts()
    clean, got = finite_elsewhere(p, key)
    assert torch.equal(got[:at], clean[:at]) and torch.equal(got[260:], clean[260:])
    assert torch.equal(got[at:260, G:], clean[at:260, G:])
    # a score of +inf or NaN makes the row NaN, one of -inf weighs nothing
    # The tolerance at the head of this file: A is that of the weights there are (one with key `at` at a score of 0, not of
    # -inf, gives its value a weight that it does not have, and so an A below sum w |v|: a row of two keys has twice that);
    # S is that of the other keys, a score of -inf having no error.
    q, k, v = to_np(p.q), to_np(p.k), to_np(p.v)
    with np.errstate(all="ignore"):
        want, A, _ = (x[at:260, :G] for x in so.attention(q, k, v, p.starts, p.scale))
        S = so.attention(q, np.where(np.isfinite(k), k, 0), v, p.starts, p.scale)[2][at:260, :G]
        n, top = max(lens), np.abs(v).max()
        tiny = n * 2.0 ** -32 * top + 2.0 ** -25 if dtype == F16 else 2.0 ** -100
        tol = HALF_STEP[dtype] * (A + np.abs(want)) + tiny + A * (
            2 * (p.d + 4) * 2.0 ** -24 * S[..., None] + 2 * (2.0 ** -22 + (n / 8 + 16) * 2.0 ** -24))
    seen = got[at:260, :G].double().numpy()
    assert np.array_equal(np.isnan(seen), np.isnan(want))
    fine = ~np.isnan(want)
    assert (np.abs(seen - want)[fine] <= tol[fine]).all(), float((np.abs(seen - want) / tol)[fine].max())

    def query(p):
        p.q[at, 1] = bad

    clean, got = finite_elsewhere(prompts(), query)
    assert got[at, 1].isnan().all()
    mask = torch.ones(got.shape[:2], dtype=torch.bool)
    mask[at, 1] = False
    assert torch.equal(got[mask], clean[mask])


def test_beside_library_products_on_its_stream_and_another():
    """Matrix products whose kernels use tensor memory too run before and behind the prompts in their stream, and on
    another stream at the same time."""
    p = Prompts([300, 77, 200], 8, 2, 64, BF16, 44).start()
    a = torch.randn((1024, 1024), device="cuda").bfloat16()
    want = (a @ a).clone()
    torch.cuda.synchronize()
    here, other = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(30):
        with torch.cuda.stream(other):
            x = a @ a
        with torch.cuda.stream(here):
            y = a @ a
            p.run()
            z = a @ a
    torch.cuda.synchronize()
    p.check()
    assert all(torch.equal(t, want) for t in (x, y, z))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_scale(sign, d, dtype):
    """Tiny elements and a large scale (bf16: 2^127, products from 2^-121 on), which are ordinary scores."""
    sizes, key_exp = ([-12, -10, -11], -5) if dtype == F16 else ([-30, -28, -29], -90)
    p = exact_scores(Prompts([3, 200], 2, 1, d, dtype, 45), sizes, key_exp)
    p.scale = sign * (2.0 ** 14 if dtype == F16 else 2.0 ** 127)
    p.start().run()
    check_exact_scores(p)
