"""The per-block entry points as programs use them: captured into graphs and
replayed with new contents, on other streams, side by side, over pools beyond
2^32 bytes, with a shared block copied on write; and what the binding refuses."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_cases import Batch, assert_close, to_np
from oracle import block_oracle as bo
from paged_kv_cache_173_gb300 import _lib, api
from paged_kv_cache_173_gb300._lib import PagedAttnError

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


class Step:
    """The device side of a batch, with every call of a sparse decode step."""

    def __init__(self, b, keep=6, first=1, last=2):
        self.b, self.keep, self.first, self.last = b, keep, first, last
        (self.q, self.kc, self.vc, self.ks, self.vs, self.bt, self.cl) = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens")
        S = len(b.lens_list)
        g = torch.Generator().manual_seed(7)
        self.key = torch.randn((S, b.Hk, b.d), generator=g).to(b.dtype).cuda()
        self.value = torch.randn((S, b.Hk, b.d), generator=g).to(b.dtype).cuda()
        slots = [int(b.tables[s, (n - 1) // b.B]) * b.B + (n - 1) % b.B for s, n in enumerate(b.lens_list)]
        self.slots = torch.tensor(slots).cuda()
        x = torch.nan_to_num(b.keys16.float(), nan=0.0).to(b.dtype).reshape(-1, b.Hk, b.d)
        codes, exps = bo.bounds(to_np(x), np.zeros((b.N, b.Hk, 2, b.d), np.int8), np.zeros((b.N, b.Hk), np.int32),
                                np.arange(b.N * b.B), b.B)
        self.bounds, self.exps = torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda()
        self.st = torch.empty((S, b.Hk, keep), dtype=torch.int32, device="cuda")
        self.sl = torch.empty((S, b.Hk), dtype=torch.int32, device="cuda")
        self.ws = api.alloc_select_workspace(S, b.Hk, b.M, "cuda")
        self.P = api.max_num_partitions_for(b.M, b.B, 2 * b.B)
        self.ws2 = api.alloc_splitk_workspace(S, b.H, b.d, self.P, "cuda")
        self.dense, self.split, self.sparse = (torch.full_like(self.q, float("nan")) for _ in range(3))

    def run(self, stream=None):
        b = self.b
        api.pa_reshape_and_cache_fp8_block(self.key, self.value, self.kc, self.vc, self.ks, self.vs, self.slots, stream=stream)
        api.pa_update_key_bounds(self.key, self.bounds, self.exps, self.slots, b.B, stream=stream)
        api.pa_decode_fp8_block(self.dense, self.q, self.kc, self.vc, self.ks, self.vs, self.bt, self.cl, b.scale, stream=stream)
        api.pa_decode_splitk_fp8_block(self.split, self.q, self.kc, self.vc, self.ks, self.vs, self.bt, self.cl, b.scale,
                                       2 * b.B, self.ws2, self.P, stream=stream)
        api.pa_splitk_reduce(self.split, self.ws2, self.cl, b.M, b.B, 2 * b.B, self.P, stream=stream)
        api.pa_select_blocks(self.st, self.sl, self.q, self.bounds, self.exps, self.bt, self.cl, b.B, self.first, self.last,
                             self.ws, stream=stream)
        api.pa_decode_sparse(self.sparse, self.q, self.kc, self.vc, self.st, self.sl, b.scale, self.ks, self.vs, stream=stream)

    def check(self):
        b = self.b
        torch.cuda.synchronize()
        kc, ks = bo.write(to_np(self.key), b.kc.numpy(), b.ks.numpy(), self.slots.cpu().numpy())
        vc, vs = bo.write(to_np(self.value), b.vc.numpy(), b.vs.numpy(), self.slots.cpu().numpy())
        assert np.array_equal(self.kc.cpu().numpy(), kc) and np.array_equal(self.vs.cpu().numpy(), vs, equal_nan=True)
        old = (b.kc, b.ks, b.vc, b.vs, b.q)
        b.kc, b.ks, b.vc, b.vs, b.q = (*[torch.from_numpy(x) for x in (kc, ks, vc, vs)], self.q.cpu())
        ref, tol = b.reference()
        assert_close(self.dense, ref, tol)
        assert_close(self.split, ref, tol)
        st, sl = bo.select(to_np(self.q), self.bounds.cpu().numpy(), self.exps.cpu().numpy(), b.tables.numpy(),
                           b.lens.numpy(), b.B, self.keep, self.first, self.last)
        assert np.array_equal(self.st.cpu().numpy(), st) and np.array_equal(self.sl.cpu().numpy(), sl)
        ref, tol = b.reference(True, st, sl)
        assert_close(self.sparse, ref, tol)
        b.kc, b.ks, b.vc, b.vs, b.q = old


def batch(seed, dtype=torch.float16, lens=(300, 47, 129, 512)):
    return Batch(list(lens), 8, 2, 64, 16, dtype, seed)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_step_captured_and_replayed_with_new_contents(dtype):
    s = Step(batch(1, dtype))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    pools = [t.clone() for t in (s.kc, s.vc, s.ks, s.vs, s.bounds, s.exps)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for seed in (3, 4):
        g = torch.Generator().manual_seed(seed)
        for t, src in zip((s.kc, s.vc, s.ks, s.vs, s.bounds, s.exps), pools):
            t.copy_(src)
        s.b.kc, s.b.vc, s.b.ks, s.b.vs = [t.cpu() for t in (s.kc, s.vc, s.ks, s.vs)]
        s.q.copy_(torch.randn(s.q.shape, generator=g).to(dtype))
        s.key.copy_((torch.randn(s.key.shape, generator=g) * 9).to(dtype))
        s.value.copy_((torch.randn(s.value.shape, generator=g) * 9).to(dtype))
        torch.cuda.synchronize()
        graph.replay()
        s.check()


def test_two_steps_at_once_on_two_streams():
    a, b = Step(batch(5)), Step(batch(6, lens=(1000, 5, 700)))
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):  # repeatable: the writes bring the same tokens again
        a.run(sa)
        b.run(sb)
    a.check()
    b.check()


def test_two_graphs_share_a_selection_workspace_in_turn():
    a, b = Step(batch(8)), Step(batch(9))
    b.ws = a.ws
    side = torch.cuda.Stream()
    graphs = []
    for s in (a, b):
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.run()
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    a.check()
    b.check()


def test_prefill_captured_and_replayed():
    b = Batch([150, 70], 8, 2, 128, 32, torch.bfloat16, 10, new=[100, 70])
    q, kc, vc, ks, vs, bt, cl, qs = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens", "starts")
    out = torch.empty_like(q)

    def run():
        api.pa_prefill_fp8_block(out, q, kc, vc, ks, vs, bt, cl, qs, 100, b.scale)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    b.q = (torch.randn(b.q.shape, generator=torch.Generator().manual_seed(1)) * 2).to(b.dtype)
    q.copy_(b.q)
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    ref, tol = b.prefill_reference()
    assert_close(out, ref, tol)


def test_pools_beyond_four_gigabytes():
    # 4.3 GB of codes per pool, 16-bit pools of 8.6 GB: the blocks in use lie at the far end
    N, B, Hk, d = 270000, 16, 8, 128
    S, n = 2, 45
    b = Batch([n] * S, 16, Hk, d, B, torch.float16, 11)
    far = torch.arange(N - b.N, N, dtype=torch.int32)
    tables = torch.where(b.tables >= 0, b.tables + (N - b.N), b.tables)
    kc, vc = (torch.zeros((N, B, Hk, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((N, Hk), device="cuda") for _ in range(2))
    slots = torch.tensor([int(tables[s, p // B]) * B + p % B for s in range(S) for p in range(n)])
    assert int(slots.max()) * Hk * d > 2 ** 32
    g = torch.Generator().manual_seed(12)
    key, value = ((torch.randn((S * n, Hk, d), generator=g)).half() for _ in range(2))
    api.pa_reshape_and_cache_fp8_block(key.cuda(), value.cuda(), kc, vc, ks, vs, slots.cuda())
    bounds, exps = torch.zeros((N, Hk, 2, d), dtype=torch.int8, device="cuda"), torch.zeros((N, Hk), dtype=torch.int32, device="cuda")
    api.pa_update_key_bounds(key.cuda(), bounds, exps, slots.cuda(), B)
    torch.cuda.synchronize()
    near = slots.numpy() - (N - b.N) * B
    zero = np.zeros((b.N, B, Hk, d), np.uint8), np.zeros((b.N, Hk), np.float32)
    wk, wks = bo.write(to_np(key), *zero, near)
    wv, wvs = bo.write(to_np(value), *zero, near)
    assert np.array_equal(kc[far.long().cuda()].cpu().numpy(), wk) and np.array_equal(vc[far.long().cuda()].cpu().numpy(), wv)
    assert not kc[: N - b.N].any()
    wb, we = bo.bounds(to_np(key), np.zeros((b.N, Hk, 2, d), np.int8), np.zeros((b.N, Hk), np.int32), near, B)
    assert np.array_equal(bounds[far.long().cuda()].cpu().numpy(), wb)
    b.kc, b.vc, b.ks, b.vs = [torch.from_numpy(x) for x in (wk, wv, wks, wvs)]
    q, bt, cl = b.q.cuda(), tables.cuda(), b.lens.cuda()
    out = torch.empty_like(q)
    api.pa_decode_fp8_block(out, q, kc, vc, ks, vs, bt, cl, b.scale)
    ref, tol = b.reference()
    assert_close(out, ref, tol)
    st, sl = torch.empty((S, Hk, 2), dtype=torch.int32, device="cuda"), torch.empty((S, Hk), dtype=torch.int32, device="cuda")
    api.pa_select_blocks(st, sl, q, bounds, exps, bt, cl, B, 0, 1, api.alloc_select_workspace(S, Hk, b.M, "cuda"))
    near_tables = b.tables.numpy()
    wt, wl = bo.select(to_np(b.q), wb, we, near_tables, b.lens.numpy(), B, 2, 0, 1)
    assert np.array_equal(st.cpu().numpy() - (N - b.N), wt) and np.array_equal(sl.cpu().numpy(), wl)
    api.pa_decode_sparse(out, q, kc, vc, st, sl, b.scale, ks, vs)
    ref, tol = b.reference(True, wt, wl)
    assert_close(out, ref, tol)
    # a prefill of the last 30 tokens of each
    p = Batch([n] * S, 16, Hk, d, B, torch.float16, 11, new=[30] * S)
    p.kc, p.vc, p.ks, p.vs = b.kc, b.vc, b.ks, b.vs
    out = torch.empty_like(p.q).cuda()
    api.pa_prefill_fp8_block(out, p.q.cuda(), kc, vc, ks, vs, bt, cl, p.starts.cuda(), 30, p.scale)
    ref, tol = p.prefill_reference()
    assert_close(out, ref, tol)


def test_copy_on_write_takes_the_scales_along():
    b = Batch([40, 33], 8, 4, 64, 16, torch.float16, 13)
    src = int(b.tables[0, 2])
    dst = sorted(set(range(b.N)) - set(b.tables.flatten().tolist()))[0]
    kc, vc, ks, vs = b.dev("kc", "vc", "ks", "vs")
    m = torch.tensor([[src, dst]]).cuda()
    api.pa_copy_blocks(kc, vc, m)
    api.pa_copy_blocks(ks.view(torch.uint8).view(b.N, 1, b.Hk, 4), vs.view(torch.uint8).view(b.N, 1, b.Hk, 4), m)
    bt = b.tables.clone()
    bt[0, 2] = dst
    out = torch.empty_like(b.q).cuda()
    api.pa_decode_fp8_block(out, b.q.cuda(), kc, vc, ks, vs, bt.cuda(), b.lens.cuda(), b.scale)
    ref, tol = b.reference()
    assert_close(out, ref, tol)
    assert torch.equal(ks[dst], ks[src]) and torch.equal(vs[dst], vs[src])


def test_empty_calls_do_nothing():
    b = batch(14)
    s = Step(b)
    before = s.kc.clone()
    none = torch.empty((0, b.Hk, b.d), dtype=b.dtype, device="cuda")
    api.pa_reshape_and_cache_fp8_block(none, none, s.kc, s.vc, s.ks, s.vs, torch.empty(0, dtype=torch.int64, device="cuda"))
    api.pa_update_key_bounds(none, s.bounds, s.exps, torch.empty(0, dtype=torch.int64, device="cuda"), b.B)
    q0 = torch.empty((0, b.H, b.d), dtype=b.dtype, device="cuda")
    bt0, cl0 = s.bt[:0], s.cl[:0]
    api.pa_decode_fp8_block(q0, q0, s.kc, s.vc, s.ks, s.vs, bt0, cl0, b.scale)
    api.pa_select_blocks(s.st[:0], s.sl[:0], q0, s.bounds, s.exps, bt0, cl0, b.B, 1, 2, s.ws)
    api.pa_decode_sparse(q0, q0, s.kc, s.vc, s.st[:0], s.sl[:0], b.scale, s.ks, s.vs)
    api.pa_prefill_fp8_block(q0, q0, s.kc, s.vc, s.ks, s.vs, s.bt, s.cl,
                             torch.zeros(len(b.lens_list) + 1, dtype=torch.int32, device="cuda"), 0, b.scale)
    torch.cuda.synchronize()
    assert torch.equal(before, s.kc)


def test_binding_refuses_what_it_cannot_take():
    b = batch(15)
    s = Step(b)
    dec = lambda **k: api.pa_decode_fp8_block(**{**dict(out=s.dense, q=s.q, k_cache=s.kc, v_cache=s.vc, k_scales=s.ks,  # noqa: E731
                                                        v_scales=s.vs, block_tables=s.bt, context_lens=s.cl, scale=b.scale), **k})
    for error, kw in [(ValueError, dict(k_scales=s.ks[:, :1])), (ValueError, dict(v_scales=s.vs[:-1])),
                      (TypeError, dict(k_scales=s.ks.double())), (ValueError, dict(k_scales=s.ks.cpu())),
                      (TypeError, dict(k_cache=s.kc.to(torch.int32))), (TypeError, dict(q=s.q.float(), out=s.dense.float())),
                      (TypeError, dict(out=s.dense.bfloat16())), (ValueError, dict(out=s.dense[:1])),
                      (ValueError, dict(block_tables=s.bt[:1])), (TypeError, dict(context_lens=s.cl.long())),
                      (ValueError, dict(q=s.q.transpose(1, 2).contiguous().transpose(1, 2))),
                      (ValueError, dict(block_tables=s.bt.t().contiguous().t()))]:
        with pytest.raises(error):
            dec(**kw)
    with pytest.raises(PagedAttnError):  # a pool whose blocks are no supported size
        dec(k_cache=s.kc[:, :8].contiguous(), v_cache=s.vc[:, :8].contiguous())
    with pytest.raises(ValueError):
        api.pa_decode_sparse(s.sparse, s.q, s.kc, s.vc, s.st, s.sl, b.scale)  # codes without scales
    with pytest.raises(ValueError):
        api.pa_decode_sparse(s.sparse, s.q, s.kc.half(), s.vc.half(), s.st, s.sl, b.scale, s.ks, s.vs)
    with pytest.raises(PagedAttnError):  # more forced blocks than are kept
        api.pa_select_blocks(s.st, s.sl, s.q, s.bounds, s.exps, s.bt, s.cl, b.B, 5, 2, s.ws)
    with pytest.raises(PagedAttnError):  # a workspace that is too small
        api.pa_select_blocks(s.st, s.sl, s.q, s.bounds, s.exps, s.bt, s.cl, b.B, 1, 2, s.ws[:8])
    with pytest.raises(ValueError):
        api.pa_update_key_bounds(s.key, s.bounds[:, :, :1], s.exps, s.slots, b.B)
    with pytest.raises(ValueError):
        api.pa_reshape_and_cache_fp8_block(s.key, s.value[:, :1], s.kc, s.vc, s.ks, s.vs, s.slots)
    with pytest.raises(TypeError):
        api.pa_reshape_and_cache_fp8_block(s.key, s.value, s.kc, s.vc, s.ks, s.vs, s.slots.int())
    torch.cuda.synchronize()


def test_short_way_takes_good_calls_and_no_others():
    """_fast launches a well-formed call itself; anything else it declines with nothing launched."""
    b = Batch([70, 1, 33], 4, 2, 128, 16, torch.float16, 12)
    q, kc, vc, ks, vs, bt, cl = b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens")
    out = torch.full_like(q, 7.0)
    fast, dev, sp = _lib.fast(), torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream
    good = [out, q, kc, vc, ks, vs, bt, cl, float(b.scale)]

    def answer(i=None, x=None, d=dev):
        a = list(good)
        if i is not None:
            a[i] = x
        return fast.decode(*a, d, sp)

    wide = torch.zeros(q.shape[0], q.shape[1], 2 * q.shape[2], dtype=q.dtype, device="cuda")
    for i, x in [(0, out.cpu()), (0, out.float()), (0, wide[..., ::2]), (1, q[:2]), (2, kc.to(torch.int8)), (3, vc[:-1]),
                 (4, ks.double()), (5, vs[:, :1]), (6, bt.long()), (6, bt[:, 0]), (7, cl[:2]), (8, 1), (8, None),
                 (8, float("nan")), (1, None), (1, q.double())]:
        assert answer(i, x) is False, (i, x)
    assert answer(d=dev + 1) is False
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    assert answer() is True
    want = torch.empty_like(q)
    api.pa_decode_fp8_block(want, q, kc, vc, ks, vs, bt, cl, b.scale)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert answer(2, kc.view(torch.float8_e4m3fn)) is True


class Prompts:
    """A prefill with more pairs of tiles than the GPU has SMs."""

    def __init__(self, seed, dtype=torch.float16, new=200, scale=None):
        g = np.random.default_rng(seed)
        lens = [int(x) for x in g.integers(new, 2 * new, 12)]
        self.b = Batch(lens, 16, 4, 64, 16, dtype, seed, new=[int(x) for x in g.integers(1, new + 1, 12)])
        if scale is not None:
            self.b.scale = scale
        self.args = self.b.dev("q", "kc", "vc", "ks", "vs", "tables", "lens", "starts")
        self.out = torch.full_like(self.args[0], float("nan"))

    def run(self, stream=None):
        api.pa_prefill_fp8_block(self.out, *self.args, max(self.b.new), self.b.scale, stream=stream)

    def check(self):
        torch.cuda.synchronize()
        self.b.q = self.args[0].cpu()
        assert_close(self.out, *self.b.prefill_reference())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prefill_captured_and_replayed_with_new_queries(dtype):
    p = Prompts(21, dtype)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.run()
        p.run()
    for seed in (5, 6):
        p.args[0].copy_(torch.randn(p.args[0].shape, generator=torch.Generator().manual_seed(seed)).to(dtype))
        p.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        p.check()


def test_prefills_and_steps_at_once_on_three_streams():
    a, b, c = Prompts(22), Prompts(23, torch.bfloat16), Step(batch(24))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(8):
        for x, s in zip((a, b, c), streams):
            x.run(s)
    for x in (a, b, c):
        x.check()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_negative_softmax_scale(dtype):
    p = Prompts(25, dtype, new=100, scale=-0.125)
    p.run()
    p.check()
    b = batch(26, dtype)
    b.scale = -0.125
    s = Step(b)
    s.run()
    s.check()
