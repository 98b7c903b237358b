"""The calls on the sequences' blocks against the oracle: every result is a whole number, so all
of them are equal to it, in any state: full pools, refused sequences, shared blocks, bad values."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import sequence_oracle as so
from paged_kv_cache_173_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Server:
    """Tables, lengths and counts on the device beside the oracle's; every call is made of both and compared."""

    def __init__(self, S, M, N, B, seed=0):
        self.S, self.M, self.N, self.B = S, M, N, B
        self.rng = np.random.default_rng(seed)
        self.set(np.full((S, M), -1, np.int32), np.zeros(S, np.int32), np.zeros(N, np.int32))
        self.ws = torch.full((api.pa_sequence_workspace_bytes(N) // 4,), 0x7F7F7F7F, dtype=torch.int32, device="cuda")

    def set(self, tables, lens, counts):
        self.host = (tables, lens, counts)
        self.tables, self.lens, self.counts = (dev(x) for x in self.host)

    def same(self):
        torch.cuda.synchronize()
        for name, got, want in zip(("tables", "lens", "counts"), (self.tables, self.lens, self.counts), self.host):
            got = got.cpu().numpy()
            assert np.array_equal(got, want), (name, np.argwhere(got != want)[:5].tolist())

    def extend(self, new, spare=3, starts=None, stream=None):
        if starts is None:
            starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = max(0, int(starts[-1]) + spare)
        slots = torch.full((T,), 77, dtype=torch.int64, device="cuda")
        copies = torch.full((self.S, 2), 77, dtype=torch.int64, device="cuda")
        left = torch.full((2,), 77, dtype=torch.int32, device="cuda")
        self.ws.fill_(0x7F7F7F7F)
        api.pa_extend_sequences(self.tables, self.lens, self.counts, dev(starts.astype(np.int32)), slots, copies, left, self.B, self.ws)
        *self.host, want_slots, want_copies, want_left = so.extend(*self.host, starts, T, self.B)
        self.same()
        assert np.array_equal(slots.cpu().numpy(), want_slots)
        assert np.array_equal(copies.cpu().numpy(), want_copies)
        assert np.array_equal(left.cpu().numpy(), want_left), (left, want_left)
        return want_slots, want_copies, want_left

    def truncate(self, to):
        api.pa_truncate_sequences(self.tables, self.lens, self.counts, dev(np.asarray(to, np.int32)), self.B)
        self.host = so.truncate(*self.host, np.asarray(to), self.B)
        self.same()

    def fork(self, source):
        api.pa_fork_sequences(self.tables, self.lens, self.counts, dev(np.asarray(source, np.int32)), self.B)
        self.host = so.fork(*self.host, np.asarray(source), self.B)
        self.same()

    def compact(self, limit, in_place=True):
        moves = torch.full((limit, 2), 77, dtype=torch.int64, device="cuda")
        num = torch.full((1,), 77, dtype=torch.int32, device="cuda")
        to, co = (self.tables, self.counts) if in_place else (torch.full_like(self.tables, 77), torch.full_like(self.counts, 77))
        before = self.host
        api.pa_compact_blocks(moves, num, self.tables, self.lens, self.counts, to, co, self.B, self.ws)
        want_moves, want_num, tables, counts = so.compact(*self.host, limit, self.B)
        if not in_place:
            self.same()
            self.tables, self.counts = to, co
        self.host = (tables, before[1], counts)
        self.same()
        assert int(num) == want_num and np.array_equal(moves.cpu().numpy(), want_moves)
        return want_moves[:want_num]

    def any_call(self, most):
        rng, S = self.rng, self.S
        op = rng.integers(0, 6)
        if op <= 1:
            return self.extend(rng.integers(0, most, S) * (rng.random(S) < 0.5))
        if op == 2:
            return self.truncate(np.where(rng.random(S) < 0.4, rng.integers(-1, self.M * self.B, S), -1))
        if op == 3:
            self.truncate(np.where(rng.random(S) < 0.2, 0, -1))
            return self.fork(np.where(rng.random(S) < 0.5, rng.integers(-1, S + 1, S), -1))
        return self.compact(int(rng.integers(0, self.N + 2)), bool(op == 4))


@pytest.mark.parametrize("S,M,N,B,most", [
    (1, 1, 1, 16, 3), (1, 40, 33, 16, 90), (5, 7, 30, 16, 40), (17, 9, 100, 32, 100), (64, 33, 700, 16, 200),
    (300, 5, 1000, 64, 100), (9, 12, 70, 256, 900), (1100, 4, 3000, 16, 20), (40, 130, 4099, 16, 700), (3, 50, 127, 128, 2000)])
def test_random_walks(S, M, N, B, most):
    s = Server(S, M, N, B, seed=S + N)
    for _ in range(25):
        s.any_call(most)
    assert np.array_equal(s.host[2], so.holders(s.host[0], s.host[1], N, B))


def test_many_sequences_and_a_large_pool():
    s = Server(20000, 3, 150001, 16, seed=3)
    for _ in range(2):
        s.extend(s.rng.integers(0, 20, s.S))
        s.truncate(np.where(s.rng.random(s.S) < 0.5, s.rng.integers(0, 12, s.S), -1))
        s.fork(np.where(s.rng.random(s.S) < 0.5, s.rng.integers(0, s.S, s.S), -1))
        s.extend(s.rng.integers(0, 3, s.S))
        s.compact(1000)
        s.compact(150001, False)


def test_a_pool_of_four_million_blocks():
    N = 4 * 1024 * 1024 + 5
    s = Server(2, 2000, N, 16, seed=4)
    counts = (s.rng.random(N) < 0.999).astype(np.int32)
    counts[-3:] = 0
    s.set(s.host[0], s.host[1], counts)
    s.extend(np.array([2000 * 16, 1500 * 16]))
    s.extend(np.array([0, 400 * 16]))
    s.compact(3000)


def test_all_sequences_of_the_largest_batch():
    S = 65535
    s = Server(S, 1, S - 7, 16, seed=5)
    slots, _, left = s.extend(np.full(S, 2))
    assert left.tolist() == [0, 7] and (slots[-14 - 3:] == -1).all()
    s.truncate(np.where(np.arange(S) % 2 == 0, 0, -1))
    s.extend(np.where(np.arange(S) % 2 == 0, 16, 0))


def test_a_full_pool_refuses_in_order():
    s = Server(4, 4, 6, 16)
    _, _, left = s.extend(np.array([40, 33, 1, 0]))  # 3 + 3 blocks, then nothing is left
    assert left.tolist() == [0, 1] and s.host[1].tolist() == [40, 33, 0, 0]
    _, _, left = s.extend(np.array([8, 16, 0, 1]))   # room in the last block; one more block; none
    assert left.tolist() == [0, 2] and s.host[1].tolist() == [48, 33, 0, 0]
    _, _, left = s.extend(np.array([17, 15, 1, 1]))  # the table ends; fits; nothing left
    assert left.tolist() == [0, 3] and s.host[1].tolist() == [48, 48, 0, 0]
    s.truncate([16, 0, -1, 5])
    _, _, left = s.extend(np.array([0, 64, 20, 1]))  # 4 of 5 blocks, then 2 of 1: the next is refused too
    assert left.tolist() == [1, 2]


def test_a_shared_last_block_is_copied_once_for_each_that_grows():
    s = Server(5, 3, 20, 16)
    s.extend(np.array([20, 0, 0, 0, 0]))
    s.fork([-1, 0, 0, 0, -1])
    s.fork([-1, -1, -1, -1, 1])
    assert s.host[2][:2].tolist() == [5, 5]
    _, copies, _ = s.extend(np.array([0, 1, 15, 0, 0]))
    assert copies.tolist() == [[-1, -1], [1, 2], [1, 3], [-1, -1], [-1, -1]]
    _, copies, _ = s.extend(np.array([1, 1, 1, 1, 1]))  # all that are left leave it: it is free afterwards
    assert copies[:, 0].tolist() == [1, -1, -1, 1, 1] and s.host[2][1] == 0
    s.truncate([16, -1, -1, -1, -1])
    _, copies, _ = s.extend(np.array([3, 0, 0, 0, 0]))  # a whole shared block needs no copy
    assert copies[0].tolist() == [-1, -1]


@pytest.mark.parametrize("S,N,T", [(1024, 16384, 4096), (1024, 16384, 4097), (1024, 16385, 4096), (1025, 16384, 4096),
                                   (1, 16384, 4097), (1023, 16383, 4095), (1024, 262144, 4096), (1024, 262145 + 31, 4097)])
def test_sizes_on_both_sides_of_every_choice(S, N, T):
    s = Server(S, 300, N, 16, seed=T)
    new = np.full(S, T // S)
    new[S // 2] += T - new.sum()
    s.extend(new, spare=0)
    s.truncate(np.where(s.rng.random(S) < 0.5, s.rng.integers(0, 3, S), -1))
    s.fork(np.where(s.rng.random(S) < 0.5, s.rng.integers(0, S, S), -1))
    counts = s.host[2].copy()
    counts[s.rng.permutation(N)[:N // 2]] += 1  # blocks that somebody else holds
    s.set(s.host[0], s.host[1], counts)
    s.compact(N // 3)
    s.extend(new, spare=0)
    s.compact(N + 1, False)


def test_compaction_with_one_result_in_place():
    for tables_in, counts_in in ((True, False), (False, True)):
        s = Server(6, 5, 40, 16, seed=9)
        s.extend(np.array([50, 20, 80, 3, 16, 17]))
        s.truncate([0, -1, 20, -1, 0, -1])
        moves, num = torch.zeros((9, 2), dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        to = s.tables if tables_in else torch.full_like(s.tables, 77)
        co = s.counts if counts_in else torch.full_like(s.counts, 77)
        api.pa_compact_blocks(moves, num, s.tables, s.lens, s.counts, to, co, 16, s.ws)
        want, n, tables, counts = so.compact(*s.host, 9, 16)
        s.tables, s.counts, s.host = to, co, (tables, s.host[1], counts)
        s.same()
        assert n > 0 and int(num) == n and np.array_equal(moves.cpu().numpy(), want)


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 16, 49, -2 ** 31])
def test_a_length_past_the_table_in_a_compaction(length):
    s = Server(2, 3, 20, 16)
    s.extend(np.array([48, 48]))
    lens = s.host[1].copy()
    lens[1] = length
    counts = s.host[2].copy()
    counts[:2] = 0
    s.set(s.host[0], lens, counts)
    s.compact(20)


def test_two_graphs_in_turn_on_one_workspace():
    B, S, N = 16, 30, 20000
    servers = [Server(S, 20, N, B, seed=x) for x in (10, 11)]
    ws = servers[0].ws
    starts = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    outs, graphs = [], []
    for s in servers:
        o = (torch.zeros(200, dtype=torch.int64, device="cuda"), torch.zeros((S, 2), dtype=torch.int64, device="cuda"),
             torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros((40, 2), dtype=torch.int64, device="cuda"),
             torch.zeros(1, dtype=torch.int32, device="cuda"))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            api.pa_compact_blocks(o[3], o[4], s.tables, s.lens, s.counts, s.tables, s.counts, B, ws)
            api.pa_extend_sequences(s.tables, s.lens, s.counts, starts, *o[:3], B, ws)
        outs.append(o)
        graphs.append(graph)
    for i in range(6):
        begin = np.concatenate([[0], np.cumsum(servers[0].rng.integers(0, 7, S))]).astype(np.int32)
        starts.copy_(torch.from_numpy(begin))
        order = (0, 1) if i % 2 else (1, 0)
        for x in order:
            graphs[x].replay()
        for x in order:
            s, o = servers[x], outs[x]
            moves, _, tables, counts = so.compact(*s.host, 40, B)
            s.host = (tables, s.host[1], counts)
            *s.host, slots, copies, left = so.extend(*s.host, begin, 200, B)
            s.same()
            for got, want in zip(o, (slots, copies, left, moves)):
                assert np.array_equal(got.cpu().numpy(), want)
            cut = np.where(s.rng.random(S) < 0.3, 0, -1)
            s.truncate(cut)


def test_the_short_way_takes_the_calls():
    from paged_kv_cache_173_gb300 import _lib
    s = Server(4, 3, 20, 16)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    i64 = lambda *n: torch.zeros(n, dtype=torch.int64, device="cuda")  # noqa: E731
    at = (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream)
    fast, state = _lib.fast(), (s.tables, s.lens, s.counts)
    assert fast.extend(*state, i32(5), i64(3), i64(4, 2), i32(2), 16, s.ws, *at) is True
    assert fast.truncate(*state, i32(4), 16, *at) is True and fast.fork(*state, i32(4) - 1, 16, *at) is True
    assert fast.compact(i64(4, 2), i32(1), *state, s.tables, s.counts, 16, s.ws, *at) is True
    pools = torch.zeros((2, 20, 16, 2, 64), dtype=torch.float16, device="cuda")
    assert fast.copy_layers(pools, i64(3, 2), *at) is True
    q, kv = torch.zeros((5, 4, 64), device="cuda").half(), torch.zeros((5, 2, 64), device="cuda").half()
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    for cache in ((None, None, None), (pools[0], pools[1], i64(5))):
        assert fast.packed(torch.empty_like(q), q, kv, kv, starts, 5, 0.1, *cache, *at) is True
    torch.cuda.synchronize()
    s.same()


def test_forks_that_are_left_alone():
    s = Server(6, 3, 20, 16)
    s.extend(np.array([20, 0, 30, 0, 0, 0]))
    # onto a live one, from an empty one, from oneself, from outside, from one that is forked onto
    s.fork([2, 3, -1, 3, 6, 3])
    assert s.host[1].tolist() == [20, 0, 30, 0, 0, 0]
    s.fork([-1, 0, -1, 1, -7, 2])
    assert s.host[1].tolist() == [20, 20, 30, 0, 0, 30]


def test_bad_values_are_passed_over():
    s = Server(6, 3, 20, 16)
    s.extend(np.array([20, 20, 20, 20, 20, 0]))
    tables, lens, counts = (x.copy() for x in s.host)
    tables[0, 1], tables[1, 0], tables[2, 1] = 20, -5, 2 ** 31 - 1  # ids outside the pool
    lens[3], lens[4] = 49, -3  # a length past the table, a negative one
    s.set(tables, lens, counts)
    s.extend(np.array([1, 1, 1, 1, 1, 1]))
    s.fork([-1, -1, -1, -1, -1, 1])
    s.truncate([0, 0, 5, 0, 0, 3])
    s.compact(20)
    s.set(tables, lens, counts)
    s.compact(20, False)


@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [0, 5, 100, 8], [-4, 2, 3, 5], [0, 0, 0, 0], [2, 4, 6, 8]])
def test_starts_that_cannot_be_refuse_their_sequences_only(starts):
    s = Server(3, 3, 20, 16)
    starts = np.array(starts, np.int32)
    slots = torch.full((12,), 77, dtype=torch.int64, device="cuda")
    copies, left = torch.empty((3, 2), dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    api.pa_extend_sequences(s.tables, s.lens, s.counts, dev(starts), slots, copies, left, 16, s.ws)
    *s.host, want_slots, want_copies, want_left = so.extend(*s.host, starts, 12, 16)
    s.same()
    assert np.array_equal(copies.cpu().numpy(), want_copies) and np.array_equal(left.cpu().numpy(), want_left)
    if (np.diff(starts) >= 0).all():
        assert np.array_equal(slots.cpu().numpy(), want_slots)


def test_no_sequences_and_no_tokens():
    s = Server(2, 3, 20, 16)
    empty, none = s.tables[:0], s.lens[:0]
    slots, left = torch.full((4,), 5, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    api.pa_extend_sequences(empty, none, s.counts, torch.zeros(1, dtype=torch.int32, device="cuda"), slots,
                            torch.zeros((0, 2), dtype=torch.int64, device="cuda"), left, 16, s.ws)
    assert slots.tolist() == [-1] * 4 and left.tolist() == [20, 0]
    api.pa_truncate_sequences(empty, none, s.counts, none, 16)
    api.pa_fork_sequences(empty, none, s.counts, none, 16)
    num = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    api.pa_compact_blocks(torch.empty((0, 2), dtype=torch.int64, device="cuda"), num, empty, none, s.counts, empty, s.counts, 16, s.ws)
    assert int(num) == 0
    s.extend(np.array([0, 0]), spare=0)


@pytest.mark.parametrize("L,N,inner,dtype,pad", [
    (1, 5, (16, 2, 64), torch.float16, 0), (3, 40, (16, 8, 128), torch.bfloat16, 0), (7, 33, (2,), torch.float32, 0),
    (2, 30, (3, 5), torch.float32, 1), (4, 9, (2, 2, 128), torch.int8, 0), (2, 6, (256, 8, 128), torch.float16, 8),
    (32, 700, (1,), torch.float32, 0), (64, 300, (16, 1, 64), torch.float16, 0)])
def test_copy_of_layers(L, N, inner, dtype, pad):
    g = torch.Generator().manual_seed(L * N)
    size = int(np.prod(inner))
    flat = torch.randint(-100, 100, (L, N * size + pad), generator=g).to(dtype).cuda()
    pools = flat[:, :N * size].view(L, N, *inner) if pad == 0 else flat.as_strided(
        (L, N) + inner, (N * size + pad, size) + tuple(int(np.prod(inner[i + 1:])) for i in range(len(inner))))
    perm = torch.randperm(N, generator=g)
    n = N // 2
    pairs = torch.stack([perm[:n], perm[n:2 * n]], 1)
    bad = torch.tensor([[-1, 0], [0, -1], [N, 1], [1, N], [2, 2], [-1, -1], [2 ** 40, 0], [0, 2 ** 40]])
    both = torch.cat([pairs, bad])[torch.randperm(n + len(bad), generator=g)]
    want = flat.clone()
    view = want.as_strided(pools.shape, pools.stride())
    view[:, pairs[:, 1]] = pools[:, pairs[:, 0]]
    api.pa_copy_layer_blocks(pools, both.cuda())
    torch.cuda.synchronize()
    assert torch.equal(flat, want)


def test_copy_of_more_pairs_than_one_round_holds():
    pools = torch.arange(2 * 9000 * 4, dtype=torch.int32, device="cuda").view(2, 9000, 4)
    pairs = torch.stack([torch.arange(4500), torch.arange(4500) + 4500], 1)
    want = pools.clone()
    want[:, 4500:] = want[:, :4500]
    api.pa_copy_layer_blocks(pools, pairs.cuda())
    assert torch.equal(pools, want)


def test_copy_past_four_gigabytes():
    N, size = 70000, 16 * 8 * 128  # 2.3 GB a pool
    pools = torch.zeros((3, N, size), dtype=torch.float16, device="cuda")
    pools[:, 7] = torch.arange(3, device="cuda").half()[:, None] + 1
    api.pa_copy_layer_blocks(pools, torch.tensor([[7, N - 1]]).cuda())
    assert pools[:, N - 1].float().mean(1).tolist() == [1, 2, 3] and not pools[:, N - 2].any()


def test_captured_steps_replay_with_new_contents():
    B, S, N = 16, 40, 400
    s = Server(S, 20, N, B, seed=6)
    s.extend(s.rng.integers(1, 60, S))
    to, source, starts = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, S, S + 1))
    slots, copies = torch.zeros(300, dtype=torch.int64, device="cuda"), torch.zeros((S, 2), dtype=torch.int64, device="cuda")
    left, num = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    moves = torch.zeros((50, 2), dtype=torch.int64, device="cuda")
    pools = torch.randn((3, N, 8), device="cuda")

    def step():
        api.pa_truncate_sequences(s.tables, s.lens, s.counts, to, B)
        api.pa_fork_sequences(s.tables, s.lens, s.counts, source, B)
        api.pa_extend_sequences(s.tables, s.lens, s.counts, starts, slots, copies, left, B, s.ws)
        api.pa_copy_layer_blocks(pools, copies)
        api.pa_compact_blocks(moves, num, s.tables, s.lens, s.counts, s.tables, s.counts, B, s.ws)
        api.pa_copy_layer_blocks(pools, moves)

    keep = [x.clone() for x in (s.tables, s.lens, s.counts, pools)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    for x, y in zip((s.tables, s.lens, s.counts, pools), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    want = pools.cpu().numpy()
    for _ in range(6):
        cut = np.where(s.rng.random(S) < 0.4, s.rng.integers(0, 60, S) * (s.rng.random(S) < 0.5), -1)
        src = np.where(s.rng.random(S) < 0.5, s.rng.integers(0, S, S), -1)
        begin = np.concatenate([[0], np.cumsum(s.rng.integers(0, 7, S))]).astype(np.int32)
        for x, y in ((to, cut), (source, src), (starts, begin)):
            x.copy_(torch.from_numpy(y.astype(np.int32)))
        graph.replay()
        s.host = so.fork(*so.truncate(*s.host, cut, B), src, B)
        *s.host, want_slots, want_copies, want_left = so.extend(*s.host, begin, 300, B)
        want_moves, n, tables, counts = so.compact(*s.host, 50, B)
        s.host = (tables, s.host[1], counts)
        s.same()
        assert np.array_equal(slots.cpu().numpy(), want_slots) and np.array_equal(left.cpu().numpy(), want_left)
        assert np.array_equal(copies.cpu().numpy(), want_copies) and np.array_equal(moves.cpu().numpy(), want_moves)
        for pairs in (want_copies, want_moves):
            old = want.copy()
            for a, b in pairs.tolist():
                if a >= 0:
                    want[:, b] = old[:, a]
        assert np.array_equal(pools.cpu().numpy(), want)


def test_two_servers_on_two_streams():
    servers = [Server(50, 12, 300, 16, seed=x) for x in (7, 8)]
    news = [s.rng.integers(0, 30, (8, 50)) for s in servers]
    streams = [torch.cuda.Stream() for _ in servers]
    bufs = [[(dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)), torch.empty(int(n.sum()), dtype=torch.int64, device="cuda"),
              torch.empty((50, 2), dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"))
             for n in new] for new in news]
    half = torch.full((50,), 20, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i in range(8):
        for s, st, b in zip(servers, streams, bufs):
            api.pa_extend_sequences(s.tables, s.lens, s.counts, *b[i], s.B, s.ws, stream=st)
            api.pa_truncate_sequences(s.tables, s.lens, s.counts, half, s.B, stream=st)
    for s, new, b in zip(servers, news, bufs):
        for i in range(8):
            starts = b[i][0].cpu().numpy()
            *s.host, slots, _, left = so.extend(*s.host, starts, int(starts[-1]), s.B)
            assert np.array_equal(b[i][1].cpu().numpy(), slots) and np.array_equal(b[i][3].cpu().numpy(), left)
            s.host = so.truncate(*s.host, half.cpu().numpy(), s.B)
        s.same()


def test_binding_refuses_what_it_cannot_take():
    s = Server(4, 3, 20, 16)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    i64 = lambda *n: torch.zeros(n, dtype=torch.int64, device="cuda")  # noqa: E731
    good = dict(block_tables=s.tables, context_lens=s.lens, ref_counts=s.counts, query_start_loc=i32(5), slot_mapping=i64(3),
                block_copies=i64(4, 2), left=i32(2), block_size=16, workspace=s.ws)
    for error, kw in [(TypeError, dict(ref_counts=s.counts.long())), (ValueError, dict(ref_counts=s.counts.view(4, 5))),
                      (ValueError, dict(context_lens=s.lens[:3])), (ValueError, dict(block_tables=s.tables.t())),
                      (ValueError, dict(query_start_loc=i32(4))), (TypeError, dict(query_start_loc=i64(5))),
                      (TypeError, dict(slot_mapping=i32(3))), (ValueError, dict(block_copies=i64(3, 2))),
                      (ValueError, dict(left=i32(1))), (ValueError, dict(workspace=s.ws.cpu())),
                      (api.PagedAttnError, dict(workspace=s.ws[:10])), (api.PagedAttnError, dict(block_size=20)),
                      (ValueError, dict(slot_mapping=i64(6)[::2]))]:
        with pytest.raises(error):
            api.pa_extend_sequences(**{**good, **kw})
    with pytest.raises(ValueError):
        api.pa_truncate_sequences(s.tables, s.lens, s.counts, i32(3), 16)
    with pytest.raises(TypeError):
        api.pa_fork_sequences(s.tables, s.lens, s.counts, i64(4), 16)
    with pytest.raises(ValueError):
        api.pa_compact_blocks(i64(4, 3), i32(1), s.tables, s.lens, s.counts, s.tables, s.counts, 16, s.ws)
    with pytest.raises(ValueError):
        api.pa_compact_blocks(i64(4, 2), i32(1), s.tables, s.lens, s.counts, s.tables[:, :2], s.counts, 16, s.ws)
    with pytest.raises(ValueError):
        api.pa_copy_layer_blocks(torch.zeros((2, 4, 8), device="cuda").transpose(1, 2), i64(1, 2))
    with pytest.raises(TypeError):
        api.pa_copy_layer_blocks(torch.zeros((2, 4, 8), device="cuda"), i32(1, 2))
    with pytest.raises(ValueError):
        api.pa_copy_layer_blocks(torch.zeros((2, 4), device="cuda"), i64(1, 2))
    with pytest.raises(api.PagedAttnError):  # blocks of 3 bytes
        api.pa_copy_layer_blocks(torch.zeros((2, 4, 3), dtype=torch.uint8, device="cuda"), i64(1, 2))
    with pytest.raises(api.PagedAttnError):  # layers that overlap
        api.pa_copy_layer_blocks(torch.zeros(100, device="cuda").as_strided((2, 4, 8), (16, 8, 1)), i64(1, 2))
    s.same()


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("S", [4, 20, 1500])  # the last: several CTAs
@pytest.mark.parametrize("starts", [[TOP] * 5, [TOP - 1023] * 4 + [TOP], [0, 5, TOP - 1, TOP, TOP], [-2 ** 31, TOP - 7, TOP, TOP, TOP],
                                    [-2 ** 31] * 5, [0, 3, 3, 7, TOP], [TOP, 0, 4, 4, 9]])
def test_starts_near_the_ends_of_32_bits(starts, S):
    """Slots are written for the tokens there are, whatever the starts say; the first and the last sequences of
    the batch (and of every CTA) take the bad ones."""
    T = 12
    front = np.asarray(starts, np.int64)
    starts = np.concatenate([front[:3], np.full(S - 4, front[2]), front[3:]])
    s = Server(S, 3, 20, 16)
    room = torch.full((T + 128,), 77, dtype=torch.int64, device="cuda")
    slots = room[64:64 + T]
    copies, left = torch.empty((S, 2), dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    api.pa_extend_sequences(s.tables, s.lens, s.counts, dev(starts.astype(np.int32)), slots, copies, left, 16, s.ws)
    *s.host, want_slots, want_copies, want_left = so.extend(*s.host, starts, T, 16)
    s.same()
    assert np.array_equal(copies.cpu().numpy(), want_copies) and left.tolist()[0] == want_left[0]
    if (np.diff(starts) >= 0).all():
        assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert bool((room[:64] == 77).all()) and bool((room[64 + T:] == 77).all())


@pytest.mark.parametrize("sizes", [((1024, 16384), (10, 11000)), ((65535, 20000), (20000, 16400))])  # one CTA, several
def test_two_threads_with_pools_of_different_size(sizes):
    """Launches of one kernel with much and with less shared memory, from two threads at once: none is refused."""
    import threading

    from paged_kv_cache_173_gb300 import _lib
    L, refused = _lib.lib(), []

    def work(S, N):
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        tables, lens, counts, starts, left = i32(S, 2), i32(S), i32(N), i32(S + 1), i32(2)
        copies, ws, stream = torch.zeros((S, 2), dtype=torch.int64, device="cuda"), api.alloc_sequence_workspace(N, "cuda"), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(2000):
            status = L.pa_extend_sequences(tables.data_ptr(), 2, lens.data_ptr(), counts.data_ptr(), starts.data_ptr(), None,
                                           copies.data_ptr(), left.data_ptr(), S, 0, N, 16, ws.data_ptr(), 4 * ws.numel(),
                                           stream.cuda_stream)
            if status != _lib.PA_OK:
                refused.append((S, N, _lib.last_error()))
        stream.synchronize()
        if left.tolist() != [N, 0]:
            refused.append((S, N, left.tolist()))

    threads = [threading.Thread(target=work, args=x) for x in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == []


@pytest.mark.parametrize("name", ["pa_compact_blocks", "pa_extend_sequences"])
def test_a_launch_that_fails_is_raised_and_not_made_again(name, monkeypatch):
    """The entry point is replaced by one that says that a launch failed: its tensors may have changed by then."""
    import ctypes

    from paged_kv_cache_173_gb300 import _lib
    s, L, fast, made = Server(4, 3, 20, 16), _lib.lib(), _lib.fast(), []
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    i64 = lambda *n: torch.zeros(n, dtype=torch.int64, device="cuda")  # noqa: E731
    state = (s.tables, s.lens, s.counts)
    call = dict(pa_compact_blocks=lambda b: api.pa_compact_blocks(i64(4, 2), i32(1), *state, s.tables, s.counts, b, s.ws),
                pa_extend_sequences=lambda b: api.pa_extend_sequences(*state, i32(5), i64(3), i64(4, 2), i32(2), b, s.ws))[name]
    status = [_lib.PA_ERR_CUDA]
    res, args = _lib.SIGNATURES[name]
    fake = ctypes.CFUNCTYPE(res, *args)(lambda *a: made.append("short") or status[0])
    monkeypatch.setattr(L, name, lambda *a: made.append("own") or status[0])
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    fast.bind_sequences(*[address(fake if n == name else getattr(L, n)) for n in _lib.FAST_SEQUENCE_ENTRIES])
    try:
        with pytest.raises(api.PagedAttnError) as e:
            call(16)
        assert e.value.status == _lib.PA_ERR_CUDA and name in str(e.value) and made == ["short"]
        for status[0] in (_lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED):  # nothing was launched: api.py's own way names it
            made.clear()
            with pytest.raises(api.PagedAttnError) as e:
                call(16)
            assert e.value.status == status[0] and made == ["short", "own"]
    finally:
        monkeypatch.undo()
        fast.bind_sequences(*[address(getattr(L, n)) for n in _lib.FAST_SEQUENCE_ENTRIES])
    call(16)
    s.same()
    with pytest.raises(api.PagedAttnError) as e:
        call(20)
    assert e.value.status == _lib.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("S", [3, 1500])
def test_sequences_without_new_tokens_are_not_refused(S):
    """left[1] counts who asked for tokens and got none: not those of bad lengths, bad blocks or empty ranges outside
    the tokens that bring nothing."""
    s = Server(S, 3, 40 + 2 * S, 16)
    first = np.zeros(S, np.int64)
    first[:3] = 20
    s.extend(first)
    tables, lens, counts = (x.copy() for x in s.host)
    lens[0], lens[1], tables[2, 1] = -3, 49, 10 ** 9
    s.set(tables, lens, counts)
    _, copies, left = s.extend(np.zeros(S, np.int64))
    assert left[1] == 0 and (copies == -1).all()
    # one sequence asks for more tokens than there are slots; those behind it have empty ranges past the last token
    starts = np.full(S + 1, 100, np.int64)
    starts[0] = 0
    slots = torch.full((50,), 77, dtype=torch.int64, device="cuda")
    copies, left = torch.empty((S, 2), dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    api.pa_extend_sequences(s.tables, s.lens, s.counts, dev(starts.astype(np.int32)), slots, copies, left, 16, s.ws)
    s.same()
    assert left.tolist() == [int((counts == 0).sum()), 1] and bool((slots == -1).all()) and bool((copies == -1).all())
