"""Whole prompts in packed rows, and the sequences' blocks kept on the device, as measured cases.

Six operators beside the paged decode and prefill:

  prompt    causal attention over packed prompts of different lengths, whose keys and
            values are the new tokens' own rows; it writes them into the pools too
  extend    room for new tokens: blocks from the pool for each sequence, a private copy
            of a shared last block, and the tokens' slots
  truncate  cut sequences to a length, or free them: blocks return to the pool
  fork      a sequence becomes a copy of another one and shares its blocks
  copy      whole blocks in the pools of all layers (what extend and compact ask for)
  compact   moves of the highest used blocks into the lowest free ones, with the tables
            and counts as they are after them

A pool's block is free where its count of holders is 0; the lowest free ones are handed
out first, to the sequences in their order.  A pass over sequences brings them back to
where it found them, so that each pass does the same.

With ``own`` false, ``run`` computes them with elementary torch operations, in float32
where there are numbers to compute; with ``own`` true it calls the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # a short question to an idle server: latency
        {"name": "prompt-one", "op": "prompt", "seqs": 1, "min_len": 61, "max_len": 61, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "block": 16, "dtype": "fp16", "fused": False, "cache": True, "pad": 0},
        # an ordinary batch of prompts of one token to two thousand, q, k and v as views of one projection
        {"name": "prompts-ragged", "op": "prompt", "seqs": 16, "min_len": 1, "max_len": 2048, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "block": 16, "dtype": "bf16", "fused": True, "cache": True, "pad": 5},
        # eight equal prompts
        {"name": "prompts-equal", "op": "prompt", "seqs": 8, "min_len": 2048, "max_len": 2048, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "block": 16, "dtype": "fp16", "fused": False, "cache": True, "pad": 0},
        # a group that does not divide a tile of rows, small heads, scoring without a cache
        {"name": "prompts-group7", "op": "prompt", "seqs": 12, "min_len": 200, "max_len": 1500, "heads": 28, "kv_heads": 4,
         "head_dim": 64, "block": 32, "dtype": "bf16", "fused": True, "cache": False, "pad": 0},
        # two long documents
        {"name": "prompts-long", "op": "prompt", "seqs": 2, "min_len": 6000, "max_len": 8192, "heads": 64, "kv_heads": 8,
         "head_dim": 128, "block": 32, "dtype": "fp16", "fused": False, "cache": True, "pad": 0},
        # the bookkeeping of one step of a few short sequences: latency
        {"name": "step-few", "op": "step", "seqs": 8, "min_len": 20, "max_len": 500, "min_new": 1, "max_new": 1, "block": 16,
         "free": 0.5},
        # a step of a full server that takes back and makes room for five guessed tokens per sequence
        {"name": "step-guesses", "op": "step", "seqs": 256, "min_len": 100, "max_len": 16000, "min_new": 5, "max_new": 5,
         "block": 16, "free": 0.3},
        # 64 finished requests leave and 64 prompts come in
        {"name": "step-admit", "op": "step", "seqs": 64, "min_len": 0, "max_len": 0, "min_new": 1, "max_new": 2048,
         "block": 16, "free": 0.5},
        # four samples of one prompt, two layers
        {"name": "sample-one", "op": "sample", "prompts": 1, "samples": 4, "min_len": 700, "max_len": 700, "pools": 4,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "fp16"},
        # sixteen prompts sampled sixteen times each, sixteen layers
        {"name": "sample-many", "op": "sample", "prompts": 16, "samples": 16, "min_len": 100, "max_len": 1500, "pools": 32,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"},
        # a bounded number of moves between two steps
        {"name": "compact-some", "op": "compact", "seqs": 32, "blocks": 4096, "used": 0.5, "limit": 64, "pools": 32,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "fp16"},
        # a pool made dense at once, to give its rear half back
        {"name": "compact-all", "op": "compact", "seqs": 64, "blocks": 4096, "used": 0.6, "limit": 2048, "pools": 32,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: lengths from one token on, odd and ragged,
    every block size, head size, group and type."""
    op = rng.choice(["prompt", "prompt", "step", "sample", "compact"])
    block = rng.choice([16, 16, 32, 64, 128, 256])
    if op == "step":
        case = {"op": op, "seqs": _log(rng, 1, 512), "block": block, "free": rng.uniform(0.05, 1.0)}
        case["max_len"] = rng.choice([0, _log(rng, 1, 16000)])
        case["min_len"] = rng.randint(0, case["max_len"])
        case["max_new"] = _log(rng, 1, 2048) if case["max_len"] == 0 else _log(rng, 1, 16)
        case["min_new"] = rng.randint(0, case["max_new"])
        return case
    case = {"op": op, "kv_heads": rng.choice([1, 2, 4, 8]), "head_dim": rng.choice([64, 128]), "block": block,
            "dtype": rng.choice(["fp16", "bf16"])}
    if op == "prompt":
        case["heads"] = case["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        case["seqs"] = _log(rng, 1, 32)
        case["max_len"] = _log(rng, 1, 8192)
        while case["seqs"] * case["max_len"] ** 2 * case["heads"] * case["head_dim"] > 2 * 8192 ** 2 * 64 * 128 * 0.7:
            case["max_len"] -= case["max_len"] // 4
        case["min_len"] = rng.randint(1, case["max_len"])
        case["fused"], case["cache"], case["pad"] = rng.random() < 0.5, rng.random() < 0.7, rng.choice([0, 0, 1, 6])
        return case
    size = block * case["kv_heads"] * case["head_dim"] * 2  # bytes of a block in one pool
    case["pools"] = 2 * _log(rng, 1, 16)
    if op == "sample":
        case["prompts"], case["samples"] = _log(rng, 1, 16), _log(rng, 1, 16)
        case["max_len"] = _log(rng, 1, 1500)
        case["min_len"] = rng.randint(1, case["max_len"])
        while size * case["pools"] * case["prompts"] * (_blocks(case["max_len"], block) + 2 * case["samples"] + 2) > 2 ** 32:
            case["prompts"] = max(1, case["prompts"] // 2)
            case["pools"] = max(2, case["pools"] // 2)
        return case
    case["blocks"] = _log(rng, 20, 4096)
    while size * case["pools"] * case["blocks"] > 2 ** 32:
        case["blocks"] = max(20, case["blocks"] // 2)
        case["pools"] = max(2, case["pools"] // 2)
    case["used"] = rng.uniform(0.05, 0.95)
    case["seqs"] = max(1, min(_log(rng, 1, 64), int(case["blocks"] * case["used"])))
    case["limit"] = _log(rng, 1, case["blocks"])
    return case


# ------------------------------------------------------------------- sizes
def _blocks(n, block):
    return -(-n // block)


def _spread(n, lo, hi):
    """n whole numbers spread over [lo, hi] by the golden ratio."""
    return [lo + int((hi - lo + 1) * (((s + 1) * 0.6180339887498949) % 1.0)) for s in range(n)]


def _held(case):
    """Blocks of the sequences of a compact case: their shares of the used part of the pool."""
    total = max(case["seqs"], int(case["blocks"] * case["used"]))
    parts = _spread(case["seqs"], 1, 7)
    held = [max(1, total * p // sum(parts)) for p in parts]
    held[0] += max(0, total - sum(held))
    return held


def _block_bytes(case):
    return case["block"] * case["kv_heads"] * case["head_dim"] * 2


def work(case):
    block = case["block"]
    if case["op"] == "prompt":
        lens = _spread(case["seqs"], case["min_len"], case["max_len"])
        d, heads, kv, rows = case["head_dim"], case["heads"], case["kv_heads"], sum(lens)
        bytes_ = rows * d * 2 * (2 * heads + 2 * kv) + rows * (8 + kv * d * 4 if case["cache"] else 0)
        return {"bytes": bytes_, "flops": 4 * d * heads * sum(n * (n + 1) // 2 for n in lens)}
    if case["op"] == "step":
        # per sequence its lengths and starts; the given and the taken blocks' table entries and
        # counts twice each; the counts of the pool once; a slot per token
        lens, new = _step_lengths(case)
        turned = sum(_blocks(a + b, block) - _blocks(a, block) for a, b in zip(lens, new))
        return {"bytes": case["seqs"] * (4 * 5 + 16) + turned * 2 * (4 + 8) + 4 * _step_blocks(case) + 8 * sum(new), "flops": 0}
    if case["op"] == "sample":
        lens = _spread(case["prompts"], case["min_len"], case["max_len"])
        entries = sum(_blocks(n, block) for n in lens)
        own_blocks = case["prompts"] * case["samples"]
        copied = sum(case["samples"] for n in lens if n % block)
        return {"bytes": copied * 2 * case["pools"] * _block_bytes(case) + case["samples"] * entries * (4 * 3 + 8 * 2)
                + own_blocks * (16 + 8 + 5 * 4 + 2 * 12), "flops": 0}
    moved = min(case["limit"], int(case["blocks"] * case["used"] * (1 - case["used"])))
    return {"bytes": moved * (2 * case["pools"] * _block_bytes(case) + 16) + case["blocks"] * 4 * 2 + sum(_held(case)) * 4 * 2,
            "flops": 0}


def _step_lengths(case):
    new = _spread(case["seqs"] + 3, case["min_new"], case["max_new"])[3:]
    return _spread(case["seqs"], case["min_len"], case["max_len"]), new


def _step_blocks(case):
    lens, new = _step_lengths(case)
    need = sum(_blocks(a + b, case["block"]) for a, b in zip(lens, new))
    return need + _cached(need) + 8 + int(need * case["free"])


def _cached(need):
    """Blocks that a program holds without a sequence: finished prompts that may come again."""
    return need // 4 + 8


# ------------------------------------------------------------------- inputs
def _tables(counts, n, gen):
    """Tables over a shuffled pool of n blocks: [S, M] int32, -1 where unused."""
    perm = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    width = max(1, max(counts))
    count = torch.tensor(counts, device="cuda")
    col = torch.arange(width, device="cuda")[None, :].expand(len(counts), width)
    start = torch.cumsum(count, 0) - count
    at = (start[:, None] + col).clamp(max=n - 1)
    return torch.where(col < count[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()


def _counts_of(tables, n):
    ids = torch.where(tables >= 0, tables, torch.full_like(tables, n)).flatten().long()
    return torch.bincount(ids, minlength=n + 1)[:n].to(torch.int32)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(new):
    return torch.nn.functional.pad(torch.cumsum(_int32(new), 0), (1, 0)).to(torch.int32)


def _plan_rows(st, new):
    """Each new token's sequence and its place among that sequence's new tokens."""
    count = torch.tensor(new, device="cuda")
    st["row_seq"] = torch.repeat_interleave(torch.arange(len(new), device="cuda"), count)
    st["row_at"] = torch.arange(sum(new), device="cuda") - (torch.cumsum(count, 0) - count)[st["row_seq"]]


def _pools(case, n, gen):
    shape = (case["pools"], n, case["block"], case["kv_heads"], case["head_dim"])
    x = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda")
    return x.normal_(generator=gen)


def _prepare_prompt(case, gen):
    dt, heads, kv, d, block = DTYPES[case["dtype"]], case["heads"], case["kv_heads"], case["head_dim"], case["block"]
    lens = _spread(case["seqs"], case["min_len"], case["max_len"])
    rows = sum(lens) + case["pad"]  # padding rows stand behind the last sequence
    st = {"op": "prompt", "scale": 1.0 / math.sqrt(d), "longest": max(lens), "starts": _starts(lens), "kv_heads": kv}
    _plan_rows(st, lens)
    q = 0.7 * torch.randn((rows, heads, d), generator=gen, device="cuda")
    k = torch.randn((rows, kv, d), generator=gen, device="cuda")
    v = torch.randn((rows, kv, d), generator=gen, device="cuda")
    chan = torch.exp(0.5 * torch.randn((kv, d), generator=gen, device="cuda"))  # keys with a few strong channels
    chan[:, :: max(1, d // 4)] *= 4.0
    k *= chan
    v *= torch.exp(0.7 * torch.randn((rows, kv, 1), generator=gen, device="cuda"))
    if case["fused"]:
        qkv = torch.cat([q, k, v], dim=1).to(dt)
        st["q"], st["key"], st["value"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    else:
        st["q"], st["key"], st["value"] = q.to(dt), k.to(dt), v.to(dt)
    st["out"] = torch.zeros((rows, heads, d), dtype=dt, device="cuda")
    st["cached"] = case["cache"]
    if case["cache"]:
        counts = [_blocks(n, block) for n in lens]
        n = sum(counts) + sum(counts) // 8 + 1
        tables = _tables(counts, n, gen)
        slots = tables[st["row_seq"], st["row_at"] // block].long() * block + st["row_at"] % block
        st["slots"] = torch.nn.functional.pad(slots, (0, case["pad"]), value=-1)
        st["k"], st["v"] = (torch.zeros((n, block, kv, d), dtype=dt, device="cuda") for _ in range(2))
    return st


def _extend_buffers(st, new, n):
    """What a program keeps for its calls of extend."""
    st["starts"] = _starts(new)
    _plan_rows(st, new)
    st["slots"] = torch.empty(sum(new), dtype=torch.int64, device="cuda")
    st["copies"] = torch.empty((len(new), 2), dtype=torch.int64, device="cuda")
    st["left"] = torch.empty(2, dtype=torch.int32, device="cuda")
    st["space"] = torch.empty(_blocks(n, 4) * 4 + 16, dtype=torch.int32, device="cuda")
    st["most"] = max(_blocks(x, st["block"]) + 1 for x in new)  # blocks that one sequence can need


def _prepare_step(case, gen):
    block = case["block"]
    lens, new = _step_lengths(case)
    n = _step_blocks(case)
    now = [a + b for a, b in zip(lens, new)]
    had = [_blocks(m, block) for m in now]
    both = _tables(had + [1] * _cached(sum(had)), n, gen)
    tables, cached = both[:len(had)].contiguous(), both[len(had):, 0]
    # every second sequence shares the blocks of its left neighbour's prompt
    share = [min(a, b) // block // 2 for a, b in zip(lens, lens[1:] + [0])]
    col = torch.arange(tables.shape[1], device="cuda")
    some = _int32([share[s - 1] if s % 2 else 0 for s in range(len(lens))])
    left = torch.cat([tables[:1], tables[:-1]])
    tables = torch.where(col < some[:, None], left, tables).contiguous()
    st = {"op": "step", "block": block, "tables": tables, "lens": _int32(now),
          "counts": _counts_of(tables, n) + _counts_of(cached, n), "keep": _int32(lens)}
    _extend_buffers(st, new, n)
    return st


def _prepare_sample(case, gen):
    block, prompts, samples = case["block"], case["prompts"], case["samples"]
    lens = _spread(prompts, case["min_len"], case["max_len"])
    seqs = prompts * (1 + samples)
    of = [-1] * prompts + [s // samples for s in range(prompts * samples)]
    had = [_blocks(m, block) for m in lens]
    width = max(had) + 1
    # the prompts, and the last round's samples, of one token more than their prompt
    n = sum(had) + 2 * prompts * samples + 2
    own_blocks = _tables(had + [1] * (prompts * samples), n, gen)
    tables = torch.nn.functional.pad(own_blocks, (0, width - own_blocks.shape[1]), value=-1)
    src = _int32(of).long()
    length = _int32(lens + [lens[p] + 1 for p in of[prompts:]])
    whole = (_int32(lens) // block)[src.clamp(min=0)]
    col = torch.arange(width, device="cuda")
    is_sample = (src >= 0)[:, None]
    shared = torch.where(col < whole[:, None], tables[src.clamp(min=0)], torch.full_like(tables, -1))
    shared = torch.where(col == whole[:, None], tables[:, :1], shared)
    tables = torch.where(is_sample, shared, tables).contiguous()
    st = {"op": "sample", "block": block, "tables": tables, "lens": length, "counts": _counts_of(tables, n),
          "from": _int32(of), "keep": _int32([-1] * prompts + [0] * (prompts * samples)), "pools": _pools(case, n, gen)}
    _extend_buffers(st, [0] * prompts + [1] * (prompts * samples), n)
    assert len(of) == seqs
    return st


def _prepare_compact(case, gen):
    block, n = case["block"], case["blocks"]
    held = _held(case)
    tables = _tables(held, n, gen)
    lens = _int32([h * block - (3 * s) % block for s, h in enumerate(held)])
    return {"op": "compact", "block": block, "tables": tables, "lens": lens, "counts": _counts_of(tables, n),
            "moves": torch.empty((case["limit"], 2), dtype=torch.int64, device="cuda"),
            "num": torch.empty(1, dtype=torch.int32, device="cuda"), "new_tables": torch.empty_like(tables),
            "new_counts": torch.empty(n, dtype=torch.int32, device="cuda"), "pools": _pools(case, n, gen),
            "space": torch.empty(_blocks(n, 4) * 4 + 16, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"prompt": _prepare_prompt, "step": _prepare_step, "sample": _prepare_sample,
            "compact": _prepare_compact}[case["op"]](case, gen)


# ------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return {"prompt": _prompt, "step": _step, "sample": _sample, "compact": _compact}[st["op"]](st)


def _run_own(st):
    from paged_kv_cache_173_gb300 import api
    op = st["op"]
    if op == "prompt":
        if st["cached"]:
            api.pa_prefill_packed(st["out"], st["q"], st["key"], st["value"], st["starts"], st["longest"], st["scale"],
                                  st["k"], st["v"], st["slots"])
            return st["out"], st["k"], st["v"]
        api.pa_prefill_packed(st["out"], st["q"], st["key"], st["value"], st["starts"], st["longest"], st["scale"])
        return st["out"]
    if op == "compact":
        api.pa_compact_blocks(st["moves"], st["num"], st["tables"], st["lens"], st["counts"], st["new_tables"],
                              st["new_counts"], st["block"], st["space"])
        api.pa_copy_layer_blocks(st["pools"], st["moves"])
        return st["moves"], st["num"], st["new_tables"], st["new_counts"], st["pools"]
    api.pa_truncate_sequences(st["tables"], st["lens"], st["counts"], st["keep"], st["block"])
    if op == "sample":
        api.pa_fork_sequences(st["tables"], st["lens"], st["counts"], st["from"], st["block"])
    api.pa_extend_sequences(st["tables"], st["lens"], st["counts"], st["starts"], st["slots"], st["copies"], st["left"],
                            st["block"], st["space"])
    if op == "sample":
        api.pa_copy_layer_blocks(st["pools"], st["copies"])
    return _sequences(st)


def _sequences(st):
    got = [st["tables"], st["lens"], st["counts"], st["slots"], st["copies"], st["left"]]
    return got + [st["pools"]] if st["op"] == "sample" else got


def _prompt(st):
    seq, at, length = st["row_seq"], st["row_at"], st["longest"]
    rows = len(seq)
    seqs, kv, (_, heads, d) = len(st["starts"]) - 1, st["kv_heads"], st["q"].shape

    def padded(x):
        y = torch.zeros((seqs, length) + tuple(x.shape[1:]), device="cuda")
        y[seq, at] = x[:rows].float()
        return y

    q = padded(st["q"]).view(seqs, length, kv, heads // kv, d).permute(0, 2, 3, 1, 4)
    k = padded(st["key"]).permute(0, 2, 3, 1)[:, :, None]
    v = padded(st["value"]).permute(0, 2, 1, 3)[:, :, None]
    s = torch.matmul(q, k) * st["scale"]
    pos = torch.arange(length, device="cuda")
    s = s.masked_fill(pos[None, :] > pos[:, None], -math.inf)
    p = torch.exp(s - s.amax(dim=-1, keepdim=True))
    del s
    o = torch.matmul(p, v) / p.sum(dim=-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, length, heads, d)
    st["out"][:rows] = o[seq, at].to(st["out"].dtype)
    if not st["cached"]:
        return st["out"]
    slots = st["slots"][:rows]
    st["k"].flatten(0, 1)[slots] = st["key"][:rows]
    st["v"].flatten(0, 1)[slots] = st["value"][:rows]
    return st["out"], st["k"], st["v"]


def _up(x, block):
    return (x + block - 1) // block


def _add_counts(counts, ids, on, by):
    """counts[id] += by for the table entries where `on` holds."""
    n = len(counts)
    change = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    change.index_add_(0, torch.where(on, ids, torch.full_like(ids, n)).flatten().long(), on.flatten().to(torch.int32))
    counts += by * change[:n]


def _truncate(st):
    tables, lens, block = st["tables"], st["lens"], st["block"]
    to = torch.where((st["keep"] >= 0) & (st["keep"] < lens), st["keep"], lens)
    col = torch.arange(tables.shape[1], device="cuda")
    out = (col >= _up(to, block)[:, None]) & (col < _up(lens, block)[:, None])
    _add_counts(st["counts"], tables, out, -1)
    tables.masked_fill_(out, -1)
    lens.copy_(to)


def _fork(st):
    tables, lens, src = st["tables"], st["lens"], st["from"]
    at = src.clamp(min=0).long()
    go = (src >= 0) & (src[at] < 0) & (lens == 0)
    col = torch.arange(tables.shape[1], device="cuda")
    on = go[:, None] & (col < _up(lens[at], st["block"])[:, None])
    ids = tables[at]
    _add_counts(st["counts"], ids, on, 1)
    tables.copy_(torch.where(on, ids, tables))
    lens.copy_(torch.where(go, lens[at], lens))


def _extend(st):
    tables, lens, counts, block = st["tables"], st["lens"], st["counts"], st["block"]
    seqs, width = tables.shape
    n = len(counts)
    new = st["starts"][1:] - st["starts"][:-1]
    had, want = _up(lens, block), _up(lens + new, block)
    row = torch.arange(seqs, device="cuda")
    last_at = (had - 1).clamp(min=0).long()
    last = tables[row, last_at].long()
    copy = (new > 0) & (lens % block != 0) & (counts[last.clamp(min=0)] > 1)
    fits = lens + new <= width * block
    need = torch.where((new > 0) & fits, want - had + copy.to(torch.int32), torch.zeros_like(new)).long()
    upto = torch.cumsum(need, 0)
    free = counts == 0
    total = free.sum()
    ok = fits & ((need == 0) | (upto <= total))
    need = torch.where(ok, need, torch.zeros_like(need))
    copy &= ok
    # the free blocks in order, and each sequence's among them
    rank = torch.cumsum(free, 0) - 1
    ids = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    ids[torch.where(free, rank, torch.full_like(rank, n))] = torch.arange(n, device="cuda")
    turn = torch.arange(st["most"], device="cuda")
    given = turn[None, :] < need[:, None]
    got = ids[((upto - need)[:, None] + turn).clamp(0, n)]
    # where each goes: the copy takes the last place, the others follow
    place = had[:, None].long() - copy[:, None].long() + turn
    wide = torch.nn.functional.pad(tables, (0, 1))
    wide[row[:, None].expand_as(place), torch.where(given, place, torch.full_like(place, width)).clamp(max=width)] = got.to(torch.int32)
    tables.copy_(wide[:, :width])
    _add_counts(counts, got, given, 1)
    _add_counts(counts, last, copy, -1)
    pair = torch.stack([last, got[:, 0]], dim=1)
    st["copies"].copy_(torch.where(copy[:, None], pair, torch.full_like(pair, -1)))
    pos = lens.long()[st["row_seq"]] + st["row_at"]
    slot = tables[st["row_seq"], (pos // block).clamp(max=width - 1)].long() * block + pos % block
    st["slots"].copy_(torch.where(ok[st["row_seq"]], slot, torch.full_like(slot, -1)))
    lens.copy_(torch.where(ok & (new > 0), lens + new, lens))
    st["left"].copy_(torch.stack([total - need.sum(), ((new > 0) & ~ok).sum()]))


def _copy(pools, pairs):
    """pools[:, dst] = pools[:, src] for the pairs that name blocks; others repeat the first of those."""
    on = pairs[:, 0] >= 0
    first = on.to(torch.int32).argmax()
    at = torch.where(on, torch.arange(len(pairs), device="cuda"), first)
    pools[:, pairs[at, 1]] = pools[:, pairs[at, 0]]


def _step(st):
    _truncate(st)
    _extend(st)
    return _sequences(st)


def _sample(st):
    _truncate(st)
    _fork(st)
    _extend(st)
    _copy(st["pools"], st["copies"])
    return _sequences(st)


def _compact(st):
    counts, limit = st["counts"], len(st["moves"])
    n = len(counts)
    used = counts != 0
    ids = torch.arange(n, device="cuda")
    low = torch.cumsum(~used, 0) - 1                # a free block's place from the bottom
    high = torch.cumsum(used.flip(0), 0).flip(0) - 1  # a used block's place from the top
    num = (~used & (ids < used.sum())).sum().clamp(max=limit)
    to, away = ~used & (low < num), used & (high < num)
    moves = torch.full((limit + 1, 2), -1, dtype=torch.int64, device="cuda")
    moves[torch.where(away, high, torch.full_like(high, limit)), 0] = ids
    moves[torch.where(to, low, torch.full_like(low, limit)), 1] = ids
    st["moves"].copy_(moves[:limit])
    st["num"].copy_(num.view(1))
    where = torch.where(away, moves[high.clamp(max=limit), 1], ids)  # each block's place after the moves
    st["new_tables"].copy_(torch.where(st["tables"] >= 0, where[st["tables"].clamp(min=0).long()].to(torch.int32), st["tables"]))
    old = torch.where(to, moves[low.clamp(0, limit), 0], ids)        # whose count a block has after them
    st["new_counts"].copy_(torch.where(away, torch.zeros_like(counts), counts[old]))
    _copy(st["pools"], st["moves"])
    return st["moves"], st["num"], st["new_tables"], st["new_counts"], st["pools"]


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The attention of a prompt case by sequence and head in float64; the pools take rows as they are, and
    the other operators compute whole numbers only."""
    if case["op"] != "prompt" or case["seqs"] * case["max_len"] ** 2 * case["heads"] * case["head_dim"] > 1.3e12:
        return None
    st = prepare(case, seed)
    begin = [int(x) for x in st["starts"]]
    heads, kv = st["q"].shape[1], st["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for a, b in zip(begin, begin[1:]):
        hidden = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").triu(1)
        for h in range(heads):
            g = h // (heads // kv)
            w = (st["q"][a:b, h].double() @ st["key"][a:b, g].double().T).mul_(st["scale"]).masked_fill_(hidden, -math.inf)
            out[a:b, h] = torch.softmax(w, -1) @ st["value"][a:b, g].double()
    return [out, None, None] if st["cached"] else out
