"""The block-scaled E4M3 cache and block-sparse decode, as measured cases.

Five operators over paged pools [N, B, Hk, d]:

  write    new tokens into E4M3 pools that hold one scale per (block, KV head)
  decode   attention of one token per sequence over such pools
  prefill  causal attention of prompts, or chunks of them, over such pools
  bounds   per-channel bounds of the keys of each (block, KV head), kept in 8 bits
  sparse   a decode step that scores the blocks by their bounds, keeps the best
           and attends to those alone

With ``own`` false, ``run`` computes them with elementary torch operations in
float32; with ``own`` true it calls the package's entry points.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE_EXP = -64
BOUND_MAX = 127
MIN_BOUND_EXP = -100
QUERY_MAX = 255
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the cache write of one decode step: a token per sequence, blocks partly filled
        {"name": "write-append", "op": "write", "mode": "append", "seqs": 64, "min_len": 128, "max_len": 2048,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "fp16"},
        # the cache write of a prefill step: eight whole prompts
        {"name": "write-prompts", "op": "write", "mode": "prompt", "seqs": 8, "min_len": 2048, "max_len": 2048,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"},
        # one short chat sequence, where the latency of the call counts
        {"name": "decode-one", "op": "decode", "seqs": 1, "min_len": 300, "max_len": 500, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "block": 16, "dtype": "fp16", "part": 0},
        # an ordinary serving batch of ragged contexts
        {"name": "decode-batch", "op": "decode", "seqs": 64, "min_len": 128, "max_len": 2048, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "fp16", "part": 0},
        # wide query groups at a long fixed context, bfloat16
        {"name": "decode-gqa8", "op": "decode", "seqs": 32, "min_len": 8192, "max_len": 8192, "heads": 64,
         "kv_heads": 8, "head_dim": 128, "block": 32, "dtype": "bf16", "part": 0},
        # few very long sequences, split over partitions
        {"name": "decode-long", "op": "decode", "seqs": 4, "min_len": 32768, "max_len": 131072, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "fp16", "part": 512},
        # whole prompts
        {"name": "prefill-prompts", "op": "prefill", "seqs": 8, "new": 2048, "cached": 0, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "block": 16, "dtype": "fp16"},
        # chunks of prompts on top of a cached context, ragged, bfloat16
        {"name": "prefill-chunks", "op": "prefill", "seqs": 16, "new": 509, "cached": 1536, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 64, "dtype": "bf16"},
        # the bounds' part of the cache write of one decode step
        {"name": "bounds-append", "op": "bounds", "mode": "append", "seqs": 64, "min_len": 128, "max_len": 2048,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "fp16"},
        # and of a prefill step
        {"name": "bounds-prompts", "op": "bounds", "mode": "prompt", "seqs": 8, "min_len": 2048, "max_len": 2048,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16"},
        # long contexts of which each token reads 2048 positions, 16-bit pools
        {"name": "sparse-long", "op": "sparse", "seqs": 4, "min_len": 32768, "max_len": 131072, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "fp16", "keep": 128, "first": 1, "last": 4,
         "pool": "16"},
        # a serving batch of middling contexts over block-scaled pools
        {"name": "sparse-batch", "op": "sparse", "seqs": 16, "min_len": 4000, "max_len": 32768, "heads": 64,
         "kv_heads": 8, "head_dim": 128, "block": 32, "dtype": "bf16", "keep": 96, "first": 2, "last": 2,
         "pool": "fp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: lengths from one token on, odd and
    ragged, every block size, head size, group and type."""
    op = rng.choice(["write", "decode", "decode", "prefill", "bounds", "sparse"])
    dim = rng.choice([64, 128, 128, 256]) if op != "prefill" else rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8] if dim == 256 else [1, 2, 4, 8, 16])
    case = {"op": op, "kv_heads": kv, "head_dim": dim, "block": rng.choice([16, 16, 32, 64, 128, 256]),
            "dtype": rng.choice(["fp16", "bf16"])}
    if op in ("write", "bounds"):
        case["mode"] = rng.choice(["append", "prompt"])
        case["seqs"] = _log(rng, 1, 192) if case["mode"] == "append" else _log(rng, 1, 8)
        case["max_len"] = _log(rng, 1, 2048)
        case["min_len"] = rng.randint(1, case["max_len"])
    elif op == "prefill":
        case["heads"] = kv * group
        case["seqs"] = _log(rng, 1, 8)
        case["new"] = _log(rng, 1, 2048)
        case["cached"] = rng.choice([0, _log(rng, 1, 2048)])
        while case["seqs"] * case["new"] * (case["new"] + 2 * case["cached"]) * case["heads"] * dim > 8 * 2048 ** 2 * 4096:
            case["new"] = max(1, case["new"] // 2)
            case["cached"] //= 2
    else:
        case["heads"] = kv * group
        case["seqs"] = _log(rng, 1, 64)
        case["max_len"] = _log(rng, 1, 65536)
        while case["seqs"] * case["max_len"] * kv * dim > 32 * 8192 * 1024:
            case["seqs"] = max(1, case["seqs"] // 2)
            case["max_len"] = max(1, case["max_len"] - case["max_len"] // 4)
        case["min_len"] = rng.randint(1, case["max_len"])
        if op == "decode":
            case["part"] = rng.choice([0, 512, 1024])
        else:
            case["keep"] = _log(rng, 4, 256)
            case["first"] = rng.randint(0, 2)
            case["last"] = rng.randint(1, 2)
            case["pool"] = rng.choice(["16", "fp8"])
    return case


# ------------------------------------------------------------------- sizes
def _lengths(case):
    """The sequences' lengths: spread over [min_len, max_len] by the golden ratio."""
    if case["op"] == "prefill":  # the chunks differ by a few tokens
        return [case["cached"] + n for n in _new_lengths(case)]
    lo, hi = case["min_len"], case["max_len"]
    return [lo + int((hi - lo + 1) * (((s + 1) * 0.6180339887498949) % 1.0)) for s in range(case["seqs"])]


def _new_lengths(case):
    return [max(1, case["new"] - (s % 3 if case["new"] % 2 else 0)) for s in range(case["seqs"])]


def _blocks(n, block):
    return -(-n // block)


def work(case):
    kv, d, block = case["kv_heads"], case["head_dim"], case["block"]
    lens = _lengths(case)
    if case["op"] in ("write", "bounds"):
        tokens = len(lens) if case["mode"] == "append" else sum(lens)
        blocks = len(lens) if case["mode"] == "append" else sum(_blocks(n, block) for n in lens)
        if case["op"] == "write":
            return {"bytes": tokens * (kv * d * 2 * (2 + 1) + 8) + blocks * kv * 2 * 4 * 2, "flops": 4 * tokens * kv * d}
        return {"bytes": tokens * (kv * d * 2 + 8) + blocks * kv * (2 * d + 4) * (2 if case["mode"] == "append" else 1),
                "flops": 4 * tokens * kv * d}
    heads, nblk = case["heads"], sum(_blocks(n, block) for n in lens)
    if case["op"] == "decode":
        return {"bytes": sum(lens) * kv * 2 * d + nblk * (kv * 8 + 4) + len(lens) * heads * d * 4,
                "flops": 4 * d * heads * sum(lens)}
    if case["op"] == "prefill":
        new = _new_lengths(case)
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for c, n in zip(lens, new))
        return {"bytes": sum(lens) * kv * 2 * d + nblk * (kv * 8 + 4) + sum(new) * heads * d * 4,
                "flops": 4 * d * heads * pairs}
    kept = sum(min(_blocks(n, block), case["keep"]) for n in lens)
    tokens = sum(min(n, case["keep"] * block) for n in lens)
    wide = 2 if case["pool"] == "16" else 1
    return {"bytes": nblk * (kv * (2 * d + 4) + 4) + kept * kv * (8 + (8 if wide == 1 else 0))
            + tokens * kv * 2 * d * wide + len(lens) * heads * d * 4,
            "flops": 2 * d * heads * nblk + 4 * d * heads * tokens}


# ------------------------------------------------------------------- inputs
def _pow2(e):
    """2**e as float32, for an integer tensor e in [-126, 127]."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _exp_for(amax, top_mantissa, top_exp, floor):
    """The smallest e >= floor with amax <= top * 2**e, where top = top_mantissa * 2**top_exp (mantissa in [0.5, 1))."""
    m, x = torch.frexp(amax)
    e = x - top_exp + (m > top_mantissa).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, floor)).clamp(min=floor)


def _to_codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scale_for(amax):
    return _pow2(_exp_for(amax, 0.875, 9, MIN_SCALE_EXP))  # 448 = 0.875 * 2**9


def _pool(shape, gen, dtype, kind):
    """Values of one pool: keys with a few strong channels, values whose size changes from block to block."""
    n, block, kv, d = shape
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if kind == "k":
        chan = torch.exp(0.5 * torch.randn((kv, d), generator=gen, device="cuda"))
        chan[:, :: max(1, d // 4)] *= 4.0
        x *= chan
    else:
        x *= torch.exp(0.7 * torch.randn((n, 1, kv, 1), generator=gen, device="cuda"))
    return x.to(dtype)


def _coded(x):
    scale = _scale_for(x.abs().amax(dim=(1, 3)).float())
    return _to_codes(x.float() / scale[:, None, :, None]), scale


def _tables(lens, block, gen):
    """Block tables over a shuffled pool: [S, M] int32, -1 where unused; and the pool's number of blocks."""
    counts = [_blocks(n, block) for n in lens]
    total = sum(counts)
    n = total + total // 8 + 1
    perm = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    width = max(counts)
    count = torch.tensor(counts, device="cuda")
    col = torch.arange(width, device="cuda")[None, :].expand(len(lens), width)
    start = torch.cumsum(count, 0) - count
    at = (start[:, None] + col).clamp(max=n - 1)
    return torch.where(col < count[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous(), n


def _bounds_of(x):
    """Bounds of whole blocks of keys x [n, B, Hk, d]: codes [n, Hk, 2, d] and exponents [n, Hk]."""
    lo, hi = x.amin(dim=1).float(), x.amax(dim=1).float()
    e = _exp_for(torch.maximum(-lo, hi).amax(dim=-1), 127 / 128, 7, MIN_BOUND_EXP)
    inv = _pow2(-e)[..., None]
    codes = torch.stack([torch.floor(lo * inv), torch.ceil(hi * inv)], dim=2)
    return codes.clamp(-BOUND_MAX, BOUND_MAX).to(torch.int8), e.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    kv, d, block, seqs = case["kv_heads"], case["head_dim"], case["block"], case["seqs"]
    lens = _lengths(case)
    tables, n = _tables(lens, block, gen)
    st = {"op": case["op"], "block": block, "scale": 1.0 / math.sqrt(d), "tables": tables,
          "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    keys = _pool((n, block, kv, d), gen, dt, "k")
    if case["op"] in ("write", "bounds"):
        if case["mode"] == "append":  # each sequence's newest position
            seq = torch.arange(seqs, device="cuda")
            pos = st["lens"].long() - 1
        else:
            seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), st["lens"].long())
            pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
        st["slots"] = tables[seq, pos // block].long() * block + pos % block
        # the step's plan: the blocks it touches, and the place of each token's block among them
        st["touched"], st["place"] = torch.unique(st["slots"] // block, return_inverse=True)
        st["key"] = _pool((1, len(pos), kv, d), gen, dt, "k")[0].contiguous()
        if case["op"] == "bounds":
            st["bounds"], st["exps"] = _bounds_of(keys)
            return st
        st["value"] = _pool((1, len(pos), kv, d), gen, dt, "v")[0].contiguous()
    if case["op"] == "sparse":
        st["bounds"], st["exps"] = _bounds_of(keys)
        st["keep"], st["first"], st["last"] = case["keep"], case["first"], case["last"]
        st["select_space"] = torch.empty(seqs * kv * _blocks(tables.shape[1], 4) * 4, dtype=torch.float32, device="cuda")
        st["sel_tables"] = torch.empty((seqs, kv, case["keep"]), dtype=torch.int32, device="cuda")
        st["sel_lens"] = torch.empty((seqs, kv), dtype=torch.int32, device="cuda")
    values = _pool((n, block, kv, d), gen, dt, "v")
    if case.get("pool") == "16":
        st["k"], st["v"], st["ks"], st["vs"] = keys, values, None, None
    else:
        (st["k"], st["ks"]), (st["v"], st["vs"]) = _coded(keys), _coded(values)
    if case["op"] == "write":
        return st
    rows = seqs
    if case["op"] == "prefill":
        new = _new_lengths(case)
        rows, st["max_new"] = sum(new), max(new)
        st["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        starts = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
        starts[1:] = torch.cumsum(st["new"], 0)
        st["starts"] = starts
        # the step's plan: each row's sequence and its place in that sequence's chunk
        st["row_seq"] = torch.repeat_interleave(torch.arange(seqs, device="cuda"), st["new"].long())
        st["row_at"] = torch.arange(rows, device="cuda") - starts.long()[st["row_seq"]]
    # queries that lean towards some of the keys, so that the weights are not flat
    q = torch.randn((rows, case["heads"], d), generator=gen, device="cuda")
    st["q"] = (q * 0.7).to(dt)
    st["out"] = torch.empty_like(st["q"])
    if case["op"] == "decode":
        st["part"] = case["part"]
        if case["part"]:
            parts = _blocks(tables.shape[1] * block, _part(case["part"], block))
            st["space"] = torch.empty(seqs * case["heads"] * parts * (d + 2), dtype=torch.float32, device="cuda")
            st["part"] = _part(case["part"], block)
    return st


def _part(part, block):
    return max(part, block)


# ------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return {"write": _write, "bounds": _bounds, "decode": _decode, "prefill": _prefill, "sparse": _sparse}[st["op"]](st)


def _run_own(st):
    from paged_kv_cache_173_gb300 import api
    op = st["op"]
    if op == "write":
        api.pa_reshape_and_cache_fp8_block(st["key"], st["value"], st["k"], st["v"], st["ks"], st["vs"], st["slots"])
        return st["k"], st["v"], st["ks"], st["vs"]
    if op == "bounds":
        api.pa_update_key_bounds(st["key"], st["bounds"], st["exps"], st["slots"], st["block"])
        return st["bounds"], st["exps"]
    if op == "prefill":
        api.pa_prefill_fp8_block(st["out"], st["q"], st["k"], st["v"], st["ks"], st["vs"], st["tables"], st["lens"],
                                 st["starts"], st["max_new"], st["scale"])
        return st["out"]
    if op == "sparse":
        api.pa_select_blocks(st["sel_tables"], st["sel_lens"], st["q"], st["bounds"], st["exps"], st["tables"], st["lens"],
                             st["block"], st["first"], st["last"], st["select_space"])
        api.pa_decode_sparse(st["out"], st["q"], st["k"], st["v"], st["sel_tables"], st["sel_lens"], st["scale"],
                             st["ks"], st["vs"])
        return st["sel_tables"], st["sel_lens"], st["out"]
    if st["part"]:
        api.pa_decode_splitk_fp8_block(st["out"], st["q"], st["k"], st["v"], st["ks"], st["vs"], st["tables"], st["lens"],
                                       st["scale"], st["part"], st["space"])
        api.pa_splitk_reduce(st["out"], st["space"], st["lens"], st["tables"].shape[1], st["block"], st["part"])
    else:
        api.pa_decode_fp8_block(st["out"], st["q"], st["k"], st["v"], st["ks"], st["vs"], st["tables"], st["lens"],
                                st["scale"])
    return st["out"]


def _finite_amax(x):
    a = x.float().abs()
    return torch.where(torch.isfinite(a), a, torch.zeros_like(a))


def _write(st):
    block, at = st["block"], st["slots"] % st["block"]
    touched, place = st["touched"], st["place"]
    fresh = torch.zeros(len(touched), device="cuda").index_add_(0, place, (at == 0).float()) > 0
    for new, codes, scales in ((st["key"], st["k"], st["ks"]), (st["value"], st["v"], st["vs"])):
        amax = _finite_amax(new).amax(dim=-1)
        top = torch.zeros((len(touched), amax.shape[1]), device="cuda").index_reduce_(0, place, amax, "amax")
        old = torch.where(fresh[:, None], torch.zeros((), device="cuda"), scales[touched])
        s = torch.maximum(old, _scale_for(top))
        ratio = torch.where(old > 0, old / s, torch.ones((), device="cuda"))
        bytes_ = codes.view(torch.uint8)
        was = bytes_[touched].view(torch.float8_e4m3fn).float()
        bytes_[touched] = _to_codes(was * ratio[:, None, :, None]).view(torch.uint8)
        bytes_[touched[place], at] = _to_codes(new.float() / s[place][..., None]).view(torch.uint8)
        scales[touched] = s
    return st["k"], st["v"], st["ks"], st["vs"]


def _bounds(st):
    at, touched, place = st["slots"] % st["block"], st["touched"], st["place"]
    x = st["key"].float()
    fresh = torch.zeros(len(touched), device="cuda").index_add_(0, place, (at == 0).float()) > 0
    shape = (len(touched),) + tuple(x.shape[1:])
    lo = torch.full(shape, math.inf, device="cuda").index_reduce_(0, place, x, "amin")
    hi = torch.full(shape, -math.inf, device="cuda").index_reduce_(0, place, x, "amax")
    need = _exp_for(torch.maximum(-lo, hi).amax(dim=-1), 127 / 128, 7, MIN_BOUND_EXP)
    old_e = torch.where(fresh[:, None], torch.full_like(need, MIN_BOUND_EXP), st["exps"][touched])
    e = torch.maximum(need, old_e)
    inv, shift = _pow2(-e)[..., None], _pow2((old_e - e).clamp(min=-126))[..., None]
    old = st["bounds"][touched].float()
    new_lo = torch.floor(lo * inv).clamp(-BOUND_MAX, BOUND_MAX)
    new_hi = torch.ceil(hi * inv).clamp(-BOUND_MAX, BOUND_MAX)
    keep = fresh[:, None, None]
    lo = torch.where(keep, new_lo, torch.minimum(new_lo, torch.floor(old[:, :, 0] * shift)))
    hi = torch.where(keep, new_hi, torch.maximum(new_hi, torch.ceil(old[:, :, 1] * shift)))
    st["bounds"][touched] = torch.stack([lo, hi], dim=2).to(torch.int8)
    st["exps"][touched] = e.to(torch.int32)
    return st["bounds"], st["exps"]


def _rows(pool, scales, tables):
    """The pool's rows along each table: [..., M * B, Hk, d] float32."""
    at = tables.clamp(min=0).long()
    if scales is None:
        x = pool[at].float()
    else:
        x = pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scales[at][..., None, :, None]
    return x.flatten(1, 2)


def _softmax(s, seen):
    s = torch.where(seen, s, torch.full((), -math.inf, device="cuda"))
    p = torch.exp(s - s.amax(dim=-1, keepdim=True))
    return p / p.sum(dim=-1, keepdim=True)


def _attend(q, k, v, seen, scale):
    """q [S, Hk, R, d], k and v [S, L, Hk, d], seen broadcast to [S, Hk, R, L]."""
    w = _softmax(torch.matmul(q, k.permute(0, 2, 3, 1)) * scale, seen)
    return torch.matmul(w, v.permute(0, 2, 1, 3))


def _decode(st):
    k, v = _rows(st["k"], st["ks"], st["tables"]), _rows(st["v"], st["vs"], st["tables"])
    seqs, length, kv, d = k.shape
    seen = (torch.arange(length, device="cuda")[None, :] < st["lens"][:, None])[:, None, None, :]
    o = _attend(st["q"].float().view(seqs, kv, -1, d), k, v, seen, st["scale"])
    return o.reshape(st["q"].shape).to(st["q"].dtype)


def _prefill(st):
    k, v = _rows(st["k"], st["ks"], st["tables"]), _rows(st["v"], st["vs"], st["tables"])
    seqs, length, kv, d = k.shape
    new, heads = st["max_new"], st["q"].shape[1]
    q = torch.zeros((seqs, new, heads, d), device="cuda")
    q[st["row_seq"], st["row_at"]] = st["q"].float()
    q = q.view(seqs, new, kv, heads // kv, d).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, d)
    last = (st["lens"] - st["new"])[:, None] + torch.arange(new, device="cuda")[None, :]  # each row's own position
    seen = torch.arange(length, device="cuda")[None, None, :] <= last[:, :, None]
    seen = seen[:, None, None].expand(seqs, 1, heads // kv, new, length).reshape(seqs, 1, -1, length)
    o = _attend(q, k, v, seen, st["scale"])
    o = o.view(seqs, kv, heads // kv, new, d).permute(0, 3, 1, 2, 4).reshape(seqs, new, heads, d)
    return o[st["row_seq"], st["row_at"]].to(st["q"].dtype)


def _sparse(st):
    tables, lens, block, keep = st["tables"], st["lens"], st["block"], st["keep"]
    seqs, width = tables.shape
    q = st["q"].float()
    kv, d = st["bounds"].shape[1], q.shape[-1]
    # whole-number queries per head, and the bound of each block's products with them
    f = _exp_for(_finite_amax(q).amax(dim=-1), 255 / 256, 8, MIN_BOUND_EXP)
    qi = torch.round(q * _pow2(-f)[..., None]).view(seqs, kv, -1, d)
    at = tables.clamp(min=0).long()
    b = st["bounds"][at].float().permute(0, 2, 3, 4, 1)  # [S, Hk, 2, d, M]
    whole = torch.matmul(qi.clamp(max=0), b[:, :, 0]) + torch.matmul(qi.clamp(min=0), b[:, :, 1])
    e = st["exps"][at].permute(0, 2, 1)[:, :, None, :] + f.view(seqs, kv, -1, 1)
    score = (whole * _pow2(e.clamp(-100, 100))).amax(dim=2)  # [S, Hk, M]
    # the first and the last blocks always, then the best; ties go to the earlier block
    count = ((lens + block - 1) // block)[:, None]
    at = torch.arange(width, device="cuda")[None, :]
    always = ((at < st["first"]) | (at >= count - st["last"])) & (at < count)
    score = torch.where(always[:, None], torch.full((), math.inf, device="cuda"), score)
    score = torch.where((at < count)[:, None], score, torch.full((), -math.inf, device="cuda"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = torch.nn.functional.pad(order, (0, max(0, keep - width)), value=width)[..., :keep]
    order = torch.where(order < count[:, None], order, torch.full_like(order, width)).sort(dim=-1).values
    taken = order < width
    ids = torch.gather(tables[:, None].expand(seqs, kv, width), 2, order.clamp(max=width - 1))
    ids = torch.where(taken, ids, torch.full_like(ids, -1))
    used = taken.sum(dim=-1)
    sel_lens = (lens[:, None] - (count - used) * block).to(torch.int32)
    # attention over the kept blocks, each KV head with its own
    head = torch.arange(kv, device="cuda")[None, :, None]
    where = ids.clamp(min=0).long()

    def rows(pool, scales):
        if scales is None:
            x = pool[where, :, head].float()
        else:
            x = pool.view(torch.uint8)[where, :, head].view(torch.float8_e4m3fn).float() * scales[where, head][..., None, None]
        return x.flatten(2, 3).transpose(1, 2)  # [S, keep * B, Hk, d]

    seen = (torch.arange(keep * block, device="cuda") < sel_lens[..., None])[:, :, None, :]
    o = _attend(q.view(seqs, kv, -1, d), rows(st["k"], st["ks"]), rows(st["v"], st["vs"]), seen, st["scale"])
    return ids.to(torch.int32), sel_lens, o.reshape(q.shape).to(st["q"].dtype)


# ------------------------------------------------------------------- in 64 bits
def _two(e):
    """2**e as float64, for whole e in [-1022, 1023] (pow and exp2 need not be exact on a GPU)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_64(x):
    """The E4M3 value nearest to each float64 x, ties to even, saturating: a step is 2^-9 below 2^-6, else 2^(exponent - 3)."""
    _, ex = torch.frexp(x)
    step = _two((ex - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _least_exp(amax, top, floor):
    """The smallest whole e >= floor with top * 2**e >= amax, by trial around the logarithm."""
    e = torch.floor(torch.log2(amax.clamp(min=1e-300) / top)) - 1
    for _ in range(3):
        e = torch.where(top * _two(e) >= amax, e, e + 1)
    return e.clamp(min=floor)


def exact(case, seed):
    st = prepare(case, seed)
    block, lens = st["block"], [int(x) for x in st["lens"]]
    if st["op"] == "write":
        out = []
        at = (st["slots"] % block)
        ids = st["touched"]
        starts = torch.zeros(len(ids), device="cuda", dtype=torch.float64).index_add_(0, st["place"], (at == 0).double()) > 0
        scales = []
        for new, codes, scale in ((st["key"], st["k"], st["ks"]), (st["value"], st["v"], st["vs"])):
            x = new.double()
            most = torch.zeros((len(ids), x.shape[1]), device="cuda", dtype=torch.float64)
            most.index_reduce_(0, st["place"], x.abs().amax(-1), "amax")
            need = _two(_least_exp(most, E4M3_MAX, MIN_SCALE_EXP))
            before = scale[ids].double()
            s = torch.where(starts[:, None], need, torch.maximum(need, before))
            full = codes.float().double()
            moved = _e4m3_64(full[ids] * (before / s)[:, None, :, None])
            full[ids] = torch.where(starts[:, None, None, None], full[ids], moved)
            full[ids[st["place"]], at] = _e4m3_64(x / s[st["place"]][..., None])
            all_scales = scale.double()
            all_scales[ids] = s
            out.append(full)
            scales.append(all_scales)
        return out + scales
    if st["op"] == "bounds":
        x, ids, at = st["key"].double(), st["touched"], st["slots"] % block
        starts = torch.zeros(len(ids), device="cuda", dtype=torch.float64).index_add_(0, st["place"], (at == 0).double()) > 0
        old = st["bounds"].double() * _two(st["exps"].double())[:, :, None, None]
        lo = torch.where(starts[:, None, None], math.inf, old[ids][:, :, 0]).index_reduce_(0, st["place"], x, "amin")
        hi = torch.where(starts[:, None, None], -math.inf, old[ids][:, :, 1]).index_reduce_(0, st["place"], x, "amax")
        most = torch.zeros((len(ids), x.shape[1]), device="cuda", dtype=torch.float64)
        most.index_reduce_(0, st["place"], x.abs().amax(-1), "amax")
        e = _least_exp(most, 127.0, MIN_BOUND_EXP)
        e = torch.where(starts[:, None], e, torch.maximum(e, st["exps"][ids].double()))
        codes, exps = st["bounds"].clone(), st["exps"].clone()
        u = _two(e)[..., None]
        codes[ids] = torch.stack([torch.floor(lo / u), torch.ceil(hi / u)], 2).clamp(-127, 127).to(torch.int8)
        exps[ids] = e.to(torch.int32)
        return [codes, exps]

    def row(s, pool, scales, ids=None, head=None):
        ids = st["tables"][s, : _blocks(lens[s], block)].long() if ids is None else ids
        if head is not None:
            pool, scales = pool[:, :, head : head + 1], None if scales is None else scales[:, head : head + 1]
        x = pool[ids] if scales is None else pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn)
        x = x.float().double()
        if scales is not None:
            x = x * scales[ids].double()[:, None, :, None]
        return x.flatten(0, 1)

    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    heads = st["q"].shape[1]
    kv = st["k"].shape[2]
    group = heads // kv
    scale = st["scale"]
    if st["op"] == "decode":
        for s, n in enumerate(lens):
            k, v = row(s, st["k"], st["ks"])[:n], row(s, st["v"], st["vs"])[:n]
            q = st["q"][s].double().view(kv, group, -1)
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * scale, -1)
            out[s] = torch.einsum("hgn,nhd->hgd", p, v).reshape(heads, -1)
        return out
    if st["op"] == "prefill":
        begin = [int(x) for x in st["starts"]]
        for s, n in enumerate(lens):
            k, v = row(s, st["k"], st["ks"])[:n], row(s, st["v"], st["vs"])[:n]
            q = st["q"][begin[s] : begin[s + 1]].double()
            pos = n - len(q) + torch.arange(len(q), device="cuda")
            hidden = torch.arange(n, device="cuda")[None, :] > pos[:, None]
            for h in range(heads):
                w = (q[:, h] @ k[:, h // group].T) * scale
                out[begin[s] : begin[s + 1], h] = torch.softmax(w.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
        return out
    sel_tables = torch.full(st["sel_tables"].shape, -1, dtype=torch.int32, device="cuda")
    sel_lens = torch.zeros(st["sel_lens"].shape, dtype=torch.int32, device="cuda")
    for s, n in enumerate(lens):
        nb = _blocks(n, block)
        ids = st["tables"][s, :nb].long()
        for h in range(kv):
            q = st["q"][s, h * group : (h + 1) * group].double()
            f = _least_exp(q.abs().amax(-1), 255.0, MIN_BOUND_EXP)
            qi = torch.round(q / _two(f)[:, None])
            b = st["bounds"][ids, h].double()
            most = torch.einsum("gd,nd->gn", qi.clamp(max=0), b[:, 0]) + torch.einsum("gd,nd->gn", qi.clamp(min=0), b[:, 1])
            score = (most * _two(f[:, None] + st["exps"][ids, h].double()[None, :])).amax(0)
            score[: st["first"]] = math.inf
            score[max(0, nb - st["last"]):] = math.inf
            best = torch.sort(score, descending=True, stable=True).indices[: st["keep"]].sort().values
            sel_tables[s, h, : len(best)] = ids[best].int()
            m = n - (nb - len(best)) * block
            sel_lens[s, h] = m
            k, v = (row(s, st[x], st[x + "s"], ids[best], h)[:m, 0] for x in ("k", "v"))
            p = torch.softmax((st["q"][s, h * group : (h + 1) * group].double() @ k.T) * scale, -1)
            out[s, h * group : (h + 1) * group] = p @ v
    return [sel_tables, sel_lens, out]
