"""Workloads of the paged serving operators: plain torch forms, the library's calls, and 64-bit results.

Four operators that a decoding step runs one after another, over the same paged cache:

  step   block tables, slot map, positions and cumulative lengths, from the requests' lengths on the GPU
  write  a step's new K and V rows stored in the cache by slot
  attn   attention of each request's new tokens (one, a few, or a chunk) over its pages
  diff   the same with differential attention: softmax map 1 minus lambda times softmax map 2

``own`` selects the library's calls; otherwise the same outputs come from elementary torch operations in
32 bits.  Lengths follow from a case alone, values from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCORES = 1 << 31  # scores that the plain form holds at once


def listed():
    return [
        # one decoding step of a small server: a token for each of 48 requests, a few rows of the batch idle
        {"name": "step_decode", "op": "step", "batch": 56, "idle": 8, "new": 1, "chunks": 0, "chunk": 0, "context": 8000,
         "finished": 0, "block": 64, "tail": 8, "lens": 11},
        # continuous batching at its largest: prompts join, requests end, everyone else decodes
        {"name": "step_mixed", "op": "step", "batch": 1000, "idle": 40, "new": 2, "chunks": 60, "chunk": 2000,
         "context": 12000, "finished": 90, "block": 16, "tail": 500, "lens": 12},
        # the K and V of a decoding step, sliced from a fused projection's output
        {"name": "write_decode", "op": "write", "tokens": 120, "tail": 8, "heads": 8, "dk": 128, "dv": 128, "block": 64,
         "spare": 900, "fused": True, "dtype": "bf16", "lens": 21},
        # the K and V of a long prompt's chunk
        {"name": "write_prefill", "op": "write", "tokens": 40000, "tail": 960, "heads": 8, "dk": 128, "dv": 128, "block": 128,
         "spare": 16, "fused": False, "dtype": "bf16", "lens": 22},
        # one user, one token: latency
        {"name": "attn_decode_one", "op": "attn", "batch": 1, "idle": 0, "new": 1, "chunks": 0, "chunk": 0, "context": 1500,
         "heads": 32, "kv_heads": 8, "d": 128, "block": 64, "mask": 9, "lse": False, "tail": 0, "dtype": "fp16", "lens": 31},
        # a full decoding batch over ragged long contexts: the cache's bytes bound it
        {"name": "attn_decode_batch", "op": "attn", "batch": 128, "idle": 4, "new": 1, "chunks": 0, "chunk": 0,
         "context": 16000, "heads": 32, "kv_heads": 8, "d": 128, "block": 64, "mask": 9, "lse": False, "tail": 4,
         "dtype": "bf16", "lens": 32},
        # speculative tokens with ALiBi, an odd group and small pages, the lse kept for a merge
        {"name": "attn_spec_alibi", "op": "attn", "batch": 33, "idle": 1, "new": 5, "chunks": 0, "chunk": 0, "context": 7000,
         "heads": 40, "kv_heads": 8, "d": 80, "block": 16, "mask": 3, "lse": True, "tail": 3, "dtype": "fp16", "lens": 33},
        # chunked prefill with decoding requests in the same batch
        {"name": "attn_chunk_mixed", "op": "attn", "batch": 40, "idle": 0, "new": 1, "chunks": 4, "chunk": 1100,
         "context": 9000, "heads": 32, "kv_heads": 4, "d": 64, "block": 32, "mask": 9, "lse": False, "tail": 7,
         "dtype": "bf16", "lens": 34},
        # the largest: long chunks over long prefixes
        {"name": "attn_chunk_long", "op": "attn", "batch": 3, "idle": 0, "new": 1, "chunks": 3, "chunk": 4096,
         "context": 20000, "heads": 32, "kv_heads": 8, "d": 128, "block": 128, "mask": 9, "lse": False, "tail": 0,
         "dtype": "bf16", "lens": 35},
        # differential attention, one token of a small batch
        {"name": "diff_decode_small", "op": "diff", "batch": 5, "idle": 0, "new": 1, "chunks": 0, "chunk": 0, "context": 2500,
         "heads": 16, "kv_heads": 4, "d": 64, "block": 64, "mask": 9, "norm": True, "tail": 3, "dtype": "bf16", "lens": 41},
        # a full decoding batch at the larger head size
        {"name": "diff_decode_batch", "op": "diff", "batch": 64, "idle": 2, "new": 1, "chunks": 0, "chunk": 0,
         "context": 12000, "heads": 16, "kv_heads": 4, "d": 128, "block": 64, "mask": 9, "norm": True, "tail": 0,
         "dtype": "bf16", "lens": 42},
        # chunks of prompts beside decoding requests
        {"name": "diff_chunk", "op": "diff", "batch": 12, "idle": 0, "new": 1, "chunks": 4, "chunk": 1500, "context": 6000,
         "heads": 16, "kv_heads": 8, "d": 64, "block": 32, "mask": 9, "norm": True, "tail": 5, "dtype": "fp16", "lens": 43},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["step", "write", "attn", "attn", "diff"])
    lens = rng.randrange(1 << 30)
    if op == "step":
        batch = _log(rng, 1, 1000)
        idle = rng.randint(0, batch // 4)
        return {"op": op, "batch": batch, "idle": idle, "new": rng.choice([1, 1, 2, 5]), "chunks": rng.randint(0, min(60, batch - idle)),
                "chunk": _log(rng, 16, 2000), "context": _log(rng, 16, 12000), "finished": rng.randint(0, batch // 8),
                "block": rng.choice([16, 32, 64, 128]), "tail": rng.randint(0, 500), "lens": lens}
    if op == "write":
        heads, dk, dv = rng.choice([(rng.randint(1, 16), 8 * rng.randint(2, 32), 0), (1, 512, 64)])
        tokens = max(1, min(_log(rng, 1, 40000), 40_000_000 // (heads * dk)))
        return {"op": op, "tokens": tokens, "tail": rng.randint(0, 100), "heads": heads, "dk": dk, "dv": dv or dk,
                "block": rng.choice([16, 32, 64, 128]), "spare": rng.randint(0, 500), "fused": dv == 0 and rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "lens": lens}
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16] if kv_heads < 8 else [1, 2, 3, 4, 5])
    kind = rng.choice(["decode", "decode", "spec", "chunk"])
    case = {"op": op, "batch": 0, "idle": 0, "new": 1, "chunks": 0, "chunk": 0, "context": _log(rng, 1, 16000),
            "heads": kv_heads * group, "kv_heads": kv_heads}
    if op == "attn":
        case["d"] = rng.choice([32, 40, 64, 64, 72, 80, 96, 112, 128, 128, 128, 192, 256])
        case["mask"] = rng.choice([9, 9, 9, 0] + ([3, 4, 5] if case["d"] <= 128 else []))
        case["lse"] = rng.random() < 0.3
    else:
        case["d"] = rng.choice([16, 32, 40, 64, 64, 96, 128])
        case["mask"] = rng.choice([9, 9, 0])
        case["norm"] = rng.random() < 0.7
    if kind == "chunk":
        case["chunk"] = _log(rng, 16, 2000)
        case["chunks"] = rng.randint(1, 3)
        case["batch"] = case["chunks"] + _log(rng, 1, 12)
        case["context"] = min(case["context"], 8000)
    else:
        case["new"] = 1 if kind == "decode" else rng.randint(2, 9)
        case["batch"] = _log(rng, 1, 96)
    case["idle"] = rng.randint(0, case["batch"] // 6)
    case.update(block=rng.choice([16, 32, 48, 64, 128]), tail=rng.randint(0, 9), dtype=rng.choice(["bf16", "fp16"]), lens=lens)
    return case


def lengths(case):
    """(new tokens, keys cached before, finished) of each row of the batch; idle rows come last."""
    rng = random.Random(case["lens"])
    live = case["batch"] - case["idle"]
    new, cached, done = [], [], []
    for b in range(case["batch"]):
        c = rng.randint(case["context"] // 8, case["context"])
        n = rng.randint(max(1, case["chunk"] // 2), case["chunk"]) if b < case["chunks"] else case["new"]
        new.append(n if b < live else 0)
        cached.append(c if b < live else 0)
        done.append(0)
    for b in rng.sample(range(live), min(case.get("finished", 0), live - 1)):
        done[b], new[b] = 1, 0
    return new, cached, done


def _pages(keys, block):
    return [-(-k // block) for k in keys]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(pages, width, order):
    """Block tables over consecutive runs of `order` (a permutation of the blocks); unused entries are -1."""
    at, rows = 0, []
    for n in pages:
        rows.append(torch.nn.functional.pad(order[at:at + n], (0, width - n), value=-1))
        at += n
    return torch.stack(rows).to("cuda", torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)

    if case["op"] == "step":
        new, cached, done = lengths(case)
        held = _pages(cached, case["block"])
        kv = [n + (0 if f else c) for n, c, f in zip(new, cached, done)]
        width = max(held + _pages(kv, case["block"])) + 3
        blocks = sum(held) + sum(_pages(kv, case["block"])) + 10
        order = torch.randperm(blocks, generator=host)
        free = torch.full((blocks,), -1, dtype=torch.int64)
        free[:blocks - sum(held)] = order[sum(held):]
        return {"op": "step", "new": _ints(new), "cached": _ints(cached), "finished": _ints(done) if case["finished"] else None,
                "tables": _tables(held, width, order), "free": free.to("cuda", torch.int32),
                "count": _ints([blocks - sum(held)]), "block": case["block"], "tokens": sum(new) + case["tail"]}

    dtype = DTYPES[case["dtype"]]
    if case["op"] == "write":
        n, h, dk, dv = case["tokens"] + case["tail"], case["heads"], case["dk"], case["dv"]
        blocks = -(-(case["tokens"] + case["spare"]) // case["block"])
        slots = torch.randperm(blocks * case["block"], generator=host)[:case["tokens"]]
        slots = torch.cat([slots, torch.full((case["tail"],), -1)]).to("cuda", torch.int32)
        if case["fused"]:  # [q | k | v] of one projection: rows of k and v lie a whole fused row apart
            fused = randn(n, h * (dk + dk + dv), dtype=dtype)
            key, value = fused[:, h * dk:2 * h * dk].view(n, h, dk), fused[:, 2 * h * dk:].view(n, h, dv)
        else:
            key, value = randn(n, h, dk, dtype=dtype), randn(n, h, dv, dtype=dtype)
        return {"op": "write", "key": key, "value": value, "slots": slots, "written": case["tokens"],
                "key_cache": randn(blocks, case["block"], h, dk, dtype=dtype),
                "value_cache": randn(blocks, case["block"], h, dv, dtype=dtype)}

    new, cached, _ = lengths(case)
    kv = [n + c for n, c in zip(new, cached)]
    pages = _pages(kv, case["block"])
    blocks = sum(pages) + 5
    tokens, heads, kv_heads, d, block = sum(new) + case["tail"], case["heads"], case["kv_heads"], case["d"], case["block"]
    state = {"op": case["op"], "new": new, "kv": kv, "seq_len": _ints(new), "kv_seq_len": _ints(kv),
             "tables": _tables(pages, max(pages) + 2, torch.randperm(blocks, generator=host)), "heads": heads,
             "kv_heads": kv_heads, "scale": 1.0 / math.sqrt(d), "mask": case["mask"]}
    if case["op"] == "attn":
        slopes = [2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]
        state.update(q=randn(tokens, heads, d, dtype=dtype), k_cache=randn(blocks, block, kv_heads, d, dtype=dtype),
                     v_cache=randn(blocks, block, kv_heads, d, dtype=dtype), out=torch.zeros((tokens, heads, d), dtype=dtype, device="cuda"),
                     slopes=torch.tensor(slopes, device="cuda") if case["mask"] in (3, 4, 5) else None,
                     lse=torch.zeros((tokens, heads), device="cuda") if case["lse"] else None)
    else:
        state.update(q=randn(tokens, 2 * heads, d, dtype=dtype), k_cache=randn(blocks, block, 2 * kv_heads, d, dtype=dtype),
                     v_cache=randn(blocks, block, kv_heads, 2 * d, dtype=dtype),
                     out=torch.zeros((tokens, heads, 2 * d), dtype=dtype, device="cuda"), lam=0.5 + randn(heads, scale=0.1),
                     norm=1.0 + randn(2 * d, scale=0.1) if case["norm"] else None, eps=1e-5, out_scale=0.2 if case["norm"] else 1.0)
    return state


# ---------------------------------------------------------------------------- the library's calls
def _own(s):
    import paged_attention_varlen_b200 as ala
    if "call" not in s:  # planned once for a state's buffers, as a server does before its loop
        if s["op"] == "step":
            s["call"], s["outs"] = ala.plan_paged_step(s["new"], s["cached"], s["tables"], s["free"], s["count"], s["block"],
                                                       s["tokens"], finished=s["finished"])
        elif s["op"] == "write":
            s["call"] = ala.plan_paged_write(s["key"], s["value"], s["slots"], s["key_cache"], s["value_cache"])
        elif s["op"] == "attn":
            s["call"], _ = ala.plan_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_len"], s["kv_seq_len"],
                                                    s["mask"], s["heads"], s["kv_heads"], s["scale"], slopes=s["slopes"],
                                                    out=s["out"], lse=s["lse"])
        else:
            s["call"], _ = ala.plan_paged_diff_attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_len"],
                                                         s["kv_seq_len"], s["lam"], s["mask"], s["heads"], s["kv_heads"],
                                                         s["scale"], norm_weight=s["norm"], norm_eps=s["eps"],
                                                         out_scale=s["out_scale"], out=s["out"])
    s["call"]()
    if s["op"] == "step":
        o = s["outs"]
        return {"kv": o.kv_seq_len, "count": o.free_count, "cu": o.cu_seq_len, "slots": o.slot_mapping, "positions": o.positions,
                "status": o.status, "tables": s["tables"], "free": s["free"]}
    if s["op"] == "write":
        return {"key_cache": s["key_cache"], "value_cache": s["value_cache"]}
    return {"out": s["out"], "lse": s.get("lse")}


# ---------------------------------------------------------------------------- the plain forms
def _step(s):
    new, cached, block, tables, free = s["new"], s["cached"], s["block"], s["tables"], s["free"]
    batch, width = tables.shape
    zero = torch.zeros_like(new)
    gone = zero.bool() if s["finished"] is None else s["finished"] != 0
    page = torch.arange(width, device="cuda")
    # blocks of finished requests go onto the free stack, in request order
    given = torch.where(gone, (cached + block - 1) // block, zero)
    at = s["count"] + given.cumsum(0) - given
    mine = page < given[:, None]
    where = torch.where(mine, at[:, None] + page, free.numel())
    free.copy_(torch.cat([free, free[:1]]).scatter(0, where.reshape(-1).long(), tables.reshape(-1))[:-1])
    top = s["count"] + given.sum(dtype=torch.int32)
    # new blocks come off its top, in request order
    before = torch.where(gone, zero, cached)
    kv = before + new
    have, want = (before + block - 1) // block, (kv + block - 1) // block
    taken = want - have
    kth = (taken.cumsum(0) - taken)[:, None] + page - have[:, None]
    fresh = (page >= have[:, None]) & (page < want[:, None])
    tables.copy_(torch.where(fresh, free[(top - 1 - kth).clamp(0, free.numel() - 1).long()], tables))
    cu = torch.cat([zero[:1], new.cumsum(0, dtype=torch.int32)])
    token = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    row = torch.searchsorted(cu[1:], token, right=True).clamp(max=batch - 1)
    pos = before[row] + token - cu[row]
    real = token < cu[-1]
    slot = tables[row, (pos // block).clamp(0, width - 1).long()] * block + pos % block
    return {"kv": kv, "count": top - taken.sum(dtype=torch.int32), "cu": cu, "slots": torch.where(real, slot, -1).to(torch.int32),
            "positions": torch.where(real, pos, 0).to(torch.int32), "status": zero[:1], "tables": tables, "free": free}


def _write(s):
    n = s["written"]
    at = s["slots"][:n].long()
    s["key_cache"].flatten(0, 1).index_copy_(0, at, s["key"][:n])
    s["value_cache"].flatten(0, 1).index_copy_(0, at, s["value"][:n])
    return {"key_cache": s["key_cache"], "value_cache": s["value_cache"]}


def _parts(s):
    """Runs of requests whose padded scores fit: (first, end, most new tokens, most keys)."""
    parts, heads = [], s["q"].shape[1]
    for b, (n, k) in enumerate(zip(s["new"], s["kv"])):
        if n == 0:
            continue
        if parts:
            lo, hi, pn, pk = parts[-1]
            if (b + 1 - lo) * max(n, pn) * max(k, pk) * heads <= SCORES and max(n, pn) <= 4 * min(n, pn):
                parts[-1] = (lo, b + 1, max(n, pn), max(k, pk))
                continue
        parts.append((b, b + 1, n, k))
    return parts


def _maps(s, lo, hi, n, k, first):
    """softmax maps [requests, heads, n, k] in fp32, their lse, and which query rows are real."""
    tables, block = s["tables"][lo:hi, :-(-k // s["k_cache"].shape[1])].clamp(min=0).long(), s["k_cache"].shape[1]
    seq, kv = s["seq_len"][lo:hi, None], s["kv_seq_len"][lo:hi, None]
    i, j = torch.arange(n, device="cuda"), torch.arange(k, device="cuda")
    row = (first + torch.cumsum(seq, 0) - seq + i).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][row].float().transpose(1, 2)
    keys = s["k_cache"][tables].flatten(1, 2)[:, :k].float().permute(0, 2, 3, 1)
    heads, kv_heads = q.shape[1], keys.shape[1]
    if s["op"] == "diff":  # query heads come as (kv head, group, map), key heads as (kv head, map)
        q = q.unflatten(1, (s["kv_heads"], -1, 2)).transpose(2, 3)
    x = torch.matmul(q.reshape(hi - lo, kv_heads, -1, q.shape[-1]), keys).view(hi - lo, heads, n, k) * s["scale"]
    last = (i + kv - seq)[:, None, :, None]  # absolute position of each new token
    if s["mask"] in (3, 4, 5):
        # left-aligned ALiBi is right-aligned ALiBi plus slope * last, a constant of the row: the softmax takes the small
        # form and the lse gets the constant in 64 bits
        slope = s["slopes"][:, None, None]
        gap = (j - last).float()
        x = x + (-slope * (-gap).clamp(min=0).sqrt() if s["mask"] == 4 else slope * gap)
    allowed = j < kv[:, None, None]
    if s["mask"] != 0:
        allowed = allowed & (j <= last)
    x = x.masked_fill_(~allowed, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.clamp(min=-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    lse = top + total.log()
    if s["mask"] == 5:
        lse = (lse.double() + slope.double() * last).float()
    lse = lse[..., 0].transpose(1, 2)
    return x.div_(total.clamp(min=1e-30)), lse, row, (i < seq), tables


def _attention(s):
    out, lse = s["out"], s.get("lse")
    for lo, hi, n, k in _parts(s):
        p, part_lse, row, real, tables = _maps(s, lo, hi, n, k, sum(s["new"][:lo]))
        values = s["v_cache"][tables].flatten(1, 2)[:, :k].float().transpose(1, 2)
        if s["op"] == "diff":
            p = p.view(hi - lo, s["kv_heads"], 2, -1, n, k)
            p = p[:, :, 0] - s["lam"].view(s["kv_heads"], -1, 1, 1) * p[:, :, 1]
        o = torch.matmul(p.reshape(hi - lo, s["kv_heads"], -1, k), values).view(hi - lo, s["heads"], n, -1).transpose(1, 2)
        if s["op"] == "diff":
            if s["norm"] is not None:
                o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + s["eps"]) * s["norm"]
            o = o * s["out_scale"]
        if sum(s["new"][lo:hi]) == (hi - lo) * n:  # every request has n new tokens: no row to leave out
            at = row.reshape(-1)
            out[at] = o.flatten(0, 1).to(out.dtype)
            if lse is not None:
                lse[at] = part_lse.flatten(0, 1)
        else:
            at = row[real]
            out[at] = o[real].to(out.dtype)
            if lse is not None:
                lse[at] = part_lse[real]
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"step": _step, "write": _write, "attn": _attention, "diff": _attention}[state["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "step":
        new, cached, done = lengths(case)
        given = sum(p for p, f in zip(_pages(cached, case["block"]), done) if f)
        kv = [n + (0 if f else c) for n, c, f in zip(new, cached, done)]
        taken = sum(_pages(kv, case["block"])) - sum(p for p, f in zip(_pages(cached, case["block"]), done) if not f)
        # lengths in and out, blocks moved from and to the stack, slot and position of every token
        return {"bytes": 4 * (4 * case["batch"] + 2 * given + 2 * taken + 2 * (sum(new) + case["tail"])), "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "write":
        return {"bytes": case["tokens"] * (2 * case["heads"] * (case["dk"] + case["dv"]) * size + 4), "flops": 0}
    new, cached, _ = lengths(case)
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["d"]
    maps = 2 if case["op"] == "diff" else 1
    pairs = sum(n * (n + c) if case["mask"] == 0 else n * c + n * (n + 1) // 2 for n, c in zip(new, cached))
    keys = sum(n + c for n, c in zip(new, cached) if n)
    moved = 2 * sum(new) * heads * maps * d * size + 2 * keys * kv_heads * maps * d * size
    # a pair costs a product of length d for its score and one of the value's length (maps * d), in each map
    return {"bytes": moved + 4 * sum(_pages([n + c for n, c in zip(new, cached)], case["block"])),
            "flops": 2 * maps * (d + maps * d) * heads * pairs}


# ---------------------------------------------------------------------------- 64 bits
def _softmax64(q, keys, scale, pos, kv, mask, slope):
    x = (q @ keys.T) * scale
    j = torch.arange(kv, device="cuda", dtype=torch.float64)
    ahead = j[None, :] - pos[:, None]
    if mask == 3:
        x = x + slope * ahead
    elif mask == 4:
        x = x - slope * torch.sqrt(torch.clamp(-ahead, min=0.0))
    elif mask == 5:
        x = x + slope * j
    if mask != 0:
        x = torch.where(ahead <= 0, x, -math.inf)
    lse = torch.logsumexp(x, dim=1)
    return torch.exp(x - lse[:, None]), lse


def exact(case, seed):
    if case["op"] == "step":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "write":
        found = []
        for rows, cache in ((s["key"], s["key_cache"]), (s["value"], s["value_cache"])):
            flat = cache.double().flatten(0, 1)
            for lo in range(0, s["written"], 4096):
                flat[s["slots"][lo:min(lo + 4096, s["written"])].long()] = rows[lo:min(lo + 4096, s["written"])].double()
            found.append(flat.view(cache.shape))
        return {"key_cache": found[0], "value_cache": found[1]}
    heads, kv_heads, d, maps = case["heads"], case["kv_heads"], case["d"], 2 if case["op"] == "diff" else 1
    group, block = heads // kv_heads, case["block"]
    out = s["out"].double()
    lse = None if s.get("lse") is None else s["lse"].double()
    at = 0
    for b, (n, kv) in enumerate(zip(s["new"], s["kv"])):
        if n == 0:
            continue
        table = s["tables"][b, :-(-kv // block)].long()
        keys = s["k_cache"][table].reshape(-1, kv_heads * maps, d)[:kv]
        values = s["v_cache"][table].reshape(-1, kv_heads, maps * d)[:kv]
        for g in range(kv_heads):
            v = values[:, g].double()
            k = [keys[:, g * maps + m].double() for m in range(maps)]
            for h in range(g * group, (g + 1) * group):
                for lo in range(0, n, 1024):
                    hi = min(lo + 1024, n)
                    pos = torch.arange(lo, hi, device="cuda", dtype=torch.float64) + (kv - n)
                    p, l = zip(*[_softmax64(s["q"][at + lo:at + hi, h * maps + m].double(), k[m], s["scale"], pos, kv, s["mask"],
                                            s["slopes"][h].double() if case["op"] == "attn" and s["slopes"] is not None else 0.0)
                                 for m in range(maps)])
                    if maps == 1:
                        o = p[0] @ v
                    else:
                        o = p[0] @ v - s["lam"][h].double() * (p[1] @ v)
                        if s["norm"] is not None:
                            o = o / torch.sqrt((o * o).sum(1, keepdim=True) / (2 * d) + s["eps"]) * s["norm"].double()
                        o = o * s["out_scale"]
                    out[at + lo:at + hi, h] = o
                    if lse is not None:
                        lse[at + lo:at + hi, h] = l[0]
        at += n
    return {"out": out, "lse": lse}
