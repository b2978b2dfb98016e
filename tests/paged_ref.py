"""Plain 64-bit forms of the paged serving operators, on the CPU, and the error bounds their GPU results are
held to.  Nothing here shares code with the library.

Bounds of an attention row (first order in the roundings).  With A_c = sum_j p_j |v_jc| and u the half step of the
input type (P and the output are rounded to it):
  * rounding P moves O_c by at most u A_c, rounding the output by u |O_c|;
  * a score is a sum of d products and a scale and a bias in 32 bits, off by at most
    delta = (d + 8) 2^-23 |scale| max_j sum_i |q_i k_ji| + 2^-21 max_j |bias_j| (natural units; the tensor core may
    truncate where it adds, hence 2^-23), which moves a weight by a relative 2 delta (itself and the sum);
  * exponentials and sums in 32 bits: n 2^-23 + 2^-19;
  * fp16 weights below 2^-14 lose up to 2^-25 each, with the largest weight at least 2^0.
"""
import math
import random

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ALIBI = (3, 4, 5)


def make_case(lens, heads, kv_heads, d, dtype, block, mask, seed, maps=1, tail=0, spare=3, norm=False):
    """lens: (new tokens, keys) per sequence.  Every slot that is not a live key holds NaN, every unused table entry -1."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g)

    pages = [-(-kv // block) for _, kv in lens]
    blocks = sum(pages) + spare
    perm = torch.randperm(blocks, generator=g)
    tables = torch.full((len(lens), max(pages + [1]) + 1), -1, dtype=torch.int32)
    k = torch.full((blocks, block, maps * kv_heads, d), float("nan"), dtype=dtype)
    v = torch.full((blocks, block, kv_heads, maps * d), float("nan"), dtype=dtype)
    at = 0
    for b, (_, kv) in enumerate(lens):
        for p in range(pages[b]):
            blk, n = int(perm[at]), min(block, kv - p * block)
            tables[b, p] = blk
            k[blk, :n] = randn(n, maps * kv_heads, d).to(dtype)
            v[blk, :n] = randn(n, kv_heads, maps * d).to(dtype)
            at += 1
    tokens = sum(n for n, _ in lens)
    case = {"q": randn(tokens + tail, maps * heads, d).to(dtype), "k": k, "v": v, "tables": tables,
            "seq": torch.tensor([n for n, _ in lens], dtype=torch.int32),
            "kv": torch.tensor([n for _, n in lens], dtype=torch.int32), "heads": heads, "kv_heads": kv_heads,
            "mask": mask, "scale": 1.0 / math.sqrt(d), "maps": maps,
            "slopes": torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]) if mask in ALIBI else None}
    if maps == 2:
        case["lam"] = torch.tensor([rng.uniform(-0.2, 0.9) for _ in range(heads)])
        case["norm"] = 1.0 + 0.1 * randn(2 * d) if norm else None
        case["eps"], case["out_scale"] = 1e-5, 0.2 if norm else 1.0
    return case


def attention(c):
    """(out, lse, bound of out, bound of lse) in 64 bits for the real tokens; lse [tokens, maps * heads]."""
    maps, heads, kv_heads, dtype = c["maps"], c["heads"], c["kv_heads"], c["q"].dtype
    group, d, dv, u = heads // kv_heads, c["q"].shape[-1], c["v"].shape[-1], HALF[c["q"].dtype]
    block = c["k"].shape[1]
    tokens = int(c["seq"].sum())
    out, tol = torch.zeros(tokens, heads, dv, dtype=torch.float64), torch.zeros(tokens, heads, dv, dtype=torch.float64)
    lse, ltol = (torch.zeros(tokens, maps * heads, dtype=torch.float64) for _ in range(2))
    at = 0
    for b, (n, kv) in enumerate(zip(c["seq"].tolist(), c["kv"].tolist())):
        if n == 0:
            continue
        table = c["tables"][b, :-(-kv // block)].long()
        keys = c["k"][table].reshape(-1, maps * kv_heads, d)[:kv].double()
        values = c["v"][table].reshape(-1, kv_heads, dv)[:kv].double()
        pos = torch.arange(n, dtype=torch.float64)[:, None] + (kv - n)
        j = torch.arange(kv, dtype=torch.float64)[None]
        for h in range(heads):
            g = h // group
            v = values[:, g]
            o, t = torch.zeros(n, dv, dtype=torch.float64), torch.zeros(n, dv, dtype=torch.float64)
            for m in range(maps):
                q, k = c["q"][at:at + n, h * maps + m].double(), keys[:, g * maps + m]
                x = q @ k.T * c["scale"]
                bias = torch.zeros_like(x)
                if c["mask"] in ALIBI:
                    slope = float(c["slopes"][h])
                    bias = (slope * (j - pos) if c["mask"] == 3 else slope * j + 0 * pos if c["mask"] == 5
                            else -slope * (pos - j).clamp(min=0).sqrt())
                allowed = torch.ones_like(x, dtype=torch.bool) if c["mask"] == 0 else j <= pos
                x = (x + bias).masked_fill(~allowed, -math.inf)
                l = torch.logsumexp(x, 1) if kv else torch.full((n,), -math.inf, dtype=torch.float64)
                p = torch.exp(x - l.clamp(min=-1e300)[:, None]).nan_to_num(0.0)
                p[~allowed] = 0.0
                # bounds
                delta = torch.zeros(n, dtype=torch.float64)
                if kv:
                    delta = (d + 8) * 2.0 ** -23 * abs(c["scale"]) * ((q.abs() @ k.abs().T) * allowed).amax(1)
                    # a bias of a key whose weight vanishes may be far larger than those that count
                    near = allowed & (p > 1e-30)
                    gap = (slope * (j - pos)).abs() if c["mask"] in (3, 5) else bias.abs()
                    delta = delta + 2.0 ** -21 * (gap * near).amax(1)
                a = p @ v.abs()
                rel = 2 * delta + kv * 2.0 ** -23 + 2.0 ** -19
                e = (u + rel)[:, None] * a
                if dtype == torch.float16 and kv:
                    e = e + 2.0 ** -25 * (allowed.double() @ v.abs())
                w = 1.0 if m == 0 else -float(c["lam"][h])
                o, t = o + w * (p @ v), t + abs(w) * e
                lse[at:at + n, h * maps + m] = l
                ltol[at:at + n, h * maps + m] = (delta + kv * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -21 * l.abs().nan_to_num(0, 0, 0) +
                                                 2.0 ** -22 * (bias.abs() * allowed).amax(1) if kv else 0.0)
            if maps == 2:
                s = c["out_scale"]
                if c["norm"] is not None:
                    r = torch.sqrt((o * o).mean(1, keepdim=True) + c["eps"])
                    weight = c["norm"].double()
                    t = weight.abs() * (t + o.abs() / r * (t * t).mean(1, keepdim=True).sqrt()) / r * (1 + 2.0 ** -4)
                    o = o / r * weight
                o, t = o * s, t * abs(s) + 2.0 ** -20 * o.abs() * abs(s)
            out[at:at + n, h] = o
            tol[at:at + n, h] = t + u * o.abs() + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133)
        at += n
    return out, lse, tol, ltol


def step(seq, ctx, done, tables, free, count, block, n_tokens):
    """A step in plain integers: (kv, count, cu, slots, positions, tables, free), or an ALA_STEP_* code."""
    width, cap = len(tables[0]) if tables else 0, len(free)
    pages = lambda keys: -(-keys // block)  # noqa: E731
    before = [0 if e else c for c, e in zip(ctx, done)]
    if any(n < 0 or c < 0 or c > width * block or n + o > width * block for n, c, o in zip(seq, ctx, before)):
        return 1
    if sum(seq) > n_tokens:
        return 2
    given = sum(pages(c) for c, e in zip(ctx, done) if e)
    if count < 0 or count + given > cap:
        return 3
    taken = sum(pages(o + n) - pages(o) for o, n in zip(before, seq))
    if taken > count + given:
        return 4
    tables, free = [list(r) for r in tables], list(free)
    for r, c, e in zip(tables, ctx, done):
        if e:
            for blk in r[:pages(c)]:
                free[count] = blk
                count += 1
    cu, slots, positions = [0], [], []
    for r, o, n in zip(tables, before, seq):
        for p in range(pages(o), pages(o + n)):
            count -= 1
            r[p] = free[count]
        for pos in range(o, o + n):
            slots.append(r[pos // block] * block + pos % block)
            positions.append(pos)
        cu.append(cu[-1] + n)
    pad = n_tokens - len(slots)
    return [o + n for o, n in zip(before, seq)], count, cu, slots + [-1] * pad, positions + [0] * pad, tables, free
