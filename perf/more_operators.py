"""Work that stands for what a step of many requests does around the packed
products and the quantized cache: page tables and slots from request lengths,
rows of a packed embedding, RMS norm into Q8_0 activations, rotary positions,
and low-rank adapters beside a shared product.

`run` computes an operator either in plain torch operations or, where `own` is
true, through the library's calls. `exact` computes the same in 64 bits, from
the definitions alone.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = {"q4_0": (32, 18), "q8_0": (32, 34), "q4_k": (256, 144), "q6_k": (256, 210)}  # elements, bytes


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step of one chat: its token's row of a 0.6B model's embedding (151936 x 1024, tied to the output head)
        {"name": "embed: one token", "op": "embed", "fmt": "q6_k", "rows": 151936, "K": 1024, "n": 1, "dtype": "f32", "lost": 0},
        # the prompts of a batch, padded to a captured size
        {"name": "embed: 16384 tokens", "op": "embed", "fmt": "q6_k", "rows": 151936, "K": 1024, "n": 16384, "dtype": "bf16", "lost": 9},
        # one chat's token in the library's own activation type: all latency
        {"name": "norm: one token", "op": "norm", "n": 1, "K": 1024, "dtype": "f32", "residual": True, "want": "rows"},
        # a decode batch of a 7B model, from the product before (fp32) to the product behind (Q8_0)
        {"name": "norm: 61 tokens to Q8_0", "op": "norm", "n": 61, "K": 4096, "dtype": "f32", "residual": True, "want": "q8"},
        # a long prompt, residual stream in bf16; its rows also go on as they are
        {"name": "norm: 8192 tokens", "op": "norm", "n": 8192, "K": 4096, "dtype": "bf16", "residual": True, "want": "both"},
        # a decode batch far into long documents, fp32 projections to fp16 queries and keys
        {"name": "rope: 64 far tokens", "op": "rope", "n": 64, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128, "axes": 1,
         "neighbours": False, "in": "f32", "out": "f16", "norm": False, "far": 1000000, "cycle": False},
        # text with pictures and a video: time, height and width, heads normed before
        {"name": "rope: 8191 tokens on 3 axes", "op": "rope", "n": 8191, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128, "axes": 3,
         "neighbours": False, "in": "bf16", "out": "bf16", "norm": True, "far": 30000, "cycle": False},
        # a decode step of 48 requests in small pages, and the token taken back
        {"name": "pages: decode of 48", "op": "pages", "seqs": 48, "tokens": 1, "past": 4000, "page": 16, "ragged": False, "short": False, "lens": 1},
        # prompts of 200 requests that arrive together behind what they have; not all of them fit
        {"name": "pages: ragged prompts", "op": "pages", "seqs": 200, "tokens": 600, "past": 3000, "page": 64, "ragged": True, "short": True, "lens": 2},
        # one chat's adapter on a projection of a 0.6B model
        {"name": "lora: one token", "op": "lora", "seqs": 1, "tokens": 1, "ragged": False, "adapters": 4, "rank": 16, "K": 1024, "M": 2048,
         "dtype": "f16", "lens": 1},
        # a decode batch of 64 requests with 24 adapters beside a 7B model's projection
        {"name": "lora: decode of 64", "op": "lora", "seqs": 64, "tokens": 1, "ragged": False, "adapters": 24, "rank": 16, "K": 4096, "M": 11008,
         "dtype": "bf16", "lens": 2},
        # ragged prompts of 7 requests, larger ranks
        {"name": "lora: ragged prompts", "op": "lora", "seqs": 7, "tokens": 509, "ragged": True, "adapters": 5, "rank": 64, "K": 11008, "M": 4096,
         "dtype": "bf16", "lens": 3},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# query heads, cache heads, head size
_HEADS = ((16, 8, 128), (32, 8, 128), (12, 12, 64), (32, 8, 64), (8, 1, 256), (16, 16, 80), (28, 4, 128))


def draw(rng):
    op = rng.choice(("embed", "norm", "norm", "rope", "rope", "pages", "pages", "lora", "lora", "lora"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op == "embed":
        fmt = rng.choice(tuple(BLOCK))
        K = 256 * _log_int(rng, 1, 16) if fmt in ("q4_k", "q6_k") else 32 * _log_int(rng, 1, 128)
        n = _log_int(rng, 1, 16384)
        while n * K > 0.9 * 16384 * 1024 or (dtype == "f32" and n * K > 0.5 * 16384 * 1024):
            n //= 2
        return {"op": op, "fmt": fmt, "rows": _log_int(rng, 100, 151936 * 1024 // max(1024, K)), "K": K, "n": n, "dtype": dtype, "lost": rng.choice((0, 1, 5))}
    if op == "norm":
        n, K = _log_int(rng, 1, 8192), 32 * _log_int(rng, 4, 344)
        while n * K > 0.45 * 8192 * 4096:
            n //= 2
        return {"op": op, "n": n, "K": K, "dtype": dtype, "residual": rng.random() < 0.7, "want": rng.choice(("rows", "q8", "both"))}
    if op == "rope":
        heads, kv_heads, head_dim = rng.choice(_HEADS)
        n = _log_int(rng, 1, 8191)
        while n * (heads + kv_heads) * head_dim > 0.5 * 8191 * 40 * 128:
            n = n * 2 // 3
        return {"op": op, "n": max(1, n), "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rot": rng.choice((head_dim, head_dim, head_dim // 2)),
                "axes": rng.choice((1, 1, 2, 3)), "neighbours": rng.random() < 0.4, "in": dtype, "out": rng.choice((dtype, "f16", "bf16")),
                "norm": rng.random() < 0.5, "far": _log_int(rng, 10, 1000000), "cycle": rng.random() < 0.4}
    if op == "pages":
        seqs, page = _log_int(rng, 1, 200), 1 << rng.randrange(4, 9)
        tokens = rng.choice((1, rng.randrange(2, 9), _log_int(rng, 9, 500)))
        return {"op": op, "seqs": seqs, "tokens": tokens, "past": _log_int(rng, 1, 3000) - 1, "page": page, "ragged": tokens > 1, "short": rng.random() < 0.4,
                "lens": rng.randrange(1 << 20)}
    tokens = rng.choice((1, 1, rng.randrange(2, 9), _log_int(rng, 9, 509)))
    c = {"op": op, "seqs": _log_int(rng, 1, 64 if tokens < 9 else 7), "tokens": tokens, "ragged": tokens > 1, "adapters": _log_int(rng, 1, 24),
         "rank": 8 * _log_int(rng, 1, 16), "K": 32 * _log_int(rng, 8, 344), "M": _log_int(rng, 256, 11008), "dtype": rng.choice(("f16", "bf16")),
         "lens": rng.randrange(1 << 20)}
    # no more than the largest listed case's products and adapters
    while c["seqs"] * c["tokens"] * c["rank"] * (c["K"] + c["M"]) > 0.5 * 7 * 509 * 64 * 15000 or c["adapters"] * c["rank"] * (c["K"] + c["M"]) > 24 * 16 * 15000:
        c["rank"], c["tokens"], c["adapters"] = max(8, c["rank"] // 16 * 8), max(1, c["tokens"] * 3 // 4), max(1, c["adapters"] - 2)
    return c


def _row_bytes(fmt, K):
    elems, size = BLOCK[fmt]
    return K // elems * size


def _lengths(case):
    """(new tokens, cells before) of each sequence, from the case alone."""
    r = random.Random(case["lens"])
    out = []
    for i in range(case["seqs"]):
        n = r.randint(1, case["tokens"]) if case["ragged"] and i else case["tokens"]
        out.append((n, int(case.get("past", 0) * (r.uniform(0.0, 1.0) if i else 1.0))))
    return out


def work(case):
    if case["op"] == "embed":
        n, K = case["n"], case["K"]
        return {"bytes": n * (4 + _row_bytes(case["fmt"], K) + K * DTYPES[case["dtype"]].itemsize), "flops": 2 * n * K}
    if case["op"] == "norm":
        values, size = case["n"] * case["K"], DTYPES[case["dtype"]].itemsize
        moved = values * size * (3 if case["residual"] else 1) + 4 * case["K"]
        if case["want"] != "q8":
            moved += values * size
        if case["want"] != "rows":  # written, then read back as fp32 values
            moved += values // 32 * 34 * 2 + 4 * values
        return {"bytes": moved, "flops": 6 * values}
    if case["op"] == "rope":
        values = case["n"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        return {"bytes": values * (DTYPES[case["in"]].itemsize + DTYPES[case["out"]].itemsize) + 4 * case["n"] * case["axes"],
                "flops": (7 if case["norm"] else 3) * values}
    lens = _lengths(case)
    if case["op"] == "pages":
        tokens, pages = sum(n for n, _ in lens), sum(-(-(n + kv) // case["page"]) for n, kv in lens)
        return {"bytes": 2 * 24 * case["seqs"] + 12 * tokens + 8 * pages, "flops": 8 * tokens}
    tokens, R, K, M = sum(n for n, _ in lens), case["rank"], case["K"], case["M"]
    ranks, of = _adapters(case)
    used = {a for a in of if a >= 0}
    with_one = [(n, ranks[a]) for (n, _), a in zip(lens, of) if a >= 0]
    return {"bytes": 2 * (K + M) * sum(ranks[a] for a in used) + tokens * (K // 32 * 34 + 8 * M),
            "flops": 2 * (K + M) * sum(n * r for n, r in with_one)}


def _adapters(case):
    """Each adapter's rank, and each sequence's adapter (-1: none)."""
    r = random.Random(case["lens"] + 1)
    ranks = [case["rank"] if a == 0 or r.random() < 0.6 else r.randint(1, case["rank"]) for a in range(case["adapters"])]
    return ranks, [-1 if case["seqs"] > 4 and r.random() < 0.1 else r.randrange(case["adapters"]) for _ in range(case["seqs"])]


# ------------------------------------------------------------- the plain forms

def _scales(raw, at):
    """fp32 values of the fp16 numbers at bytes at, at + 1 of each block [..., bytes]."""
    return raw[..., at:at + 2].contiguous().view(torch.float16).to(torch.float32)


def _nibbles(codes):
    """Low nibbles, then high ones, of [..., bytes]."""
    return torch.cat((codes & 15, codes >> 4), -1).to(torch.float32)


def _values(fmt, rows):
    """fp32 values of packed rows: uint8 [n, row bytes] -> [n, K]."""
    raw = rows.view(rows.shape[0], -1, BLOCK[fmt][1])
    if fmt == "q4_0":
        return (_scales(raw, 0) * (_nibbles(raw[..., 2:]) - 8)).flatten(1)
    if fmt == "q8_0":
        return (_scales(raw, 0) * raw[..., 2:].view(torch.int8).to(torch.float32)).flatten(1)
    if fmt == "q4_k":
        bits = raw[..., 4:16].to(torch.int32)
        bits = torch.cat((bits, torch.zeros_like(bits[..., :1])), -1)
        f = torch.arange(16, device=rows.device) * 6
        fields = ((bits[..., f // 8] + 256 * bits[..., f // 8 + 1]) >> (f % 8).to(torch.int32)) & 63
        q = _nibbles(raw[..., 16:].reshape(*raw.shape[:-1], 8, 16))
        up = (_scales(raw, 0) * fields[..., :8].to(torch.float32))[..., None]
        down = (_scales(raw, 2) * fields[..., 8:].to(torch.float32))[..., None]
        return (up * q - down).flatten(1)
    groups = raw[..., 2:].reshape(*raw.shape[:-1], 8, 26)
    low = torch.cat((groups[..., 2:18] & 15, groups[..., 2:18] >> 4), -1)
    e = torch.arange(32, device=rows.device)
    high = (groups[..., 18 + e // 16 * 4 + e % 4] >> (e % 16 // 4 * 2).to(torch.uint8)) & 3
    c = (low + 16 * high).to(torch.float32) - 32
    sc = groups[..., :2].contiguous().view(torch.int8).to(torch.float32).repeat_interleave(16, -1)
    return ((_scales(raw, 0)[..., None] * sc) * c).flatten(1)


def _pack8(x):
    """Q8_0 rows of fp32 x [n, K]."""
    b = x.view(x.shape[0], -1, 32)
    d = b.abs().amax(-1, keepdim=True)
    d = (d / torch.full_like(d, 127.0)).to(torch.float16)  # by a tensor: a number would be turned into its reciprocal
    D = d.to(torch.float32)
    t = b / torch.where(D == 0, torch.ones_like(D), D)
    whole = torch.trunc(t)
    c = (whole + torch.sign(t) * ((t - whole).abs() >= 0.5)).clamp(-127.0, 127.0)  # half away from zero
    c = torch.where(D == 0, torch.zeros_like(c), c)
    return torch.cat((d.view(torch.uint8), c.to(torch.int8).view(torch.uint8)), -1).flatten(1)


def _plain_embed(s):
    at = s["ids"].long()
    there = (at >= 0) & (at < s["table"].shape[0])
    x = _values(s["fmt"], s["table"][torch.where(there, at, torch.zeros_like(at))])
    return torch.where(there[:, None], x, torch.zeros_like(x)).to(s["dtype"])


def _plain_norm(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.to(torch.float32) + s["residual"].to(torch.float32)).to(h.dtype)
    # 64 bits: a code next to a border must not depend on how a sum is ordered
    d = h.to(torch.float64)
    y = (d / torch.sqrt((d * d).mean(-1, keepdim=True) + s["eps"]) * s["weight"].to(torch.float64)).to(torch.float32)
    q8 = _values("q8_0", _pack8(y)) if s["want"] != "rows" else None
    return y.to(h.dtype) if s["want"] != "q8" else None, q8, h if s["residual"] is not None else None


def _plain_rope(s):
    pos, axis = s["pos"], s["axis"].long()
    theta = pos.to(torch.float64)[axis].t() * s["freq"][None, :]  # [n, pairs]; far positions lose their angle in 32 bits
    cos, sin = torch.cos(theta).to(torch.float32)[:, None], torch.sin(theta).to(torch.float32)[:, None]
    pairs = s["freq"].numel()
    out = []
    for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])):
        x = x.to(torch.float32)
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        if s["neighbours"]:
            a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :pairs], x[..., pairs:2 * pairs]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        out.append(torch.cat((y, x[..., 2 * pairs:]), -1).to(s["out"]))
    return tuple(out)


def _plain_page_step(s, add, keep, rows):
    """One change of lengths; kv_len, table, free and count are updated."""
    ps, table, free = s["page"], s["table"], s["free"]
    B, wide = table.shape
    held = s["kv_len"].long().clamp(0, wide * ps)
    kept = torch.minimum(held, keep.long().clamp(min=0)) if keep is not None else held
    add = add.long().clamp(min=0)
    goal = kept + add
    old, new = (held + ps - 1) // ps, (goal + ps - 1) // ps
    fits = (goal <= wide * ps) & ((add == 0) | (add.cumsum(0) <= rows))
    back = torch.where(fits, (old - new).clamp(min=0), 0)
    need = torch.where(fits, (new - old).clamp(min=0), 0)
    count = s["count"].long().clamp(0, free.numel())
    total_back = back.cumsum(0)
    there = count + total_back[-1:]
    ok = fits & ((need == 0) | (need.cumsum(0) <= there))
    status = torch.where(ok, 0, torch.where(fits, 2, 1)).to(torch.int32)
    # pages given back, the last one lowest
    k = torch.arange(free.numel(), device=free.device)
    b = torch.searchsorted(total_back, k, right=True).clamp(max=B - 1)
    j = new[b] + k - (total_back - back)[b]
    live = k < total_back[-1]
    free[(there - 1 - k)[live]] = table[b, j.clamp(0, wide - 1)][live]
    # pages taken
    need = torch.where(ok, need, 0)
    total = need.cumsum(0)
    b = torch.searchsorted(total, k, right=True).clamp(max=B - 1)
    j = old[b] + k - (total - need)[b]
    live = k < total[-1]
    table[b[live], j[live]] = free[(there - 1 - k)[live]]
    s["count"].copy_(there - total[-1:])
    add = torch.where(ok, add, 0)
    s["kv_len"].copy_(torch.where(ok, goal, s["kv_len"].long()))
    start = torch.cat((torch.zeros_like(add[:1]), add.cumsum(0)))
    t = torch.arange(rows, device=free.device)
    live = t < start[-1]
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=B - 1)
    at = torch.where(live, kept[b] + t - start[b], 0)
    page = table[b, at // ps].long()
    slots = torch.where(live & (page >= 0) & (page < free.numel()), page * ps + at % ps, -1)
    return start.to(torch.int32), slots.to(torch.int32), at.to(torch.int32), torch.where(live, b, -1).to(torch.int32), status


def _plain_lora(s):
    n = s["y"].shape[0]
    A, R, K = s["a"].shape
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["q_start"][1:].contiguous(), t, right=True)
    of = torch.where(t < s["q_start"][-1], s["adapter"][b.clamp(max=s["adapter"].numel() - 1)], -1)
    # all adapters' products, of which a token keeps its own adapter's
    x = _values("q8_0", s["x"])
    mine = (torch.arange(A, device="cuda")[None, :] == of[:, None])[:, :, None] & (torch.arange(R, device="cuda")[None, :] < s["ranks"][:, None])[None]
    z = torch.matmul(x, s["a"].to(torch.float32).view(A * R, K).t()).view(n, A, R) * s["scale"][None, :, None]
    z = torch.where(mine, z, torch.zeros_like(z)).view(n, A * R)
    s["y"].copy_(s["base"] + torch.matmul(z, s["b"].to(torch.float32).transpose(1, 2).reshape(A * R, -1)))
    return s["y"]


# --------------------------------------------------------------- state and run

def _table(fmt, rows, K, gen):
    """Packed rows: any codes, scales as a weight matrix has them."""
    elems, size = BLOCK[fmt]
    raw = torch.randint(0, 256, (rows, K // elems, size), dtype=torch.uint8, device="cuda", generator=gen)
    d = 0.01 * (0.5 + torch.rand(rows, K // elems, device="cuda", generator=gen)) / {"q4_0": 1, "q8_0": 16, "q4_k": 32, "q6_k": 256}[fmt]
    raw[..., 0:2] = d.to(torch.float16)[..., None].view(torch.uint8)
    if fmt == "q4_k":
        raw[..., 2:4] = (7 * d).to(torch.float16)[..., None].view(torch.uint8)
    if fmt == "q6_k":  # sub-scales are not negative
        sub = 2 + 26 * torch.arange(8, device="cuda")[:, None] + torch.arange(2, device="cuda")
        raw[..., sub.flatten()] &= 127
    return raw.view(rows, -1)


def _positions(case, gen):
    """Positions of each axis: runs of text, on which they agree, and pictures, on which height and width count up."""
    n, axes = case["n"], case["axes"]
    t = torch.arange(n, device="cuda")
    first = torch.randint(0, case["far"], (1,), device="cuda", generator=gen)
    if axes == 1:  # requests at places of their own
        return ((first + t * torch.randint(1, 997, (1,), device="cuda", generator=gen)) % case["far"]).to(torch.int32)
    picture = (t // 256) % 2 == 1
    place = torch.stack([t // 256 * 32 + part for part in (t % 256 * 0, t % 256 // 16, t % 16)][:axes])
    return torch.where(picture[None, :], first + place, first + t[None, :]).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = {"op": case["op"]}
    if case["op"] == "embed":
        s.update(fmt=case["fmt"], K=case["K"], dtype=DTYPES[case["dtype"]], table=_table(case["fmt"], case["rows"], case["K"], gen))
        s["ids"] = torch.randint(0, case["rows"], (case["n"],), dtype=torch.int32, device="cuda", generator=gen)
        if case["lost"]:  # rows of padding
            s["ids"][max(0, case["n"] - case["lost"]):] = -1
        return s
    if case["op"] == "norm":
        n, K, dtype = case["n"], case["K"], DTYPES[case["dtype"]]
        x = normal(n, K)
        x[:, torch.randint(0, K, (max(1, K // 512),), device="cuda", generator=gen)] *= 30.0  # a model's few loud channels
        s.update(x=x.to(dtype), residual=(3 * normal(n, K)).to(dtype) if case["residual"] else None, weight=1 + 0.2 * normal(K), eps=1e-6,
                 want=case["want"], K=K)
        return s
    if case["op"] == "rope":
        n, H, HK, D = case["n"], case["heads"], case["kv_heads"], case["head_dim"]
        qkv = normal(n, H + 2 * HK, D).to(DTYPES[case["in"]])  # one fused projection
        pairs = case["rot"] // 2
        s.update(q=qkv[:, :H], k=qkv[:, H:H + HK], neighbours=case["neighbours"], eps=1e-6, out=DTYPES[case["out"]])
        s["freq"] = torch.tensor([10000.0 ** (-i / pairs) for i in range(pairs)], dtype=torch.float64, device="cuda")
        i = torch.arange(pairs, device="cuda")
        s["axis"] = (i % case["axes"] if case["cycle"] else i * case["axes"] // pairs).to(torch.int32)
        s["pos"] = _positions(case, gen).view(case["axes"], n)
        s["q_norm"], s["k_norm"] = (1 + 0.2 * normal(D), 1 + 0.2 * normal(D)) if case["norm"] else (None, None)
        return s
    lens = _lengths(case)
    if case["op"] == "pages":
        ps, B = case["page"], case["seqs"]
        need = [-(-kv // ps) for _, kv in lens]
        wide = max(1, max(-(-(kv + n) // ps) for n, kv in lens))
        room = sum(-(-(kv + n) // ps) for n, kv in lens) - sum(need)
        room = room // 2 if case["short"] else room + 5
        pages = sum(need) + room
        order = torch.randperm(max(1, pages), device="cuda", generator=gen).to(torch.int32)
        first = torch.tensor([sum(need[:b]) for b in range(B)], device="cuda")
        col = torch.arange(wide, device="cuda")
        inside = col[None, :] < torch.tensor(need, device="cuda")[:, None]
        s["table"] = torch.where(inside, order[(first[:, None] + col).clamp(max=max(0, pages - 1))], -torch.ones_like(order[:1])).contiguous()
        s["free"] = torch.zeros_like(order)
        s["free"][:room] = order[sum(need):pages]
        s["count"] = torch.tensor([room], dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")
        s["before"] = s["kv_len"].clone()
        s["add"] = torch.tensor([n for n, _ in lens], dtype=torch.int32, device="cuda")
        s["none"] = torch.zeros_like(s["add"])
        s.update(page=ps, rows=sum(n for n, _ in lens) + (3 if B > 1 else 0))
        return s
    tokens, R, K, M, A = sum(n for n, _ in lens), case["rank"], case["K"], case["M"], case["adapters"]
    ranks, of = _adapters(case)
    dtype = DTYPES[case["dtype"]]
    s["x"] = _pack8(normal(tokens, K))
    s["a"] = (normal(A, R, K) / math.sqrt(K)).to(dtype)
    s["b"] = (normal(A, M, R) / math.sqrt(R)).to(dtype)
    s["scale"] = 0.5 + 1.5 * torch.rand(A, device="cuda", generator=gen)
    s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
    s["adapter"] = torch.tensor(of, dtype=torch.int32, device="cuda")
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["base"], s["y"] = normal(tokens, M), torch.zeros(tokens, M, device="cuda")
    s["max_q"] = max(n for n, _ in lens)
    return s


def _own(s):
    import block_quantized_weight_qmat_amd as qmat
    if s["op"] == "embed":
        return qmat.embed(s["fmt"], s["table"], s["K"], s["ids"], dtype=s["dtype"])
    if s["op"] == "norm":
        rows, q8, h = qmat.rms_norm(s["x"], s["weight"], eps=s["eps"], residual=s["residual"], want=s["want"])
        return rows, None if q8 is None else qmat.embed("q8_0", q8, s["K"]), h
    if s["op"] == "rope":
        return qmat.rope(s["q"], s["k"], s["pos"], s["freq"], axis=s["axis"], neighbours=s["neighbours"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                         eps=s["eps"], dtype=s["out"])
    if s["op"] == "lora":
        return qmat.lora(s["x"], s["a"], s["b"], s["adapter"], s["q_start"], s["y"], base=s["base"], scale=s["scale"], ranks=s["ranks"],
                         max_q=s["max_q"])
    got = qmat.page_step(s["kv_len"], s["add"], s["table"], s["free"], s["count"], s["page"], s["rows"])
    qmat.page_step(s["kv_len"], s["none"], s["table"], s["free"], s["count"], s["page"], 0, keep=s["before"])
    return (*got, s["table"], s["free"], s["count"], s["kv_len"])


def run(s):
    if own:
        return _own(s)
    if s["op"] == "embed":
        return _plain_embed(s)
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "lora":
        return _plain_lora(s)
    # the step, then its tokens taken back, as drafted tokens are that were turned down
    got = _plain_page_step(s, s["add"], None, s["rows"])
    _plain_page_step(s, s["none"], s["before"], 0)
    return (*got, s["table"], s["free"], s["count"], s["kv_len"])


# ------------------------------------------------------------------- in 64 bits

def _half(b0, b1):
    """The number that two bytes of a binary16 stand for."""
    bits = b0.to(torch.int64) + 256 * b1.to(torch.int64)
    e, m = (bits >> 10) & 31, (bits & 1023).double()
    v = torch.where(e == 0, m * 2.0 ** -24, (1024 + m) * torch.pow(2.0, e.double() - 25))
    return torch.where(bits >= 32768, -v, v)


def _exact_values(fmt, rows):
    """Packed rows in 64 bits, one element of all blocks at a time."""
    elems, size = BLOCK[fmt]
    raw = rows.reshape(rows.shape[0], -1, size)
    w = torch.empty(*raw.shape[:2], elems, dtype=torch.float64, device=rows.device)
    d = _half(raw[..., 0], raw[..., 1])
    signed = lambda v: v.double() - 256 * (v > 127)  # noqa: E731
    for e in range(elems):
        if fmt == "q8_0":
            w[..., e] = d * signed(raw[..., 2 + e])
        elif fmt == "q4_0":
            c = raw[..., 2 + e % 16] // 16 if e >= 16 else raw[..., 2 + e] % 16
            w[..., e] = d * (c.double() - 8)
        elif fmt == "q4_k":
            j, i = e // 32, e % 32
            byte = raw[..., 16 + 16 * j + i % 16]
            q = (byte // 16 if i >= 16 else byte % 16).double()
            both = []
            for f in (j, 8 + j):
                v = 0
                for bit in range(6):
                    at = 6 * f + bit
                    v = v + ((raw[..., 4 + at // 8] >> (at % 8)) % 2).double() * 2 ** bit
                both.append(v)
            w[..., e] = d * both[0] * q - _half(raw[..., 2], raw[..., 3]) * both[1]
        else:
            g, i = e // 32, e % 32
            at = 2 + 26 * g
            byte = raw[..., at + 2 + i % 16]
            low = byte // 16 if i >= 16 else byte % 16
            high = (raw[..., at + 18 + 4 * (i // 16) + i % 4] // 4 ** (i % 16 // 4)) % 4
            w[..., e] = d * signed(raw[..., at + i // 16]) * (low.double() + 16 * high.double() - 32)
    return w.reshape(rows.shape[0], -1)


def _exact_q8(y):
    """The values that fp32 rows y are held as: the rule's fp32 quotients, all else in 64 bits."""
    b = y.double().reshape(y.shape[0], -1, 32)
    d = (b.abs().amax(2, keepdim=True) / 127).float().half().double()
    t = (b / d).float().double()
    c = (torch.sign(t) * torch.floor(t.abs() + 0.5)).clamp(-127, 127)
    return (torch.where(d > 0, c, torch.zeros_like(c)) * d).reshape(y.shape[0], -1)


def _exact_pages(case, s):
    """The step and its taking back, one sequence after the other."""
    ps, rows = s["page"], s["rows"]
    kv, add = s["kv_len"].tolist(), s["add"].tolist()
    table, free, count = s["table"].tolist(), s["free"].tolist(), int(s["count"])
    start, slots, pos, seq, status = [0], [], [], [], []
    asked = blocked = 0
    for b in range(case["seqs"]):
        goal, asked = kv[b] + add[b], asked + add[b]
        more = -(-goal // ps) - -(-kv[b] // ps)
        refused = 1 if goal > len(table[b]) * ps or (add[b] and asked > rows) else 2 if more and (blocked or more > count) else 0
        status.append(refused)
        blocked = blocked or refused == 2
        if not refused:
            for j in range(more):
                count -= 1
                table[b][-(-kv[b] // ps) + j] = free[count]
            for i in range(kv[b], goal):
                slots.append(table[b][i // ps] * ps + i % ps)
                pos.append(i)
                seq.append(b)
        start.append(len(slots))
    pad = rows - len(slots)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return (ints(start), ints(slots + [-1] * pad), ints(pos + [0] * pad), ints(seq + [-1] * pad), ints(status), ints(table), s["free"], s["count"], s["kv_len"])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(case, s)
    if case["op"] == "embed":
        at = s["ids"].long()
        w = _exact_values(case["fmt"], s["table"][at.clamp(min=0)])
        w[at < 0] = 0
        return w
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        r = (h.square().sum(1, keepdim=True) / case["K"] + s["eps"]).pow(-0.5)
        y = h * r * s["weight"].double()
        return (y if case["want"] != "q8" else None, _exact_q8(y.float()) if case["want"] != "rows" else None, h if case["residual"] else None)
    if case["op"] == "rope":
        out = []
        pairs = case["rot"] // 2
        for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])):
            x = x.double().clone()
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.double()
            y = x.clone()
            for i in range(pairs):
                u, v = (2 * i, 2 * i + 1) if case["neighbours"] else (i, i + pairs)
                theta = s["pos"][int(s["axis"][i])].double() * 10000.0 ** (-i / pairs)
                turn = torch.complex(torch.cos(theta), torch.sin(theta))[:, None]
                z = torch.complex(x[..., u], x[..., v]) * turn
                y[..., u], y[..., v] = z.real, z.imag
            out.append(y)
        return tuple(out)
    ranks, of = _adapters(case)
    x = _exact_values("q8_0", s["x"])
    y = s["base"].double()
    t = 0
    for (n, _), a in zip(_lengths(case), of):
        if a >= 0:
            r = ranks[a]
            y[t:t + n] += float(s["scale"][a]) * ((x[t:t + n] @ s["a"][a, :r].double().t()) @ s["b"][a, :, :r].double().t())
        t += n
    return y
