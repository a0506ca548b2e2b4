"""Work that stands for the quantized KV cache in real use: writing new keys
and values into it, reading rows back, and attention over it.

`run` computes an operator either in plain torch operations (fp32) or, where
`own` is true, through the library's calls. `exact` computes the same in
64 bits, from the definitions alone.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK_BYTES = {"q4_0": 18, "q8_0": 34}


# ------------------------------------------------------------------ the cases

def _attn(name, **kw):
    c = {"name": name, "op": "attn", "seqs": 1, "tokens": 1, "ragged_q": False, "past": 0, "heads": 16, "kv_heads": 8,
         "head_dim": 128, "k": "q4_0", "v": "q4_0", "dtype": "bf16", "page": 64, "window": 0, "causal": True, "pad": 0,
         "lens": 1}
    c.update(kw)
    return c


def listed():
    return [
        # the first tokens of a chat on a 0.6B model (16 query and 8 key/value heads of 128): all latency
        _attn("decode, one short sequence", past=76, dtype="f32", page=16),
        # one user far into a long document, grouped heads: the cache is split over the whole GPU
        _attn("decode, one long sequence", past=65520, heads=32, kv_heads=8, page=64),
        # a serving batch of the 0.6B model in the library's own activation type, 8-bit cache, small
        # pages, padded to a captured batch size
        _attn("decode, batch of 48", seqs=48, past=4000, k="q8_0", v="q8_0", dtype="f32", page=16, pad=16),
        # a large serving batch, eight query heads on each cache head, long contexts
        _attn("decode, batch of 64, long", seqs=64, past=16383, heads=64, kv_heads=8, page=64),
        # checking five drafted tokens at once on a 7B model (32 heads of 128, one cache head each), 8-bit keys, 4-bit values
        _attn("verify 5 tokens, 7B heads", seqs=16, tokens=5, past=2995, heads=32, kv_heads=32, k="q8_0", v="q4_0",
              dtype="f16", page=32),
        # the 512-token prompt of the library's prefill benchmark, in its activation type
        _attn("prompt of 512", tokens=512, k="q8_0", v="q8_0", dtype="f32", page=128),
        # a chunk of a long prompt behind 16K cells already written
        _attn("prompt chunk behind 16K", tokens=2048, past=16384, heads=32, kv_heads=8, page=64),
        # mixed prompts of a batch, heads of 64, sliding window
        _attn("ragged prompts, window", seqs=6, tokens=1531, ragged_q=True, past=777, heads=32, kv_heads=8, head_dim=64,
              k="q8_0", v="q4_0", dtype="f16", page=32, window=1000, lens=5),
        # one decode step's new keys and values of a batch into their cells, keys centred
        {"name": "store, 64 tokens", "op": "store", "n": 64, "dim": 1024, "k": "q8_0", "v": "q4_0", "dtype": "f32",
         "bias": True, "pad": 3},
        # a prompt's keys and values of a 0.6B model's layer
        {"name": "store, 16000 tokens", "op": "store", "n": 16000, "dim": 1024, "k": "q4_0", "v": "q4_0", "dtype": "bf16",
         "bias": False, "pad": 0},
        # a short shared prefix read back
        {"name": "load, 333 cells", "op": "load", "n": 333, "dim": 1024, "k": "q4_0", "v": "q4_0", "dtype": "f32",
         "bias": False, "pad": 0},
        # a long context read back for another consumer, keys centred
        {"name": "load, 131000 cells", "op": "load", "n": 131000, "dim": 1024, "k": "q8_0", "v": "q4_0", "dtype": "bf16",
         "bias": True, "pad": 17},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# query heads, cache heads, head size
_HEADS = ((16, 8, 128), (32, 8, 128), (64, 8, 128), (32, 32, 128), (12, 12, 64), (32, 8, 64), (8, 4, 256), (8, 1, 256),
          (28, 4, 128), (16, 16, 128))


def draw(rng):
    op = rng.choice(("decode", "decode", "verify", "prompt", "prompt", "store", "load"))
    fmts = {"k": rng.choice(("q4_0", "q8_0")), "v": rng.choice(("q4_0", "q8_0"))}
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op in ("store", "load"):
        n = _log_int(rng, 1, 16000 if op == "store" else 131000)
        return {"op": op, "n": n, "dim": 32 * _log_int(rng, 2, 32), **fmts, "dtype": dtype,
                "bias": rng.random() < 0.5, "pad": rng.randrange(0, 1 + n // 8)}
    heads, kv_heads, head_dim = rng.choice(_HEADS)
    c = {"op": "attn", "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, **fmts, "dtype": dtype,
         "page": 1 << rng.randrange(4, 9), "lens": rng.randrange(1 << 20),
         "window": _log_int(rng, 16, 4096) if rng.random() < 0.25 else 0, "causal": rng.random() < 0.9}
    if op == "prompt":
        c["seqs"], c["tokens"], c["past"] = _log_int(rng, 1, 8), _log_int(rng, 9, 2048), _log_int(rng, 1, 16384) - 1
        c["ragged_q"], most = c["seqs"] > 1, 0.8 * 2048 * 18432 * 32
    else:
        c["seqs"], c["tokens"], c["past"] = _log_int(rng, 1, 64), 1 if op == "decode" else rng.randrange(2, 9), _log_int(rng, 1, 65536) - 1
        c["ragged_q"], most = False, 0.8 * 64 * 16384 * 64
    c["pad"] = rng.choice((0, 0, 1, 7))
    # no more than the largest listed cases' scores and cache
    while c["seqs"] * c["tokens"] * (c["past"] + c["tokens"]) * heads > most or \
            c["seqs"] * (c["past"] + c["tokens"]) * kv_heads * head_dim > 0.8 * 64 * 16384 * 1024:
        c["past"] //= 2
        c["tokens"] = c["tokens"] if op != "prompt" else max(9, c["tokens"] * 3 // 4)
    return c


def _row_bytes(fmt, dim):
    return dim // 32 * BLOCK_BYTES[fmt]


def _lengths(case):
    """(new tokens, cells) of each sequence, from the case alone."""
    r = random.Random(case["lens"])
    out = []
    for i in range(case["seqs"]):
        n = r.randint(1, case["tokens"]) if case["ragged_q"] and i else case["tokens"]
        cells = n + int(case["past"] * (r.uniform(0.1, 1.0) if i else 1.0))
        # an admitted request whose cells are not there yet sees nothing
        out.append((n, 0 if case["seqs"] >= 8 and i == 3 else cells))
    return out


def _seen(case, n, cells, i):
    """Cells [lo, hi) that token i of n sees."""
    at = cells - n + i
    lo = max(0, at - case["window"] + 1) if case["window"] else 0
    hi = min(cells, at + 1) if case["causal"] else cells
    return lo, max(lo, hi)


def work(case):
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] != "attn":
        n, dim = case["n"], case["dim"]
        rows = n * (_row_bytes(case["k"], dim) + _row_bytes(case["v"], dim))
        values = 2 * n * dim
        if case["op"] == "load":
            return {"bytes": rows + values * size + 4 * n, "flops": values}
        # written, then read back as fp32 values
        return {"bytes": values * size + 2 * rows + 4 * values + 4 * n, "flops": 5 * values}
    pairs, cells, tokens = 0, 0, 0
    for n, kv in _lengths(case):
        lo_min, hi_max = kv, 0
        for i in range(n):
            lo, hi = _seen(case, n, kv, i)
            pairs += hi - lo
            if hi > lo:
                lo_min, hi_max = min(lo_min, lo), max(hi_max, hi)
        cells += max(0, hi_max - lo_min)
        tokens += n
    dim = case["kv_heads"] * case["head_dim"]
    row = _row_bytes(case["k"], dim) + _row_bytes(case["v"], dim)
    return {"bytes": cells * row + 2 * tokens * case["heads"] * case["head_dim"] * size,
            "flops": 4 * pairs * case["heads"] * case["head_dim"]}


# ------------------------------------------------------------- the plain forms

def _halves(rows, bb):
    """Scales (fp16 bits as values) and code bytes of packed rows [..., blocks * bb]."""
    blocks = rows.view(*rows.shape[:-1], -1, bb)
    return blocks[..., :2].contiguous().view(torch.float16)[..., 0], blocks[..., 2:]


def _values(fmt, rows):
    """fp32 values of packed rows: uint8 [..., row bytes] -> [..., dim]."""
    d, codes = _halves(rows, BLOCK_BYTES[fmt])
    if fmt == "q4_0":
        c = torch.cat((codes & 15, codes >> 4), -1).to(torch.float32) - 8
    else:
        c = codes.view(torch.int8).to(torch.float32)
    return (d.to(torch.float32)[..., None] * c).flatten(-2)


def _pack(fmt, x):
    """Packed rows of fp32 x [n, dim]."""
    most = 7.0 if fmt == "q4_0" else 127.0
    b = x.view(x.shape[0], x.shape[1] // 32, 32)
    d = b.abs().amax(-1, keepdim=True)
    d = (d / torch.full_like(d, most)).to(torch.float16)  # by a tensor: a number would be turned into its reciprocal
    D = d.to(torch.float32)
    t = b / torch.where(D == 0, torch.ones_like(D), D)
    whole = torch.trunc(t)
    c = whole + torch.sign(t) * ((t - whole).abs() >= 0.5)  # half away from zero
    c = torch.where(D == 0, torch.zeros_like(c), c.clamp(-8.0 if fmt == "q4_0" else -127.0, most))
    if fmt == "q4_0":
        u = (c + 8).to(torch.uint8)
        codes = u[..., :16] | (u[..., 16:] << 4)
    else:
        codes = c.to(torch.int8).view(torch.uint8)
    return torch.cat((d.view(torch.uint8), codes), -1).flatten(-2)


def _plain_store(s):
    at = s["slots"].long()
    keep = at >= 0
    for fmt, x, bias, cache in ((s["k_fmt"], s["k"], s["bias"], s["k_cache"]), (s["v_fmt"], s["v"], None, s["v_cache"])):
        x = x.to(torch.float32)
        rows = _pack(fmt, x if bias is None else x - bias)
        cache[at[keep]] = rows[keep]
    return _plain_load(s, torch.float32, None)


def _plain_load(s, dtype, bias):
    at = s["slots"].long()
    keep = (at >= 0)[:, None]
    at = at.clamp(min=0)
    k = _values(s["k_fmt"], s["k_cache"][at])
    if bias is not None:
        k = k + bias
    v = _values(s["v_fmt"], s["v_cache"][at])
    return torch.where(keep, k, torch.zeros_like(k)).to(dtype), torch.where(keep, v, torch.zeros_like(v)).to(dtype)


def _plain_attn(s):
    B, n, L = s["seqs"], s["max_q"], s["max_kv"]
    H, HK, D, T = s["heads"], s["kv_heads"], s["head_dim"], s["q"].shape[0]
    G = H // HK
    dev = s["q"].device
    j = torch.arange(L, device=dev)
    real = j[None, :] < s["kv_len"][:, None]
    cell = (s["table"].long()[:, j // s["page"]] * s["page"] + j % s["page"])
    cell = torch.where(real, cell, torch.zeros_like(cell))
    k = _values(s["k_fmt"], s["k_cache"][cell]).view(B, L, HK, D)
    v = _values(s["v_fmt"], s["v_cache"][cell]).view(B, L, HK, D)
    v = torch.where(real[:, :, None, None], v, torch.zeros_like(v))
    count = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(n, device=dev)
    token = (s["q_start"][:-1].long()[:, None] + i[None, :]).clamp(max=T - 1)
    q = s["q"].to(torch.float32)[token].view(B, n, HK, G, D).permute(0, 2, 1, 3, 4).reshape(B, HK, n * G, D)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * s["scale"]  # [B, HK, n * G, L]
    del k, q
    at = s["kv_len"].long()[:, None] - count[:, None] + i[None, :]
    seen = real[:, None, :].expand(B, n, L)
    if s["causal"]:
        seen = seen & (j[None, None, :] <= at[:, :, None])
    if s["window"]:
        seen = seen & (j[None, None, :] > at[:, :, None] - s["window"])
    seen = seen[:, None, :, None, :].expand(B, 1, n, G, L).reshape(B, 1, n * G, L)
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = torch.exp(scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = scores.sum(-1, keepdim=True)
    o = torch.matmul(scores, v.permute(0, 2, 1, 3).contiguous()) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(B, HK, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, H, D)
    there = i[None, :] < count[:, None]
    s["out"][token[there]] = o[there].to(s["out"].dtype)
    return s["out"]


# --------------------------------------------------------------- state and run

def _rows(case, gen, n, bias=None):
    """fp32 keys and values as a model makes them: a few strong channels with a mean of their own in the keys."""
    dim = case["dim"] if "dim" in case else case["kv_heads"] * case["head_dim"]
    k = torch.randn(n, dim, device="cuda", generator=gen)
    if bias is not None:
        k += bias
    v = torch.randn(n, dim, device="cuda", generator=gen)
    return k, v


def _key_bias(dim, gen):
    b = 0.2 * torch.randn(dim, device="cuda", generator=gen)
    b[torch.randint(0, dim, (max(1, dim // 64),), device="cuda", generator=gen)] = 3.0
    return b


def _cache(fmt, cells, dim, gen):
    """A cache whose cells hold what was there before: any bytes."""
    return torch.randint(0, 256, (cells, _row_bytes(fmt, dim)), dtype=torch.uint8, device="cuda", generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]
    s = {"op": case["op"], "k_fmt": case["k"], "v_fmt": case["v"], "dtype": dtype}
    if case["op"] != "attn":
        n, dim = case["n"], case["dim"]
        cells = n + n // 3 + 64
        bias = _key_bias(dim, gen)
        s["bias"] = bias if case["bias"] else None
        s["k_cache"], s["v_cache"] = _cache(case["k"], cells, dim, gen), _cache(case["v"], cells, dim, gen)
        slots = torch.randperm(cells, device="cuda", generator=gen)[:n].to(torch.int32)
        if case["pad"]:
            slots[n - case["pad"]:] = -1
        s["slots"], s["dim"] = slots, dim
        k, v = _rows(case, gen, n, bias)
        if case["op"] == "load":
            keep = slots >= 0
            s["k_cache"][slots[keep].long()] = _pack(case["k"], k - bias if case["bias"] else k)[keep]
            s["v_cache"][slots[keep].long()] = _pack(case["v"], v)[keep]
        else:
            # keys and values as slices of one fused projection
            kv = torch.cat((k, v), 1).to(dtype)
            s["k"], s["v"] = kv[:, :dim], kv[:, dim:]
        return s
    H, HK, D, ps = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    lens = _lengths(case)
    tokens = sum(n for n, _ in lens)
    need = [-(-kv // ps) for _, kv in lens]
    pages = sum(need) + 3
    wide = max(1, max(need))
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(len(lens))], device="cuda")
    need_t = torch.tensor(need, device="cuda")
    col = torch.arange(wide, device="cuda")
    inside = col[None, :] < need_t[:, None]
    table = torch.where(inside, order[(first[:, None] + col[None, :]).clamp(max=pages - 1)], -torch.ones_like(order[:1]))
    s["table"] = table.contiguous()
    for x, fmt in (("k", case["k"]), ("v", case["v"])):
        cache = _cache(fmt, pages * ps, HK * D, gen)
        bias = _key_bias(HK * D, gen) if x == "k" else None
        for b, (_, kv) in enumerate(lens):  # cells past a sequence's end keep their old bytes
            p = table[b, :need[b]].long()
            cell = (p[:, None] * ps + torch.arange(ps, device="cuda")[None, :]).flatten()[:kv]
            rows = torch.randn(kv, HK * D, device="cuda", generator=gen)
            if bias is not None:
                rows += bias
            cache[cell] = _pack(fmt, rows)
        s[x + "_cache"] = cache
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")
    # queries as a slice of one fused projection
    qkv = torch.randn(tokens + case["pad"], H + 2 * HK, D, device="cuda", generator=gen).to(dtype)
    s["q"] = qkv[:, :H]
    s["out"] = torch.zeros(tokens + case["pad"], H, D, dtype=dtype, device="cuda")
    s.update(seqs=case["seqs"], max_q=max(n for n, _ in lens), max_kv=max(1, max(kv for _, kv in lens)), heads=H, kv_heads=HK,
             head_dim=D, page=ps, window=case["window"], causal=case["causal"], scale=1.0 / math.sqrt(D))
    return s


def run(s):
    if own:
        import block_quantized_weight_qmat_amd as qmat
        if s["op"] == "attn":
            return qmat.attn(s["k_fmt"], s["v_fmt"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"],
                             kv_heads=s["kv_heads"], page_size=s["page"], scale=s["scale"], causal=s["causal"],
                             window=s["window"], max_q=s["max_q"], max_kv=s["max_kv"], out=s["out"])
        if s["op"] == "store":
            qmat.kv_store(s["k_fmt"], s["v_fmt"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_bias=s["bias"])
            return qmat.kv_load(s["k_fmt"], s["v_fmt"], s["k_cache"], s["v_cache"], s["slots"], s["dim"], dtype=torch.float32)
        return qmat.kv_load(s["k_fmt"], s["v_fmt"], s["k_cache"], s["v_cache"], s["slots"], s["dim"], dtype=s["dtype"],
                            k_bias=s["bias"])
    if s["op"] == "attn":
        return _plain_attn(s)
    return _plain_store(s) if s["op"] == "store" else _plain_load(s, s["dtype"], s["bias"])


# ------------------------------------------------------------------- in 64 bits

def _exact_values(fmt, rows):
    """Packed rows in 64 bits: byte t of a Q4_0 block holds elements t and t + 16."""
    n = rows.shape[0]
    raw = rows.reshape(n, -1, BLOCK_BYTES[fmt]).to(torch.int64)
    bits = raw[:, :, 0] + 256 * raw[:, :, 1]
    sign = 1.0 - 2.0 * (bits >> 15).double()
    e, m = (bits >> 10) & 31, (bits & 1023).double()
    d = sign * torch.where(e == 0, m * 2.0 ** -24, (1024 + m) * torch.pow(2.0, e.double() - 25))
    if fmt == "q4_0":
        c = torch.empty(n, raw.shape[1], 32, dtype=torch.float64, device=rows.device)
        c[:, :, :16] = (raw[:, :, 2:] % 16 - 8).double()
        c[:, :, 16:] = (raw[:, :, 2:] // 16 - 8).double()
    else:
        c = raw[:, :, 2:].double()
        c = c - 256 * (c >= 128)
    return (c * d[:, :, None]).reshape(n, -1)


def _exact_rounded(fmt, x):
    """The values that rows x (fp32 numbers) are held as: the rule's fp32 quotients, all else in 64 bits."""
    most, least = (7, -8) if fmt == "q4_0" else (127, -127)
    b = x.double().reshape(x.shape[0], -1, 32)
    d = (b.abs().amax(2, keepdim=True) / most).float().half().double()
    t = (b / d).float().double()
    c = torch.sign(t) * torch.floor(t.abs() + 0.5)
    c = torch.where(d > 0, c.clamp(least, most), torch.zeros_like(c))
    return (c * d).reshape(x.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attn":
        out = []
        for x, fmt, bias in (("k", case["k"], s["bias"]), ("v", case["v"], None)):
            gone = s["slots"] < 0
            if case["op"] == "store":
                rows = s[x].float()
                v = _exact_rounded(fmt, rows if bias is None else rows - bias)
            else:
                v = _exact_values(fmt, s[x + "_cache"][s["slots"].long().clamp(min=0)])
                v = v if bias is None else v + bias.double()
            v[gone] = 0
            out.append(v)
        return tuple(out)
    H, HK, D, ps = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    out = torch.zeros(s["q"].shape[0], H, D, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, kv) in enumerate(_lengths(case)):
        if kv:
            j = torch.arange(kv, device="cuda")
            cell = s["table"][b].long()[j // ps] * ps + j % ps
            k = _exact_values(case["k"], s["k_cache"][cell]).view(kv, HK, D)
            v = _exact_values(case["v"], s["v_cache"][cell]).view(kv, HK, D)
            at = kv - n + torch.arange(n, device="cuda")
            hide = torch.zeros(n, kv, dtype=torch.bool, device="cuda")
            if case["causal"]:
                hide |= j[None, :] > at[:, None]
            if case["window"]:
                hide |= j[None, :] <= at[:, None] - case["window"]
            some = ~hide.all(1)
            for h in range(H):
                g = h // (H // HK)
                z = (s["q"][t0:t0 + n, h].double() @ k[:, g].t()) / math.sqrt(D)
                p = torch.softmax(z.masked_fill(hide, -math.inf)[some], 1)
                out[t0:t0 + n, h][some] = p @ v[:, g]
        t0 += n
    return out
