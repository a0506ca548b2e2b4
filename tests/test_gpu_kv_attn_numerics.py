"""Attention over the quantized cache where its arithmetic is strained: V scales
far apart, between cells and between the blocks of one, infinite key scales, large
scores, queries that are not finite. Held to the 64-bit formula within
kv_reference's bounds.
"""
import numpy as np
import pytest

import kv_reference as ref
import oracle
from test_gpu_kv_attn import DTYPES, Case, dev, largest_scale, lib, say, torch_type  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_of(c, b):
    """Cache rows of the cells of sequence b."""
    j = np.arange(c.seqs[b][1])
    return c.table[b, j // c.page].astype(np.int64) * c.page + j % c.page


def blocks_of(packed, fmt):
    """A view [cells][blocks][bytes] of packed rows."""
    return packed.reshape(packed.shape[0], -1, oracle.block_bytes(fmt))


def set_scales(packed, fmt, rows, bits):
    """Gives all blocks of the named rows the fp16 scale of these bits."""
    blocks_of(packed, fmt)[rows, :, :2] = np.frombuffer(np.uint16(bits).tobytes(), np.uint8)


def again(c):
    """The 64-bit answer and its bound from what c.k, c.v and c.qt hold now."""
    dim = c.kv_heads * c.head_dim
    kd, vd = (oracle.dequant(f, p, p.shape[0], dim) for f, p in ((c.k_fmt, c.k), (c.v_fmt, c.v)))
    qd = c.qt.double().numpy()[:, 1:1 + c.heads]
    for b, (n, kv) in enumerate(c.seqs):
        s, rows = slice(c.start[b], c.start[b + 1]), rows_of(c, b)
        o, mag = ref.attention(qd[s], kd, vd, rows, c.kv_heads, n, kv, c.scale, c.causal, c.window)
        d, dv = (largest_scale(f, p[rows]) for f, p in ((c.k_fmt, c.k), (c.v_fmt, c.v)))
        c.want[s] = o
        c.bound[s] = ref.element_bound(qd[s], d, 15 if c.k_fmt == "q4_0" else 255, max(kv, 1), abs(c.scale), mag, o, c.dtype,
                                       dv * (8 if c.v_fmt == "q4_0" else 128))


def keep_first(c, out, n):
    """c and its output without the tokens from n on (of one sequence)."""
    c.start[-1] = c.T = n
    c.want, c.bound = c.want[:n], c.bound[:n]
    return out[:n]


MAX_HALF, INF, NAN = 0x7BFF, 0x7C00, 0x7E00


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v_fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_small_values_beside_large_unseen_ones(lib, head_dim, v_fmt, dtype):  # noqa: F811
    """V scales of cells that a row does not see, the largest there are among them, cost it no precision: cells just before a
    window, and later tokens' cells of the same tile."""
    v_scale = 1e-3 if dtype == "f16" else 1e-5  # fp16 results stay above its subnormals
    for bits in (MAX_HALF, INF, NAN):
        for seqs, window, away, sure in (([(1, 200)], 50, range(128, 150), 1), ([(4, 60)], 0, (58, 59), 2),
                                         ([(100, 130)], 0, (128, 129), 98), ([(90, 600)], 70, range(384, 441), 90)):
            say(f"attn small values {head_dim} {v_fmt} {dtype} {seqs} scale bits {bits:x}")
            c = Case(seqs, 4, 2, head_dim, "q8_0", v_fmt, dtype, window=window, seed=head_dim, v_scale=v_scale)
            set_scales(c.v, v_fmt, rows_of(c, 0)[list(away)], bits)
            c.check(keep_first(c, c.run(lib), sure))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 4, 70])
def test_attn_small_values_beside_a_large_improbable_one(lib, n, dtype):  # noqa: F811
    """A cell with the largest V scale whose probability is next to nothing costs the others no precision."""
    v_scale = 1e-3 if dtype == "f16" else 1e-5
    for head_dim in (64, 128, 256):
        for v_fmt in ("q4_0", "q8_0"):
            for at in (0, 40, 90):  # first, in the middle, last (for prompts: before the first token's own)
                say(f"attn improbable {head_dim} {v_fmt} {dtype} n={n} at {at}")
                c = Case([(n, 100 + n)], 2, 2, head_dim, "q8_0", v_fmt, dtype, seed=n, v_scale=v_scale)
                # all queries lean to one direction, the cell's key is far against it: score about -90
                rng = np.random.default_rng(1)
                lean = rng.choice([-1.0, 1.0], head_dim).astype(np.float32)
                c.qt = (c.qt.float() * 0.25 + torch_of(lean)).to(torch_type(dtype))
                row = rows_of(c, 0)[at]
                key = np.tile(-90.0 / head_dim ** 0.5 * lean, 2).astype(np.float32)
                c.k[row] = oracle.quantize("q8_0", key[None])[0]
                before = c.v[row].copy()
                set_scales(c.v, v_fmt, [row], MAX_HALF)
                again(c)
                # the bound without that cell, whose part of the result is below 1e-20
                c.v[row], large = before, c.v[row].copy()
                want = c.want.copy()
                again(c)
                c.want, c.v[row] = want, large
                c.check(c.run(lib))


def torch_of(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v_fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_blocks_of_different_size(lib, head_dim, v_fmt, dtype):  # noqa: F811
    """Channels whose values are far smaller than others' keep their relative precision."""
    for n in (1, 70, 300):
        for ratio in (14, 18, 20):
            say(f"attn blocks {head_dim} {v_fmt} {dtype} n={n} ratio 2^-{ratio}")
            c = Case([(n, n + 60)], 4, 2, head_dim, "q8_0", v_fmt, dtype, seed=ratio + n, v_scale=300.0 if dtype == "f16" else 3e3)
            b = blocks_of(c.v, v_fmt)[:, 1::2, :2]
            d = np.ascontiguousarray(b).view(np.float16)
            d = np.where(np.isfinite(d), d.astype(np.float32) * 2.0 ** -ratio, d).astype(np.float16)
            b[:] = d.view(np.uint8).reshape(b.shape)
            again(c)
            out = c.run(lib)
            c.check(out)
            if dtype == "f16":
                continue  # the small channels' results are among fp16's subnormals: held by the bound alone
            small = (np.arange(head_dim) // 32) % 2 == 1
            got, want = out[:n, :c.heads].double().cpu().numpy()[..., small], c.want[:n][..., small]
            # half of fp16's smallest step in each product, as in element_bound: relative to the large blocks' scales
            least = (n + 60) * 2.0 ** -38 * largest_scale(v_fmt, c.v[rows_of(c, 0)]) * (8 if v_fmt == "q4_0" else 128)
            norm = np.linalg.norm(want)
            l2 = np.linalg.norm(got - want) / norm
            say(f"  small channels rel_l2 {l2:.2e}")
            assert l2 <= ref.l2_bound(dtype) + least * want.size ** 0.5 / norm


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k_fmt", ["q4_0", "q8_0"])
def test_attn_infinite_key_scale(lib, k_fmt, dtype):  # noqa: F811
    """A row that sees a cell with an infinite key scale has no finite result, whatever the signs of its codes; others do."""
    import torch
    for n, cells, at in ((1, 60, 20), (3, 1500, 700), (70, 130, 50), (80, 1300, 100)):
        for code in (0x00, 0x99, 0xFF):
            for bits in (INF, INF | 0x8000):
                say(f"attn infinite key scale {k_fmt} {dtype} n={n} cells={cells} codes {code:x}")
                c = Case([(n, cells), (1, 40)], 4, 2, 128, k_fmt, "q4_0", dtype, seed=3)
                c.qt = torch.ones_like(c.qt)
                blocks_of(c.k, k_fmt)[rows_of(c, 0)[at], :, 2:] = code
                set_scales(c.k, k_fmt, rows_of(c, 0)[[at]], bits)
                out = c.run(lib)
                assert not torch.any(torch.isfinite(out[:n, :c.heads])).item()
                assert torch.all(torch.isfinite(out[n:])).item()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k_fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("n", [1, 4, 70])
def test_attn_large_scores(lib, n, k_fmt, dtype):  # noqa: F811
    """Queries and keys with means of their own: scores of hundreds and thousands that differ little from each other, where the
    fp32 rounding of a score, 2^-24 of its size, changes every probability by as much. The header's limits hold to scores of 100
    and grow with them from there: 2^-24 of 100 is 6e-6 of its 1e-5."""
    for head_dim in (64, 128, 256):
        for k_mean, q_mean in ((0, 0), (2, 2), (10, 3), (20, 10), (5, 40)):
            c = Case([(n, 300 + n)], 4, 2, head_dim, k_fmt, "q8_0", dtype, seed=n + head_dim)
            rng, rows = np.random.default_rng(n), rows_of(c, 0)
            c.k[rows] = oracle.quantize(k_fmt, (k_mean + rng.standard_normal((len(rows), 2 * head_dim))).astype(np.float32))
            c.qt = (q_mean + 0.3 * torch_of(rng.standard_normal(c.qt.shape))).to(torch_type(dtype))
            again(c)
            kd = oracle.dequant(k_fmt, c.k[rows], len(rows), 2 * head_dim)
            qd = c.qt.double().numpy()[:, 1:1 + c.heads]
            top = max(np.abs(kd[:, (h // 2) * head_dim:(h // 2 + 1) * head_dim] @ qd[:, h].T).max() for h in range(4)) * c.scale
            out = c.run(lib)[:n, :c.heads].double().cpu().numpy()
            l2 = np.linalg.norm(out - c.want) / np.linalg.norm(c.want)
            limit = ref.L2[dtype] * max(1.0, top / 100) + ref.EPS[dtype] / 2
            say(f"attn large scores {head_dim} {k_fmt} {dtype} n={n} up to {top:.0f}: rel_l2 {l2:.2e} of {limit:.2e}")
            assert np.all(np.abs(out - c.want) <= c.bound) and l2 <= limit


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 70])
def test_attn_largest_scores(lib, n, dtype):  # noqa: F811
    """Scores near the limit of 2^22 and the largest V scales: finite means of the values that are seen."""
    import torch
    for head_dim in (64, 128, 256):
        say(f"attn largest scores {head_dim} {dtype} n={n}")
        c = Case([(n, 300 + n)], 4, 2, head_dim, "q8_0", "q4_0", dtype, seed=2, q_scale=1e4 / head_dim ** 0.5, scale=80.0,
                 v_scale=1e4 if dtype == "f16" else 5e4)
        out = c.run(lib)[:n, :c.heads].double()
        vd = oracle.dequant("q4_0", c.v[rows_of(c, 0)], 300 + n, 2 * head_dim)
        assert np.all(np.isfinite(vd))
        assert torch.all(torch.isfinite(out)).item()
        assert float(out.abs().max()) <= np.abs(vd).max() * (1 + ref.EPS[dtype]) * (1 + 2.0 ** -10)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 4, 70])
def test_attn_queries_that_are_not_finite(lib, n, dtype):  # noqa: F811
    """A query row with a NaN or an infinity has no finite result; every other row has the one it has without it."""
    import torch
    for head_dim in (64, 128, 256):
        for bad in (float("nan"), float("inf"), -float("inf")):
            say(f"attn query {bad} {head_dim} {dtype} n={n}")
            c = Case([(n, 90 + n), (1, 700)], 4, 2, head_dim, "q4_0", "q8_0", dtype, seed=6)
            whole = c.run(lib)
            c.qt[n - 1, 1 + 2, 5] = bad
            out = c.run(lib)
            hit = torch.zeros_like(whole, dtype=torch.bool)
            hit[n - 1, 2] = True
            assert not torch.any(torch.isfinite(out[hit])).item() and torch.equal(out[~hit], whole[~hit])


def test_attn_more_tokens_than_there_are(lib):  # noqa: F811
    """Starts past the tokens: a sequence has no more tokens than q has rows, counted from its first."""
    c = Case([(6, 40), (0, 33)], 4, 2, 64, seed=8)
    c.start[:] = [0, 9, 7]
    for max_q in (6, 9, 100):
        say(f"attn starts past the tokens, max_q {max_q}")
        out = c.run(lib, max_q=max_q)
        c.start[-1] = 6
        c.check(out)
        c.start[:] = [0, 9, 7]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k_fmt,v_fmt", [("q4_0", "q4_0"), ("q8_0", "q4_0"), ("q4_0", "q8_0"), ("q8_0", "q8_0")])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_error_before_the_outputs_rounding(lib, head_dim, k_fmt, v_fmt, dtype):  # noqa: F811
    """The header's limits without the slack of a whole half step: what the output's rounding does to these very answers is
    measured on the exact ones (a tenth is left for the two being rounded apart)."""
    import torch
    for n in (1, 5, 140):
        c = Case([(n, 400 + n), (n, 97 + n)], 8, 2, head_dim, k_fmt, v_fmt, dtype, page=32, seed=n)
        out = c.run(lib)[:2 * n, :c.heads].double().cpu().numpy()
        rounded = torch.from_numpy(c.want).to(torch_type(dtype)).double().numpy()
        norm = np.linalg.norm(c.want)
        own, l2 = np.linalg.norm(rounded - c.want) / norm, np.linalg.norm(out - c.want) / norm
        say(f"attn error {head_dim} {k_fmt} {v_fmt} {dtype} n={n}: rel_l2 {l2:.2e}, {own:.2e} of it the rounding")
        assert l2 <= 1.1 * own + ref.L2[dtype]
