"""Attention over a quantized cache in 64 bits, on the CPU, for the tests:
plain numpy from the definition, with the oracle's dequantized cells."""
import numpy as np

import oracle

EPS = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}  # torch.finfo(t).eps


def seen(n, cells, i, causal, window):
    """Cells [lo, hi) that token i of n sees."""
    at = cells - n + i
    lo = max(0, at - window + 1) if window else 0
    hi = max(0, min(cells, at + 1)) if causal else cells
    return lo, hi


def attention(q, k_rows, v_rows, cell_of, kv_heads, n, cells, scale, causal, window):
    """One sequence. q fp64 [n][heads][D]; k_rows, v_rows fp64 [cache rows][kv_heads * D];
    cell_of: cache row of cell j, -1 for one that counts as not seen.
    Returns out [n][heads][D] and sum_j p_j |v_j| of the same shape."""
    heads, D = q.shape[1:]
    out = np.zeros((n, heads, D))
    mag = np.zeros((n, heads, D))
    for i in range(n):
        lo, hi = seen(n, cells, i, causal, window)
        rows = np.array([cell_of[j] for j in range(lo, hi)], dtype=np.int64)
        rows = rows[rows >= 0] if rows.size else rows
        if rows.size == 0:
            continue
        for h in range(heads):
            c = slice(h // (heads // kv_heads) * D, (h // (heads // kv_heads) + 1) * D)
            s = scale * (k_rows[rows, c] @ q[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ v_rows[rows, c]
            mag[i, h] = p @ np.abs(v_rows[rows, c])
    return out, mag


def element_bound(q, k_blocks_d, z2, n_cells, scale, mag, out, dtype, v_unit):
    """Bound of each output's error, by arithmetic.

    q fp64 [n][heads][D] of one cache head's rows; k_blocks_d: largest |block scale|
    of the keys; z2: the codes' range (15 or 255). A score is a sum of D products q u d
    plus one start value per block, |each| <= |q| z2 d, in fp32: its error is at most
    2^-24 (D + D/32 + 8) of sum |q| z2 d scale; a probability changes by the factor of the
    score's error, once in the numerator and once in the sum (n/32 + 8 additions, 2^-24
    each). Probability times V scale is rounded to 11 bits (half a step 2^-11; a pair of
    fp16: 2^-22); prompts of 16-bit types round the probability and code times V scale, each to
    11 bits, 2 * 2^-11 together. And by half of fp16's smallest step, 2^-25, where it is tiny; these numbers
    are scaled so that 2^14 stands for probability 1 (relative to the largest) times a power of
    two below 2 d_max, so that is 2^-38 d_max for each cell, times the code: v_unit = d_max * 8
    (Q4_0) or * 128 (Q8_0). It shows where one cell dominates a row and its code is 0. Then the output's own rounding, half a step: a half of eps
    relative to the value, and for fp16 at least half of its smallest step, 2^-25 (an
    element of a row that one cell dominates, where that cell's code is 0, is that small)."""
    D = q.shape[-1]
    amp = np.abs(q).sum(-1, keepdims=True) * z2 * k_blocks_d * scale
    score = 2.0 ** -24 * (D + D / 32 + 8) * amp + 2.0 ** -22 * (1 + amp)
    rel = 2 * np.expm1(score) + 2.0 ** -24 * (n_cells / 16 + 40)
    rel = rel + (2.0 ** -21 if dtype == "f32" else 2.0 ** -10 + 2.0 ** -20)
    least = 2.0 ** -25 if dtype == "f16" else 1e-30
    rel_least = n_cells * 2.0 ** -38 * v_unit
    return rel_least + rel * mag + np.abs(out) * EPS[dtype] / 2 * (1 + 2.0 ** -8) + least


#: Relative L2 error against exact arithmetic before the output's rounding, as the
#: header states it; half a step of the output's type comes on top.
L2 = {"f32": 1e-5, "f16": 5e-4, "bf16": 5e-4}


def l2_bound(dtype):
    return L2[dtype] + EPS[dtype] / 2


def random_cache(rng, fmt, cells, dim, scale=1.0):
    """Packed cells of N(0, scale^2) rows and their values in 64 bits."""
    rows = (scale * rng.standard_normal((cells, dim))).astype(np.float32)
    packed = oracle.quantize(fmt, rows)
    return packed, oracle.dequant(fmt, packed, cells, dim)


def poison(packed, fmt, rows):
    """Gives the named cells scales of NaN and infinities and codes of any value."""
    bb = oracle.block_bytes(fmt)
    blocks = packed.reshape(packed.shape[0], -1, bb)
    bits = np.array([0x7E00, 0x7C00, 0xFC00, 0xFFFF], dtype=np.uint16)
    for x, r in enumerate(rows):
        blocks[r, :, 2:] = 0xFF - x % 7
        blocks[r, :, 0:2] = np.frombuffer(bits[(x + np.arange(blocks.shape[1])) % 4].tobytes(),
                                          dtype=np.uint8).reshape(-1, 2)
    return packed
