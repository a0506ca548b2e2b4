"""The ways of dividing attention over the quantized cache that only many cells or
many sequences take: a row's parts joined by a whole workgroup, and a wave, or two,
for each head. That a batch takes the way it is meant for shows in its workspace.
"""
import numpy as np
import pytest

from test_gpu_kv_attn import DTYPES, Case, dev, lib, say  # noqa: F401

pytestmark = pytest.mark.gpu


def needed(c, max_kv):
    """Workspace bytes of c's call."""
    import block_quantized_weight_qmat_amd as qmat
    q = c.qt.cuda()[:, 1:1 + c.heads]
    return qmat.attn_workspace_bytes(qmat.attn_args(c.k_fmt, c.v_fmt, q, dev(c.k), dev(c.v), dev(c.table), dev(c.start), dev(c.kv_len),
                                                    c.kv_heads, c.page, q.clone(), max_q=max(n for n, _ in c.seqs), max_kv=max_kv))


def shares(c, max_kv):
    """The shares that c's cells are divided into, from the workspace's size: partial rows of D + 2 numbers for shares + items of
    them, and a number for each item and one more."""
    rows = max(n for n, _ in c.seqs) * c.heads // c.kv_heads
    items = len(c.seqs)
    assert rows <= 16
    left, none = divmod(needed(c, max_kv) - 4 * (items + 1), c.kv_heads * rows * (c.head_dim + 2) * 4)
    assert none == 0
    return left - items


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_one_sequence_in_many_shares(lib, head_dim, dtype):  # noqa: F811
    """A long sequence whose parts are joined by a whole workgroup per row (more than 32 parts), drafted tokens among them."""
    for n in (1, 3):
        c = Case([(n, 16000 + n)], 4, 2, head_dim, "q8_0", "q4_0", dtype, page=64, seed=head_dim)
        s = shares(c, None)
        say(f"attn many shares {head_dim} {dtype} n={n}: {s}")
        assert s > 32
        c.check(c.run(lib))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,seqs,per_group", [(16, 8, 33, 4), (12, 6, 45, 2), (4, 2, 132, 2)])
def test_attn_wave_per_head(lib, heads, kv_heads, seqs, per_group, head_dim, dtype):  # noqa: F811
    """Batches large enough that a wave, or two, take a head each: ragged and empty sequences, shares that end inside them."""
    rng = np.random.default_rng(seqs)
    for page, n in ((16, 1), (64, 3)):
        lens = [(n, int(x)) for x in rng.integers(0, 500, seqs)]
        lens[0], lens[1], lens[2], lens[seqs // 2], lens[-1] = (n, 4000), (1, 0), (n, 1), (n, 0), (2, 1500)
        c = Case(lens, heads, kv_heads, head_dim, "q4_0", "q8_0" if page == 16 else "q4_0", dtype, page=page, pad=1, seed=seqs)
        s = shares(c, 4000)
        say(f"attn wave per head {heads}/{kv_heads} x {head_dim} {dtype} page {page}: {s} shares")
        assert s == 512 // (kv_heads // per_group)
        c.check(c.run(lib, max_kv=4000))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_wave_per_head_undivided(lib, head_dim, dtype):  # noqa: F811
    """Many sequences of few cells, whose items nobody shares: a wave each for four cache heads."""
    rng = np.random.default_rng(7)
    lens = [(1 + int(x) % 2, int(x)) for x in rng.integers(0, 40, 300)]
    lens[5], lens[299] = (0, 9), (1, 200)
    c = Case(lens, 16, 8, head_dim, "q8_0", "q4_0", dtype, seed=head_dim)
    say(f"attn wave per head, undivided {head_dim} {dtype}")
    assert needed(c, 256) == 0
    c.check(c.run(lib, max_kv=256))
