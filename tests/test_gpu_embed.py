"""Rows of a packed matrix by id on the GPU, against the oracle's dequantized
values in 64 bits.

Q4_0, Q8_0 and Q6_K values have at most 24 significant bits (an fp16 scale of
11, a code of up to 7, a sub-scale of 7 with a 6-bit code), so fp32 holds them
exactly; a Q4_K value is the difference of two exact products, rounded once.
So an fp32 result is the oracle's value rounded, and a 16-bit one that rounded
again: both are compared bit for bit."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

FMTS = ("q4_0", "q8_0", "q4_k", "q6_k")
DTYPES = ("f32", "f16", "bf16")


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_qmat_amd as qmat
    qmat.library_path()
    return qmat


def torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def table(fmt, rows, K, seed):
    W = (0.02 * np.random.default_rng(seed).standard_normal((rows, K))).astype(np.float32)
    W[0, :32] = 0.0
    packed = oracle.quantize(fmt, W).reshape(rows, -1)
    return packed, oracle.dequant(fmt, packed, rows, K).reshape(rows, K)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,blocks,n", [(1, 1, 1), (37, 3, 5), (300, 5, 1000)])
def test_rows(lib, fmt, dtype, rows, blocks, n):
    import torch
    K = blocks * oracle.block_elems(fmt)
    packed, want = table(fmt, rows, K, rows + blocks)
    rng = np.random.default_rng(n)
    ids = rng.integers(0, rows, n).astype(np.int32)
    if n > 3:
        ids[1], ids[2], ids[3] = -1, rows, 2 ** 31 - 1
    out = torch.full((n, K + 16), 9.0, dtype=torch_type(dtype), device="cuda")
    got = lib.embed(fmt, torch.from_numpy(packed).cuda(), K, torch.from_numpy(ids).cuda(), dtype=torch_type(dtype),
                    out=out[:, :K])
    there = (ids >= 0) & (ids < rows)
    w = np.where(there[:, None], want[np.where(there, ids, 0)], 0.0).astype(np.float32)
    assert torch.equal(got.cpu(), torch.from_numpy(w).to(torch_type(dtype)))
    assert torch.all(out[:, K:] == 9.0).item()


@pytest.mark.parametrize("fmt", FMTS)
def test_all_rows_in_order(lib, fmt):
    """Without ids: the way back from quantize()."""
    import torch
    K = 2 * oracle.block_elems(fmt)
    packed, want = table(fmt, 19, K, 3)
    got = lib.embed(fmt, torch.from_numpy(packed).cuda(), K)
    assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)))


def test_any_bytes(lib):
    """Scales and codes that no quantizer writes: negative and subnormal scales, negative sub-scales."""
    import torch
    rng = np.random.default_rng(5)
    for fmt in FMTS:
        K = 3 * oracle.block_elems(fmt)
        packed = rng.integers(0, 256, (65, oracle.row_bytes(fmt, K)), dtype=np.uint8)
        blocks = packed.reshape(65, 3, -1)
        d = (rng.standard_normal((65, 3)) * 10.0 ** rng.integers(-7, 1, (65, 3))).astype(np.float16)
        blocks[..., 0:2] = d[..., None].view(np.uint8)
        if fmt == "q4_k":
            blocks[..., 2:4] = d[:, ::-1, None].copy().view(np.uint8)
        want = oracle.dequant(fmt, packed, 65, K).reshape(65, K).astype(np.float32)
        got = lib.embed(fmt, torch.from_numpy(packed).cuda(), K)
        assert torch.equal(got.cpu(), torch.from_numpy(want)), fmt


def test_rows_past_4_gib(lib):
    """A matrix whose last rows lie past 32-bit offsets, in bytes read and written."""
    import torch
    K, rows = 8192, 520000  # 4.5 GB of Q8_0
    blocks = torch.zeros((rows, lib.row_bytes("q8_0", K)), dtype=torch.uint8, device="cuda")
    x = torch.randn((3, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    blocks[-3:] = lib.quantize("q8_0", x)
    want = lib.embed("q8_0", blocks[-3:], K)
    ids = torch.tensor([rows - 3, 0, rows - 1, rows - 2, rows], dtype=torch.int32, device="cuda")
    got = lib.embed("q8_0", blocks, K, ids)
    zero = torch.zeros_like(want[0])
    for g, w in zip(got, (want[0], zero, want[2], want[1], zero)):
        assert torch.equal(g, w)


def test_nothing_to_do(lib):
    import torch
    t = torch.zeros((4, 34), dtype=torch.uint8, device="cuda")
    assert lib.embed("q8_0", t, 32, torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 32)
    got = lib.embed("q8_0", t[:0], 32, torch.zeros(3, dtype=torch.int32, device="cuda"), dtype=torch.float16)
    assert got.shape == (3, 32) and not got.any().item()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_results(lib, dtype):
    """Results that are written past the caches are those of smaller calls."""
    import torch
    fmt, K, n = "q6_k", 1024, 70001  # 143 MB
    packed, _ = table(fmt, 50, K, 8)
    dev = torch.from_numpy(packed).cuda()
    ids = torch.randint(-1, 51, (n,), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    got = lib.embed(fmt, dev, K, ids, dtype=torch_type(dtype))
    for at in range(0, n, 20000):
        part = ids[at:at + 20000].clone()
        assert torch.equal(got[at:at + 20000], lib.embed(fmt, dev, K, part, dtype=torch_type(dtype)))
