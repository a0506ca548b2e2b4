"""RMS norm with residual on the GPU, against the formula in 64 bits.

y is the 64-bit formula rounded once to fp32, so the Q8_0 bytes have to be the
oracle's quantization of that number, byte for byte, and rows its rounding to
the type. The kernel's 64-bit value is off by at most about (K + 10) 2^-53 of
itself (K additions of positive terms, the root, the products); where it
lies that near to a rounding border of fp32, y may be the neighbour: a chance of
about (K + 10) 2^-53 / 2^-24 per element, 2^-29 K, below 1e-3 for all elements of
the cases here but the largest."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

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


def formula(x, residual, weight, eps):
    """(h as stored, y rounded to fp32), from tensors on the CPU."""
    import torch
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    d = h.double()
    y = d * (1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + eps)) * weight.double()
    return h, y.float()


def draw(n, K, dtype, seed, pad=16):
    """n rows of K with pad elements between them."""
    import torch
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn(n, K + pad, generator=g)
    buf[:, :K:97] *= 40.0
    return buf.to(torch_type(dtype))


def check(lib, x, residual, weight, eps, want, got):
    import torch
    rows, q8, h = got
    hw, y = formula(x.cpu(), None if residual is None else residual.cpu(), weight.cpu(), eps)
    if residual is not None:
        assert torch.equal(h.cpu(), hw)
    else:
        assert h is None
    if want != "q8":
        assert torch.equal(rows.cpu(), y.to(x.dtype))
    if want != "rows":
        assert np.array_equal(q8.cpu().numpy(), oracle.quantize("q8_0", y.numpy()))


@pytest.mark.parametrize("want,with_residual", [("q8", True), ("rows", False), ("both", True), ("both", False)])
@pytest.mark.parametrize("dtype", DTYPES)
# a wave for a row, and each larger split at its edges; rows read twice from 16416 on
@pytest.mark.parametrize("n,K", [(1, 32), (5, 96), (3, 512), (2, 544), (7, 1024), (3, 1056), (2, 2080), (3, 4096), (2, 4128), (2, 8224),
                                 (1, 16384), (2, 16416), (1, 40000)])
def test_formula(lib, n, K, dtype, want, with_residual):
    import torch
    x = draw(n, K, dtype, n + K).cuda()[:, :K]
    r = draw(n, K, dtype, n * K + 1, 32).cuda()[:, :K] if with_residual else None
    w = (1 + 0.3 * torch.randn(K, generator=torch.Generator().manual_seed(3))).cuda()
    check(lib, x, r, w, 1e-5, want, lib.rms_norm(x, w, eps=1e-5, residual=r, want=want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [255, 1025])
def test_many_rows(lib, n, dtype):
    import torch
    x, r = draw(n, 320, dtype, n).cuda()[:, :320], draw(n, 320, dtype, n + 1).cuda()[:, :320]
    w = torch.rand(320, generator=torch.Generator().manual_seed(4)).cuda()
    check(lib, x, r, w, 1e-6, "both", lib.rms_norm(x, w, residual=r, want="both"))


@pytest.mark.parametrize("K", [256, 4096, 20000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place(lib, K, dtype):
    """h over the residual and rows over x; h over x. What lies between rows stays."""
    import torch
    w = torch.ones(K, device="cuda")
    for over in ("residual", "x"):
        xb, rb = draw(3, K, dtype, 1).cuda(), draw(3, K, dtype, 2).cuda()
        x0, r0 = xb[:, :K].clone(), rb[:, :K].clone()
        x, r = xb[:, :K], rb[:, :K]
        gaps = (xb[:, K:].clone(), rb[:, K:].clone())
        if over == "residual":
            got = lib.rms_norm(x, w, residual=r, residual_out=r, rows=x, want="both")
            assert got[0].data_ptr() == x.data_ptr() and got[2].data_ptr() == r.data_ptr()
        else:
            got = lib.rms_norm(x, w, residual=r, residual_out=x, want="both")
            assert torch.equal(r, r0)
        check(lib, x0, r0, w, 1e-6, "both", got)
        assert torch.equal(xb[:, K:], gaps[0]) and torch.equal(rb[:, K:], gaps[1])


def test_extremes(lib):
    """Rows of zeros, of the largest and of the smallest numbers; no eps; a row of NaN beside others."""
    import torch
    K = 128
    x = torch.randn(7, K, generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1] *= 1e37
    x[2] *= 1e-42
    x[3] = 0.0
    x[3, 5] = -2.0
    w = torch.ones(K)
    for eps in (0.0, 1e-6):
        rows, q8, _ = lib.rms_norm(x.cuda(), w.cuda(), eps=eps, want="both")
        _, y = formula(x, None, w, eps)
        first = 1 if eps == 0.0 else 0  # 0 / 0: unspecified bytes, NaN in rows
        assert torch.equal(rows[first:].cpu(), y[first:])
        assert np.array_equal(q8[first:].cpu().numpy(), oracle.quantize("q8_0", y[first:].numpy()))
        if eps == 0.0:
            assert torch.isnan(rows[0]).all().item()
    x[4, 3], x[5, 7] = float("nan"), float("inf")
    rows, q8, _ = lib.rms_norm(x.cuda(), w.cuda(), want="both")
    _, y = formula(x, None, w, 1e-6)
    assert torch.isnan(rows[4]).all().item() and torch.isnan(rows[5, 7]).item() and torch.isfinite(rows[5, :7]).all().item()
    keep = [0, 1, 2, 3, 6]
    assert torch.equal(rows[keep].cpu(), y[keep])
    assert np.array_equal(q8[keep].cpu().numpy(), oracle.quantize("q8_0", y[keep].numpy()))


def test_nothing_to_do(lib):
    import torch
    x = torch.zeros((0, 64), device="cuda")
    rows, q8, h = lib.rms_norm(x, torch.ones(64, device="cuda"), residual=x, want="both")
    assert rows.shape == (0, 64) and q8.shape == (0, 68) and h.shape == (0, 64)


def test_more_rows_than_a_launch(lib):
    """Rows past the 2^21 of one launch, and past 2^32 bytes of each buffer, get what the same rows alone get."""
    import torch
    n, K = (1 << 21) + 70001, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, K, device="cuda", generator=g, dtype=torch.float16)
    w = torch.rand(K, device="cuda", generator=g)
    rows, q8, _ = lib.rms_norm(x, w, want="both")
    for at in (0, (1 << 21) - 3, n - 5):
        part = lib.rms_norm(x[at:at + 5].clone(), w, want="both")
        assert torch.equal(rows[at:at + 5], part[0]) and torch.equal(q8[at:at + 5], part[1])
