"""A step's calls through the binding where buffers meet: what is refused leaves
every tensor as it was, what the next call takes fits it."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_qmat_amd as qmat
    qmat.library_path()
    return qmat


@pytest.mark.parametrize("K", [64, 4096, 20000])
@pytest.mark.parametrize("want", ["rows", "both"])
def test_norm_refuses_rows_over_the_residual(lib, want, K):
    """rows over x and the sum over x, each allowed, would leave one tensor for both."""
    import torch
    x, r = torch.randn(3, K, device="cuda"), torch.randn(3, K, device="cuda")
    w, h = torch.ones(K, device="cuda"), torch.zeros(3, K, device="cuda")
    before = [t.clone() for t in (x, r, h)]
    for kw in ({"residual_out": x, "rows": x}, {"residual_out": h, "rows": h}, {"residual_out": r, "rows": r}, {"rows": r}):
        with pytest.raises(lib.QmatError) as e:
            lib.rms_norm(x, w, residual=r, want=want, **kw)
        assert e.value.status == 2
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((x, r, h), before))
