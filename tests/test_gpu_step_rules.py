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


@pytest.mark.parametrize("seqs,tokens", [(1, 1), (3, 2), (5, 7), (2, 33)])
def test_a_steps_results_fit_the_calls_behind(lib, seqs, tokens):
    """What page_step allocates goes into kv_store (slots at 16 bytes), rope and attn as it is, whatever the sizes."""
    import torch
    page, pages, heads, D = 16, 20, 2, 64
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv, table = ints([0] * seqs), torch.full((seqs, 4), -1, dtype=torch.int32, device="cuda")
    q_start, slots, positions, _, status = lib.page_step(kv, ints([tokens] * seqs), table, ints(list(range(pages))), ints([pages]), page,
                                                         seqs * tokens + 1)
    assert status.tolist() == [0] * seqs and slots.data_ptr() % 16 == 0
    n = seqs * tokens + 1
    x = torch.randn(n, heads, D, device="cuda")
    q, k = lib.rope(x, x.clone(), positions, lib.rope_freq(D))
    caches = [torch.zeros((pages * page, lib.row_bytes("q8_0", heads * D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    lib.kv_store("q8_0", "q8_0", k, x, slots, *caches)
    out = lib.attn("q8_0", "q8_0", q, *caches, table, q_start, kv, heads, page, max_q=tokens)
    assert torch.isfinite(out).all().item() and out[:-1].any(-1).all().item()
    with pytest.raises(lib.QmatError) as e:  # a slice that begins between 16 bytes
        lib.kv_store("q8_0", "q8_0", k, x, torch.cat((slots[:1], slots))[1:], *caches)
    assert e.value.status == 5


def test_a_request_that_never_fits_holds_up_those_behind_it(lib):
    """As the header says: its tokens count while it asks for them, and no longer when its add is 0."""
    import torch
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for large in (65, 40):  # more than its four pages of 16 hold; more than a step has
        kv, table = ints([5, 0, 7]), ints([[0, -1, -1, -1], [-1] * 4, [1, -1, -1, -1]])
        free, count, add = ints(list(range(2, 12)) + [0, 0]), ints([10]), ints([1, large, 1])
        for _ in range(2):
            got = lib.page_step(kv, add, table, free, count, 16, 32)
            assert got[4].tolist() == [0, 1, 1]
        add[1] = 0
        got = lib.page_step(kv, add, table, free, count, 16, 32)
        assert got[4].tolist() == [0, 0, 0] and kv.tolist() == [8, 0, 8] and count.tolist() == [10]
