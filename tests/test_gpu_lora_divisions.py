"""Low-rank adapters on the GPU, each division of the work where its loops go
round more than once, against the formula in 64 bits (bound: test_gpu_lora.py).

Which kernel takes a call is the plan's choice from the sizes; a call that takes a
token at a time needs no workspace, tiles of tokens do. Every test says which
one it means."""
import ctypes

import numpy as np
import pytest

from test_gpu_lora import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_qmat_amd as qmat
    qmat.library_path()
    return qmat


def in_tiles(case, max_q=None):
    """Whether a call for this case takes tiles of tokens."""
    from block_quantized_weight_qmat_amd import binding
    dtype = 1 if str(case.a.dtype) == "torch.float16" else 2
    args = binding.LoraArgs(dtype, None, None, None, None, None, None, None, None, None, case.M, case.M, case.n, len(case.lens),
                            case.a.shape[0], case.rank, case.M, case.K, max(case.lens, default=0) if max_q is None else max_q)
    need = binding.load_library().qmat_lora_workspace_bytes(ctypes.byref(args))
    assert need >= 0
    return need > 0


def poisoned(case):
    """The case's codes and adapters on the GPU between numbers that are not to be read as theirs."""
    import torch
    def between(t, fill):
        t = t.cuda()
        whole = torch.full((t.shape[0] + 2, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")
        whole[1:-1] = t
        return whole[1:-1]
    x = torch.from_numpy(case.x).cuda()
    rows = torch.full((case.n * x.shape[1] + 256,), 255, dtype=torch.uint8, device="cuda")  # scales of NaN
    rows[:x.numel()] = x.flatten()
    return rows[:x.numel()].view(x.shape), between(case.a, float("nan")), between(case.b, float("nan"))


def check(lib, case, tiles, max_q=None):
    import torch
    assert in_tiles(case, max_q) == tiles
    want, bound, has = case.formula()
    x, a, b = poisoned(case)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    y = torch.full((case.n + 1, case.M), 7.0, device="cuda")
    got = lib.lora(x, a, b, ints(case.of), ints(case.starts), y[:-1], base=case.base.cuda(),
                   scale=None if case.scale is None else case.scale.cuda(), ranks=None if case.ranks is None else ints(case.ranks),
                   max_q=max(case.lens) if max_q is None else max_q)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= bound), f"{np.nanmax(err / bound)} of the bound"
    assert torch.equal(got.cpu()[~torch.from_numpy(has)], case.base[~torch.from_numpy(has)])
    assert torch.all(y[-1] == 7.0).item()


# many tokens: tiles, however short their rows are
LENS, OF = [900, 1, 33, 700, 0, 16, 397], [0, 2, 1, 3, 0, -1, 2]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("K", [32, 64, 96, 224, 256, 288, 480, 544, 1024])
def test_tiles_of_short_rows(lib, K, dtype):
    """A chunk of eight blocks that one wave, some or all have work in; the last row's end is the buffer's."""
    for max_q in (None, 16):  # tiles of 32 and of 16 tokens
        check(lib, Case(LENS, OF, 4, 16, K, 72, dtype, seed=K, tail=1, lead=2), True, max_q)
        check(lib, Case(LENS, OF, 4, 16, K, 72, dtype, seed=K), True, max_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rank,ranks", [(8, [8, 3, 1, 8]), (24, None), (32, [32, 17, 16, 1]), (40, [33, 40, 32, 9]), (64, None), (72, [65, 72, 64, 40]),
                                        (136, [129, 136, 128, 64]), (256, [256, 255, 193, 70])])
def test_tiles_of_each_rank(lib, rank, ranks, dtype):
    for K, M in ((96, 33), (288, 520)):
        check(lib, Case(LENS, OF, 4, rank, K, M, dtype, ranks=ranks, seed=rank), True)
        check(lib, Case(LENS, OF, 4, rank, K, M, dtype, ranks=ranks, seed=rank), True, 16)


@pytest.mark.parametrize("M", [1, 31, 511, 512, 513, 1025])
def test_tiles_of_many_rows_of_b(lib, M):
    """Parts of M that several workgroups have, the last one with few rows."""
    check(lib, Case(LENS, OF, 4, 24, 128, M, seed=M), True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rank,ranks", [(8, [8, 5, 0]), (24, [24, 17, 9]), (64, None), (128, [128, 121, 66])])
@pytest.mark.parametrize("M", [1023, 1025, 2047, 5000])
def test_a_token_at_a_time_in_many_workgroups(lib, M, rank, ranks, dtype):
    """Rows of b past a workgroup's 1024: blockIdx.y counts."""
    for lens, of in (([1], [0]), ([1, 1, 1], [2, 0, 1]), ([1, 2], [1, 3])):
        check(lib, Case(lens, of, 3, rank, 160, M, dtype, ranks=ranks, seed=M + rank), False, 1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rank,ranks,tokens,M", [(8, [8, 3, 0, 7], 256, 2900), (8, None, 300, 1025), (16, [16, 9, 15, 1], 257, 2049), (24, [24, 23, 8, 17], 300, 2500),
                                                 (40, [40, 33, 39, 1], 260, 1100), (64, None, 256, 1200), (256, [256, 249, 256, 130], 256, 1100)])
def test_a_token_at_a_time_in_several_passes(lib, rank, ranks, tokens, M, dtype):
    """More rows of b than a workgroup has at a time: its waves go on 1024 rows behind, with two loads ahead."""
    r = np.random.default_rng(rank + M)
    check(lib, Case([1] * tokens, r.integers(-1, 4, tokens).tolist(), 4, rank, 64, M, dtype, ranks=ranks, seed=M), False, 1)


@pytest.mark.parametrize("K", [32, 512, 4096, 8192, 16384])
def test_a_token_at_a_time_of_each_length(lib, K):
    """Codes and scales of up to the longest row that this division takes."""
    check(lib, Case([1, 1, 1], [0, 1, 0], 2, 16, K, 1500, ranks=[16, 11], seed=K), False, 1)


def test_in_place_past_1024_rows(lib):
    """base is y: rows of another workgroup, and of the same one's next pass, are still base when they are read."""
    import torch
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for tokens, M in ((2, 5000), (256, 2900)):
        c = Case([1] * tokens, [t % 3 for t in range(tokens)], 3, 8, 64, M, seed=M)
        assert not in_tiles(c)
        want, bound, _ = c.formula()
        y = c.base.cuda()
        lib.lora(torch.from_numpy(c.x).cuda(), c.a.cuda(), c.b.cuda(), ints(c.of), ints(c.starts), y, scale=c.scale.cuda(), max_q=1)
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= bound)
