"""Low-rank adapters of many requests on the GPU, against the formula in 64
bits, element by element.

Bound, by arithmetic: a code times an element of a is exact; a block's 32
products are added in fp32 by the matrix cores, each step at most 2^-23 of the sum of
sizes: 2^-18 together; the blocks are scaled and added in fp32 (K / 32 steps of 2^-24, and as
many parts at most), the R products with b likewise, then the scale and the
sum with base. So an element is off by at most
  |s| sum_r |b_r| Z_r (2^-18 + (K / 32 + R + 16) 2^-24) + 2^-24 |y|,
Z_r = sum_k |a_rk| |x_k|."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

# Rows of this many elements are too long for the kernel that takes a token at a time, so the one
# for tiles of tokens takes them however few tokens there are; 513 blocks are no whole chunks.
LONG = 16416


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_qmat_amd as qmat
    qmat.library_path()
    return qmat


def torch_type(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


class Case:
    """lens: tokens of each sequence; of: its adapter; tail: tokens of no sequence behind the last one."""

    def __init__(self, lens, of, adapters, rank, K, M, dtype="bf16", ranks=None, tail=0, scaled=True, seed=0, lead=0):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.lens, self.of, self.rank, self.K, self.M, self.lead = lens, of, rank, K, M, lead
        self.n = lead + sum(lens) + tail
        self.x = oracle.quantize("q8_0", torch.randn(self.n, K, generator=g).numpy()) if K else np.zeros((self.n, 0), np.uint8)
        self.a = (torch.randn(adapters, rank, K, generator=g) / max(K, 1) ** 0.5).to(torch_type(dtype))
        self.b = (torch.randn(adapters, M, rank, generator=g) / rank ** 0.5).to(torch_type(dtype))
        self.scale = 0.5 + torch.rand(adapters, generator=g) if scaled else None
        self.ranks = ranks
        self.base = torch.randn(self.n, M, generator=g)
        self.starts = [lead]
        for n in lens:
            self.starts.append(self.starts[-1] + n)

    def formula(self):
        """(y, bound, has an adapter) in fp64."""
        y, bound, has = self.base.double().numpy().copy(), np.zeros((self.n, self.M)), np.zeros(self.n, dtype=bool)
        x = oracle.dequant("q8_0", self.x, self.n, self.K).reshape(self.n, self.K) if self.K else np.zeros((self.n, 0))
        for i, a in enumerate(self.of):
            t = slice(self.starts[i], self.starts[i + 1])
            if not 0 <= a < self.a.shape[0]:
                continue
            R = self.rank if self.ranks is None else max(0, min(self.rank, self.ranks[a]))
            if R == 0:
                continue
            has[t] = True
            A, B = self.a[a, :R].double().numpy(), self.b[a, :, :R].double().numpy()
            s = 1.0 if self.scale is None else float(self.scale[a])
            y[t] += s * (x[t] @ A.T) @ B.T
            bound[t] = abs(s) * ((np.abs(x[t]) @ np.abs(A).T) @ np.abs(B).T) * (2.0 ** -18 + (self.K / 32 + R + 16) * 2.0 ** -24)
        return y, bound + 2.0 ** -24 * np.abs(y), has

    def run(self, lib, max_q=None, in_place=False, pad=0, **kw):
        import torch
        dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        buf = torch.full((self.n, self.M + pad), 7.0, device="cuda")
        y = buf[:, :self.M]
        base = None
        if in_place:
            y.copy_(self.base)
        else:
            base = torch.full((self.n, self.M + pad), 5.0, device="cuda")[:, :self.M]
            base.copy_(self.base)
        got = lib.lora(torch.from_numpy(self.x).cuda(), self.a.cuda(), self.b.cuda(), dev(self.of), dev(self.starts), y, base=base,
                       scale=None if self.scale is None else self.scale.cuda(), ranks=None if self.ranks is None else dev(self.ranks),
                       max_q=max(self.lens, default=0) if max_q is None else max_q, **kw)
        assert got.data_ptr() == y.data_ptr()
        assert torch.all(buf[:, self.M:] == 7.0).item()
        return got

    def check(self, lib, **kw):
        import torch
        y, bound, has = self.formula()
        got = self.run(lib, **kw)
        err = np.abs(got.double().cpu().numpy() - y)
        assert np.all(err <= bound), f"{np.nanmax(err / bound)} of the bound"
        assert torch.equal(got.cpu()[~torch.from_numpy(has)], self.base[~torch.from_numpy(has)])
        return got


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("rank,K,M", [(8, 32, 1), (16, 64, 16), (24, 1024, 100), (40, 96, 257), (64, 4096, 64), (128, 320, 33), (136, 256, 31),
                                      (256, 1024, 130), (16, 11008, 40)])
def test_sizes(lib, rank, K, M, max_q, dtype):
    """Both divisions of the work, for the same sequences."""
    Case([1, 3, 1, 30, 2], [0, 2, 1, 0, 2], 3, rank, K, M, dtype, seed=rank + M).check(lib, max_q=max_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_q", [1, 17])
@pytest.mark.parametrize("rank,M", [(8, 1), (16, 257), (24, 100), (32, 31), (40, 64), (64, 600), (72, 33), (136, 20), (256, 130)])
def test_sizes_in_tiles(lib, rank, M, max_q, dtype):
    """Tiles of 16 and of 32 tokens; sequences that start and end inside one."""
    Case([1, 3, 41, 2, 17], [0, 2, 1, 0, 2], 3, rank, LONG, M, dtype, seed=rank + M, tail=2).check(lib, max_q=max_q)


@pytest.mark.parametrize("K", [32 * 8 * 64 + 32 * n for n in (1, 2, 7, 8, 9, 63)])
def test_ends_of_rows(lib, K):
    """Chunks of eight blocks of which the last holds 1 to 8; the last row's end is the buffer's."""
    c = Case([20, 13], [1, 0], 2, 16, K, 40)
    first = c.check(lib)
    assert first.shape == (33, 40)
    Case([1, 1], [1, 0], 2, 64, K, 40, "f16").check(lib)


@pytest.mark.parametrize("lens,rank,K", [([700, 1, 300, 5], 24, 1056), ([4096], 8, 512), ([1] * 500, 64, 11008), ([1000, 64, 1, 1, 1, 999], 64, 1024)])
def test_many_tokens(lib, lens, rank, K):
    r = np.random.default_rng(len(lens))
    Case(lens, r.integers(-1, 4, len(lens)).tolist(), 4, rank, K, 72, seed=rank, tail=1).check(lib)


@pytest.mark.parametrize("seqs", [1, 2, 15, 16, 17, 64, 200])
def test_decode(lib, seqs):
    r = np.random.default_rng(seqs)
    Case([1] * seqs, r.integers(-1, 24, seqs).tolist(), 23, 16, 512, 300, seed=seqs).check(lib)


@pytest.mark.parametrize("max_q", [1, 4, 5, 70])
def test_all_adapters_different(lib, max_q):
    """As many adapters as tokens, in one tile and over several; none of them shares a column."""
    Case([1] * 70, list(range(70)), 70, 8, 256, 70).check(lib, max_q=max_q)
    Case([1] * 70, list(range(69, -1, -1)), 70, 24, 96, 36, "f16").check(lib, max_q=max_q)
    Case([1] * 70, list(range(70)), 70, 8, LONG, 36).check(lib, max_q=max_q)


@pytest.mark.parametrize("lens", [[33], [1, 100, 1], [0, 17, 0, 0, 15, 32, 0], [509, 3, 64, 127], [0, 0]])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompts(lib, lens, dtype):
    r = np.random.default_rng(sum(lens))
    Case(lens, r.integers(0, 3, len(lens)).tolist(), 3, 32, 1056, 132, dtype, tail=3).check(lib)


@pytest.mark.parametrize("K", [160, LONG])
@pytest.mark.parametrize("max_q", [1, 64])
def test_ranks_and_strangers(lib, max_q, K):
    """Smaller ranks, rank 0, numbers outside the range, adapters that are not there, tokens of no sequence."""
    c = Case([2, 1, 20, 5, 1, 1, 3], [0, 1, 2, 3, -1, 4, 5], 5, 48, K, 65, ranks=[48, 5, 17, 0, 1000], tail=4, lead=3)
    c.check(lib, max_q=max_q)
    c.ranks = [-4, 1, 33, 16, 8]
    c.check(lib, max_q=max_q, in_place=True, pad=3)
    c.ranks, c.scale = None, None
    c.of = [2 ** 31 - 1, -2 ** 31, 5, 1, 1, 0, 0]
    c.check(lib, max_q=max_q, pad=4)


@pytest.mark.parametrize("K", [160, LONG])
@pytest.mark.parametrize("max_q", [1, 64])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_others_stay_clean(lib, dtype, max_q, K):
    """NaN and infinities of another adapter, of another token, past a rank and of base stay where they are."""
    import torch
    c = Case([1, 1, 6, 9, 3], [0, 1, 2, 0, -1], 3, 32, K, 50, dtype, ranks=[20, 32, 32])
    want = c.run(lib, max_q=max_q).cpu()
    c.a[0, 20:] = float("nan")
    c.b[0, :, 20:] = float("inf")
    c.a[1, 3, 7] = float("inf")
    c.b[1, 4, 5] = float("nan")
    blocks = c.x.reshape(c.n, -1, 34)
    blocks[3, 1, 0:2] = (0x00, 0x7E)  # token 3, of adapter 2: a NaN scale
    c.base[18, 2] = float("nan")
    got = c.run(lib, max_q=max_q).cpu()
    clean = [0, 2, 4, 5, 6, 7] + list(range(8, 17)) + [17, 19]
    assert torch.equal(got[clean], want[clean])
    assert torch.isnan(got[3]).all().item()
    assert not torch.isfinite(got[1]).any().item()
    keep = [m for m in range(50) if m != 2]
    assert torch.equal(got[18][keep], want[18][keep]) and torch.isnan(got[18, 2]).item()


@pytest.mark.parametrize("K", [160, LONG])
@pytest.mark.parametrize("max_q", [1, 64])
def test_row_strides(lib, max_q, K):
    """Slices of a wider product, 16-byte rows or not; rows behind the last token of any sequence stay."""
    for M, pad in ((64, 64), (64, 1), (63, 1), (30, 2)):
        Case([5, 1, 12], [1, 0, 1], 2, 16, K, M, tail=2).check(lib, max_q=max_q, in_place=True, pad=pad)
        Case([5, 1, 12], [1, 0, 1], 2, 16, K, M, tail=2).check(lib, max_q=max_q, pad=pad)


@pytest.mark.parametrize("K", [160, LONG])
@pytest.mark.parametrize("max_q", [1, 64])
def test_nothing(lib, max_q, K):
    """No adapters, no sequences, no elements, no rows, no tokens."""
    import torch
    Case([3, 1], [0, -1], 0, 8, K, 20).check(lib, max_q=max_q)
    Case([], [], 2, 8, K, 20, tail=5).check(lib, max_q=max_q)
    Case([3, 1], [0, 1], 2, 8, 0, 20).check(lib, max_q=max_q)
    assert Case([3, 1], [0, 1], 2, 8, K, 0).run(lib, max_q=max_q).shape == (4, 0)
    c = Case([0], [0], 1, 8, K, 20)
    assert c.n == 0 and c.run(lib, max_q=max_q).shape == (0, 20)


@pytest.mark.parametrize("K", [160, LONG])
def test_null_where_nothing_is_read(lib, K):
    """Through the C ABI: without adapters their buffers and the activations may be NULL; base is copied."""
    import ctypes
    import torch
    from block_quantized_weight_qmat_amd import binding
    base, y = torch.randn(40, 24, device="cuda"), torch.zeros(40, 24, device="cuda")
    adapter, starts = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([0, 30, 40], dtype=torch.int32, device="cuda")
    for seqs in (2, 0):
        y.zero_()
        args = binding.LoraArgs(1, None, None, None, None, None, adapter.data_ptr() if seqs else None, starts.data_ptr() if seqs else None,
                                base.data_ptr(), y.data_ptr(), 24, 24, 40, seqs, 0, 16, 24, K, 30)
        n = binding.load_library().qmat_lora_workspace_bytes(ctypes.byref(args))
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        assert binding.load_library().qmat_lora(ctypes.byref(args), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(y, base)


@pytest.mark.parametrize("K", [160, LONG])
def test_many_empty_sequences(lib, K):
    """More sequences than one probe of 64 lanes tells apart, and than a grid's rows; all but a few without tokens."""
    lens = [0] * 70001
    for i, n in ((0, 2), (63, 40), (64, 1), (4095, 5), (4096, 33), (69999, 7), (70000, 1)):
        lens[i] = n
    Case(lens, [i % 3 for i in range(len(lens))], 3, 16, K, 20, tail=3).check(lib, max_q=40)


@pytest.mark.parametrize("K", [160, LONG])
@pytest.mark.parametrize("max_q", [1, 64])
def test_bad_starts(lib, max_q, K):
    """Starts that decrease or lie outside the tokens harm no memory, and no token of a sound sequence behind."""
    c = Case([4, 4, 4], [0, 1, 0], 2, 16, K, 40)
    c.starts = [-7, 4, 8, 2 ** 31 - 1]
    got = c.run(lib, max_q=max_q)
    sound = Case([4, 4, 4], [0, 1, 0], 2, 16, K, 40).run(lib, max_q=max_q)
    import torch
    assert torch.equal(got, sound)
    c.starts = [9, 3, -1, 0]
    c.run(lib, max_q=max_q)
    torch.cuda.synchronize()


def test_beside_the_product(lib):
    """What it is for: gemm's Y of a packed matrix, the requests' adapters added in place."""
    import torch
    r = np.random.default_rng(1)
    N, K, M = 37, 1024, 96
    W = oracle.quantize("q4_0", (0.02 * r.standard_normal((M, K))).astype(np.float32))
    c = Case([20, 1, 16], [1, 0, 2], 3, 16, K, M)
    xq = torch.from_numpy(c.x).cuda()
    y = lib.gemm("q4_0", torch.from_numpy(W).cuda(), xq, M, K, N)
    c.base = y.cpu().clone()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = lib.lora(xq, c.a.cuda(), c.b.cuda(), ints(c.of), ints(c.starts), y, scale=c.scale.cuda(), max_q=20)
    want, bound, _ = c.formula()
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)


def test_same_bits_again(lib):
    """Repeated, on another stream and captured: the same bits; a caller's workspace is enough where the call says so."""
    import ctypes
    import torch
    from block_quantized_weight_qmat_amd import binding
    for lens, max_q in (([1] * 40, 1), ([100, 7, 300], 300)):
        c = Case(lens, [i % 3 for i in range(len(lens))], 3, 64, 2048, 200)
        first = c.run(lib, max_q=max_q)
        args = binding.LoraArgs(2, None, None, None, None, None, None, None, None, None, 200, 200, c.n, len(lens), 3, 64, 200, 2048, max_q)
        need = binding.load_library().qmat_lora_workspace_bytes(ctypes.byref(args))
        assert (need > 0) == (max_q > 1)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
        assert torch.equal(c.run(lib, max_q=max_q, workspace=ws), first)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        fixed = (torch.from_numpy(c.x).cuda(), c.a.cuda(), c.b.cuda(), ints(c.of), ints(c.starts))
        base, y, scale = c.base.cuda(), torch.zeros(c.n, 200, device="cuda"), c.scale.cuda()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lib.lora(*fixed, y, base=base, scale=scale, max_q=max_q)
        side.synchronize()
        assert torch.equal(y, first)
        with torch.cuda.graph(graph):
            lib.lora(*fixed, y, base=base, scale=scale, max_q=max_q)
        for _ in range(3):
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, first)
            assert torch.equal(c.run(lib, max_q=max_q), first)


@pytest.mark.parametrize("max_q", [1, 64])
def test_two_calls_at_once(lib, max_q):
    """Calls on two streams, each with its own workspace, give what they give alone."""
    import torch
    cases = [Case([40, 1, 64], [0, 2, 1], 3, 32, LONG, 520, seed=5), Case([1, 64, 33], [1, 0, 2], 3, 32, LONG, 520, seed=6)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    alone = [c.run(lib, max_q=max_q) for c in cases]
    held = [(torch.from_numpy(c.x).cuda(), c.a.cuda(), c.b.cuda(), ints(c.of), ints(c.starts)) for c in cases]
    more = [(c.base.cuda(), c.scale.cuda(), torch.zeros(c.n, 520, device="cuda")) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for h, (base, scale, y), s in zip(held, more, streams):
            with torch.cuda.stream(s):
                lib.lora(*h, y, base=base, scale=scale, max_q=max_q)
    torch.cuda.synchronize()
    for (_, _, y), first in zip(more, alone):
        assert torch.equal(y, first)
