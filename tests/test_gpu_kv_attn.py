"""The quantized KV cache on the GPU: storing rows, loading them, attention.

Stored bytes equal the oracle's quantizer; loaded values equal the oracle's
dequantized ones rounded once; attention is held to the 64-bit formula within
kv_reference's bounds, which are derived there. Outputs are prefilled with a
sentinel, so that an element that should be written and is not fails, and one
that should not be written and is fails too.
"""
import sys

import numpy as np
import pytest

import kv_reference as ref
import oracle

pytestmark = pytest.mark.gpu

FMTS = ("q4_0", "q8_0")
DTYPES = ("f32", "f16", "bf16")


def say(msg):
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


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


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- store and load

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k_fmt", FMTS)
@pytest.mark.parametrize("v_fmt", FMTS)
@pytest.mark.parametrize("n,dim,bias", [(1, 32, False), (3, 96, True), (65, 1024, True), (257, 160, False)])
def test_store_bytes(lib, k_fmt, v_fmt, dtype, n, dim, bias):
    import torch
    say(f"store {k_fmt} {v_fmt} {dtype} n={n} dim={dim} bias={bias}")
    rng = np.random.default_rng(n * dim + len(dtype))
    cells = n + 7
    rows = rng.standard_normal((n, 2 * dim + 32)).astype(np.float32)
    rows[0, :32] = 0.0                       # a zero block
    rows[n - 1, dim:dim + 32] *= 1e-7        # subnormal scales
    kv = torch.from_numpy(rows).to(torch_type(dtype)).cuda()
    k, v = kv[:, :dim], kv[:, dim:2 * dim]   # slices of one projection
    b = rng.standard_normal(dim).astype(np.float32) if bias else None
    slots = rng.permutation(cells)[:n].astype(np.int32)
    if n > 2:
        slots[1], slots[2] = -1, cells       # outside: skipped
    caches = [np.full((cells, oracle.row_bytes(f, dim)), 0xA5, np.uint8) for f in (k_fmt, v_fmt)]
    kc, vc = dev(caches[0]), dev(caches[1])
    lib.kv_store(k_fmt, v_fmt, k, v, dev(slots), kc, vc, k_bias=None if b is None else dev(b))
    torch.cuda.synchronize()
    for x, fmt, cache, got, sub in ((k, k_fmt, caches[0], kc, b), (v, v_fmt, caches[1], vc, None)):
        x = x.float().cpu().numpy()
        want = cache.copy()
        packed = oracle.quantize(fmt, x if sub is None else x - sub)
        for i, s in enumerate(slots):
            if 0 <= s < cells:
                want[s] = packed[i]
        assert np.array_equal(got.cpu().numpy(), want), f"{fmt} bytes differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k_fmt", FMTS)
@pytest.mark.parametrize("v_fmt", FMTS)
@pytest.mark.parametrize("n,dim,bias", [(1, 32, True), (5, 96, False), (130, 1024, True)])
def test_load_values(lib, k_fmt, v_fmt, dtype, n, dim, bias):
    import torch
    say(f"load {k_fmt} {v_fmt} {dtype} n={n} dim={dim} bias={bias}")
    rng = np.random.default_rng(7 * n + dim)
    cells = 41
    (kp, kd), (vp, vd) = (ref.random_cache(rng, f, cells, dim) for f in (k_fmt, v_fmt))
    b = rng.standard_normal(dim).astype(np.float32) if bias else None
    slots = rng.integers(0, cells, n).astype(np.int32)  # cells named more than once
    if n > 3:
        slots[2], slots[3] = -5, cells
    out = torch.full((n, 2 * dim + 32), 9.0, dtype=torch_type(dtype), device="cuda")
    lib.kv_load(k_fmt, v_fmt, dev(kp), dev(vp), dev(slots), dim, dtype=torch_type(dtype),
                k_bias=None if b is None else dev(b), k=out[:, :dim], v=out[:, dim:2 * dim])
    torch.cuda.synchronize()
    # a scale times a code is exact in fp32; the sum with the bias rounds once there
    kw, vw = kd.astype(np.float32)[slots % cells], vd.astype(np.float32)[slots % cells]
    if b is not None:
        kw = kw + b
    gone = (slots < 0) | (slots >= cells)
    kw[gone], vw[gone] = 0.0, 0.0
    for got, want in ((out[:, :dim], kw), (out[:, dim:2 * dim], vw)):
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch_type(dtype)))
    assert torch.all(out[:, 2 * dim:] == 9.0).item()


@pytest.mark.parametrize("dtype", DTYPES)
def test_store_load_large(lib, dtype):
    """One call for many rows (several blocks a lane; results past the caches) does what calls for a few do."""
    import torch
    n, dim, cells = 33001, 1056, 33100
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn((n, dim), generator=g, device="cuda").to(torch_type(dtype)) for _ in range(2))
    bias = torch.randn(dim, generator=g, device="cuda")
    slots = torch.randperm(cells, generator=g, device="cuda")[:n].int()
    slots[::997] = -1
    slots[-1] = cells
    caches = [torch.full((cells, oracle.row_bytes(f, dim)), 0xA5, dtype=torch.uint8, device="cuda")
              for f in ("q8_0", "q4_0") * 2]
    say(f"store of {n} rows {dtype}")
    lib.kv_store("q8_0", "q4_0", k, v, slots, *caches[:2], k_bias=bias)
    step = 2000
    for i in range(0, n, step):
        lib.kv_store("q8_0", "q4_0", k[i:i + step], v[i:i + step], slots[i:i + step].clone(), *caches[2:], k_bias=bias)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    say(f"load of {n} rows {dtype}")
    got = lib.kv_load("q8_0", "q4_0", *caches[:2], slots, dim, dtype=k.dtype, k_bias=bias)
    for i in range(0, n, step):
        want = lib.kv_load("q8_0", "q4_0", *caches[:2], slots[i:i + step].clone(), dim, dtype=k.dtype, k_bias=bias)
        assert torch.equal(got[0][i:i + step], want[0]) and torch.equal(got[1][i:i + step], want[1])


# ------------------------------------------------------------------------ attention

def largest_scale(fmt, packed):
    """Largest finite |block scale| of packed rows."""
    bb = oracle.block_bytes(fmt)
    raw = packed.reshape(-1, bb)[:, :2]
    d = np.abs(np.ascontiguousarray(raw).view(np.float16).astype(np.float64))
    return d[np.isfinite(d)].max(initial=0.0)


class Case:
    """A batch with its caches, page table and 64-bit answer. seqs: (new tokens, cells) each."""

    def __init__(self, seqs, heads, kv_heads, head_dim, k_fmt="q4_0", v_fmt="q4_0", dtype="f32", page=16, causal=True,
                 window=0, pad=0, seed=0, q_scale=1.0, v_scale=1.0, bad_pages=(), hurt=(), scale=None):
        rng = np.random.default_rng(seed)
        self.__dict__.update(seqs=seqs, heads=heads, kv_heads=kv_heads, head_dim=head_dim, k_fmt=k_fmt, v_fmt=v_fmt,
                             dtype=dtype, page=page, causal=causal, window=window)
        dim = kv_heads * head_dim
        need = [-(-kv // page) for _, kv in seqs]
        pages = sum(need) + 2
        cells = pages * page
        self.k, kd = ref.random_cache(rng, k_fmt, cells, dim)
        self.v, vd = ref.random_cache(rng, v_fmt, cells, dim, v_scale)
        order = rng.permutation(pages)
        self.table = np.full((len(seqs), max(1, max(need))), 0x7FFFFFFF, np.int32)  # unused: nonsense
        at, used = 0, np.zeros(cells, bool)
        self.start = np.zeros(len(seqs) + 1, np.int32)
        self.kv_len = np.array([kv for _, kv in seqs], np.int32)
        maps = []
        for b, (n, kv) in enumerate(seqs):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            for x in bad_pages:
                if x < need[b]:
                    self.table[b, x] = (-1, pages, -2 ** 31)[(b + x) % 3]
            m = np.array([self.table[b, j // page] * page + j % page if 0 <= self.table[b, j // page] < pages else -1
                          for j in range(kv)], np.int64)
            used[m[m >= 0]] = True
            maps.append(m)
            self.start[b + 1] = self.start[b] + n
        # cells that no token sees hold NaN and infinite scales
        for f, p in ((k_fmt, self.k), (v_fmt, self.v)):
            ref.poison(p, f, np.flatnonzero(~used))
            for b, j in hurt:
                ref.poison(p, f, [maps[b][j]])
        T = int(self.start[-1]) + pad
        q = (q_scale * rng.standard_normal((T, heads + 2, head_dim))).astype(np.float32)
        import torch
        self.qt = torch.from_numpy(q).to(torch_type(dtype))
        qd = self.qt.double().numpy()[:, 1:1 + heads]
        self.scale = head_dim ** -0.5 if scale is None else scale
        self.want, self.bound = np.zeros((T, heads, head_dim)), np.zeros((T, heads, head_dim))
        for b, (n, kv) in enumerate(seqs):
            s = slice(self.start[b], self.start[b + 1])
            o, mag = ref.attention(qd[s], kd, vd, maps[b], kv_heads, n, kv, self.scale, causal, window)
            rows = maps[b][maps[b] >= 0]
            d, dv = (largest_scale(f, p[rows]) for f, p in ((k_fmt, self.k), (v_fmt, self.v)))
            self.want[s] = o
            self.bound[s] = ref.element_bound(qd[s], d, 15 if k_fmt == "q4_0" else 255, max(kv, 1), abs(self.scale), mag, o, dtype,
                                              dv * (8 if v_fmt == "q4_0" else 128))
        self.T = T

    def run(self, lib, **kw):
        import torch
        q = self.qt.cuda()[:, 1:1 + self.heads]  # a slice: rows are heads + 2 apart
        out = torch.full((self.T, self.heads + 1, self.head_dim), 77.0, dtype=q.dtype, device="cuda")
        args = dict(causal=self.causal, window=self.window, scale=self.scale, max_q=max(n for n, _ in self.seqs), out=out[:, :self.heads])
        args.update(kw)
        lib.attn(self.k_fmt, self.v_fmt, q, dev(self.k), dev(self.v), dev(self.table), dev(self.start), dev(self.kv_len),
                 self.kv_heads, self.page, **args)
        torch.cuda.synchronize()
        return out

    def check(self, out):
        import torch
        n = int(self.start[-1])
        assert torch.all(out[:, self.heads:] == 77.0).item() and torch.all(out[n:] == 77.0).item()
        got = out[:n, :self.heads].double().cpu().numpy()
        want, bound = self.want[:n], self.bound[:n]
        assert np.all(np.isfinite(got)), "not finite"
        off = np.abs(got - want)
        worst = float((off / bound).max()) if off.size else 0.0
        norm = np.linalg.norm(want)
        l2 = np.linalg.norm(got - want) / norm if norm else float(off.max(initial=0.0))
        say(f"  worst element {worst:.3f} of its bound, rel_l2 {l2:.2e} of {ref.l2_bound(self.dtype):.2e}")
        assert worst <= 1.0 and l2 <= ref.l2_bound(self.dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k_fmt", FMTS)
@pytest.mark.parametrize("v_fmt", FMTS)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_types(lib, head_dim, k_fmt, v_fmt, dtype):
    say(f"attn {head_dim} {k_fmt} {v_fmt} {dtype}")
    c = Case([(1, 77), (1, 1), (1, 33), (3, 130)], 4, 2, head_dim, k_fmt, v_fmt, dtype, seed=head_dim)
    c.check(c.run(lib))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (7, 1), (16, 1), (20, 1), (40, 2), (6, 2)])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_attn_head_layouts(lib, heads, kv_heads, n):
    say(f"attn heads {heads}/{kv_heads} n={n}")
    c = Case([(n, 70), (n, n), (n, 200)], heads, kv_heads, 64, "q8_0", "q4_0", "f16", seed=heads + n)
    c.check(c.run(lib))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cells", [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_attn_lengths(lib, cells, dtype):
    say(f"attn cells {cells} {dtype}")
    c = Case([(1, cells)], 4, 2, 128, dtype=dtype, seed=cells)
    c.check(c.run(lib))


@pytest.mark.parametrize("page", [1, 2, 16, 64, 1024])
def test_attn_page_sizes(lib, page):
    say(f"attn page {page}")
    c = Case([(1, 300), (2, 100), (1, page)], 4, 2, 64, page=page, seed=page)
    c.check(c.run(lib))


@pytest.mark.parametrize("window", [1, 7, 32, 100, 1000000])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_windows(lib, window, causal):
    say(f"attn window {window} causal={causal}")
    c = Case([(1, 300), (9, 200), (40, 40), (6, 3), (5, 0)], 4, 2, 64, "q8_0", "q8_0", "f16", window=window, causal=causal,
             seed=window % 97)
    c.check(c.run(lib))


def test_attn_not_causal(lib):
    c = Case([(1, 300), (9, 200), (40, 40), (6, 3)], 4, 2, 128, causal=False, seed=3)
    c.check(c.run(lib))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k_fmt,v_fmt", [("q4_0", "q4_0"), ("q8_0", "q4_0"), ("q4_0", "q8_0"), ("q8_0", "q8_0")])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_prompts(lib, head_dim, k_fmt, v_fmt, dtype):
    """Whole prompts, alone and behind cells of earlier ones, odd lengths."""
    say(f"attn prompts {head_dim} {k_fmt} {v_fmt} {dtype}")
    c = Case([(67, 67), (1, 40), (130, 201), (0, 9), (33, 600)], 4, 2, head_dim, k_fmt, v_fmt, dtype, pad=5, seed=head_dim + 1)
    c.check(c.run(lib))


@pytest.mark.parametrize("heads,kv_heads", [(5, 5), (6, 2), (14, 2), (16, 1), (33, 1)])
def test_attn_prompt_head_layouts(lib, heads, kv_heads):
    say(f"attn prompt heads {heads}/{kv_heads}")
    c = Case([(150, 170), (70, 70)], heads, kv_heads, 64, "q4_0", "q8_0", "bf16", seed=heads)
    c.check(c.run(lib))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30, 0.3])
@pytest.mark.parametrize("n", [1, 70])
def test_attn_scales(lib, n, scale):
    """Any finite scale: 0 averages the cells, a negative one prefers the least alike."""
    for dtype in DTYPES:
        say(f"attn scale {scale} n={n} {dtype}")
        c = Case([(n, 300), (n, n - 1), (n, 80)], 4, 2, 64, "q8_0", "q4_0", dtype, window=60, scale=scale, seed=n)
        c.check(c.run(lib))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attn_prompts_shared(lib, head_dim, dtype):
    """Few rows behind many cells: their cells are shared out over workgroups, whole items beside parts of them."""
    for seqs, fmts, kw in (([(70, 1500)], ("q4_0", "q4_0"), {}),
                           ([(33, 1000), (0, 50), (90, 700), (1, 1), (40, 64)], ("q8_0", "q4_0"), {"pad": 3}),
                           ([(80, 900)], ("q8_0", "q8_0"), {"window": 333, "page": 128}),
                           ([(80, 900)], ("q4_0", "q8_0"), {"causal": False, "page": 1, "bad_pages": (0, 400, 401)})):
        say(f"attn prompts shared {head_dim} {dtype} {seqs}")
        c = Case(seqs, 4, 2, head_dim, *fmts, dtype, seed=head_dim + 2, **kw)
        c.check(c.run(lib))
        c.check(c.run(lib, max_kv=10 ** 6))


def test_attn_many_sequences(lib):
    """More sequences than are dealt out together, and a batch where one has many more tokens than the others."""
    rng = np.random.default_rng(41)
    for n, long in ((1100, 1), (400, 20), (90, 300)):
        seqs = [(1, int(x)) for x in rng.integers(0, 40, n)]
        seqs[7], seqs[8] = (long, 280 + long), (0, 12)
        say(f"attn {n} sequences, one of {long} tokens")
        c = Case(seqs, 4, 2, 64, "q4_0", "q8_0", "f16", seed=n)
        c.check(c.run(lib))


def test_attn_no_cells(lib):
    """Empty caches and tables without columns: zeros for every token of a sequence."""
    import torch
    for n in (1, 70):
        for pages, cells in ((0, 0), (0, 32), (3, 0)):
            say(f"attn no cells n={n} pages={pages} cells={cells}")
            q = torch.ones((2 * n, 4, 64), device="cuda")
            out = torch.full_like(q, 3.0)
            kc = torch.zeros((cells, oracle.row_bytes("q8_0", 128)), dtype=torch.uint8, device="cuda")
            lib.attn("q8_0", "q8_0", q, kc, kc.clone(), torch.zeros((2, pages), dtype=torch.int32, device="cuda"),
                     dev(np.array([0, n, 2 * n], np.int32)), dev(np.array([40, 7], np.int32)), 2, 16, out=out)
            assert torch.all(out == 0).item()


def test_attn_sees_a_cell_without_finite_value(lib):
    """Rows that see a cell with infinite and NaN scales have no finite result; the others are exact (checked above)."""
    import torch
    for dtype in DTYPES:
        for n, cells in ((1, 60), (100, 130), (80, 1200)):
            say(f"attn hurt {dtype} n={n}")
            c = Case([(n, cells)], 4, 2, 128, "q8_0", "q4_0", dtype, hurt=[(0, cells - n)], seed=10)
            out = c.run(lib)[:n, :c.heads]
            assert not torch.any(torch.isfinite(out).all(-1)).item()


def test_attn_two_streams(lib):
    """Calls on two streams at once, each with its own workspace, give what they give alone."""
    import torch
    cases = [Case([(1, 3000), (1, 70)], 8, 2, 128, "q8_0", "q4_0", "bf16", page=32, seed=51),
             Case([(70, 1500)], 4, 2, 64, "q4_0", "q4_0", "f16", seed=52)]
    alone = [c.run(lib) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    held = []
    for c in cases:
        q = c.qt.cuda()[:, 1:1 + c.heads]
        held.append((q, dev(c.k), dev(c.v), dev(c.table), dev(c.start), dev(c.kv_len)))
    outs = [[] for _ in cases]
    torch.cuda.synchronize()
    for i in range(6):
        for c, s, h, o in zip(cases, streams, held, outs):
            with torch.cuda.stream(s):
                o.append(lib.attn(c.k_fmt, c.v_fmt, *h, c.kv_heads, c.page, scale=c.scale, max_q=max(n for n, _ in c.seqs)))
    torch.cuda.synchronize()
    for c, a, o in zip(cases, alone, outs):
        for x in o:
            assert torch.equal(x, a[:, :c.heads])


def test_attn_any_numbers_in_q_start_and_kv_len(lib):
    """Starts that fall, are negative or past the tokens, lengths outside the table: nothing but rows of out is written."""
    import torch
    big = 2 ** 31 - 1
    for n, cells, max_q in ((8, 40, 8), (8, 400, 8), (90, 100, 90), (90, 1500, 90)):
        for start in ([3, 1, big, -big, 5, n + 7, n], [-big - 1, -5, 0, 2, big, 1, 0], [0, 2, 2, 4, 4, 6, big]):
            say(f"attn q_start {start} cells {cells}")
            q = torch.ones((n, 8, 64), device="cuda", dtype=torch.bfloat16)
            whole = torch.full((n + 40, 8, 64), 7.0, device="cuda", dtype=torch.bfloat16)
            kc = torch.zeros((2048, oracle.row_bytes("q4_0", 128)), dtype=torch.uint8, device="cuda")
            table = torch.arange(6 * 100, device="cuda").int().reshape(6, 100) % 128
            lib.attn("q4_0", "q4_0", q, kc, kc.clone(), table, dev(np.array(start, np.int64).astype(np.int32)),
                     dev(np.array([cells, -7, big, cells, -big, 5], np.int32)), 2, 16, max_q=max_q, max_kv=cells,
                     out=whole[20:20 + n])
            torch.cuda.synchronize()
            assert torch.all(whole[:20] == 7.0).item() and torch.all(whole[20 + n:] == 7.0).item()
            assert torch.all((whole == 7.0) | (whole == 0.0)).item()  # scales of 0: every value is 0


def test_attn_max_q(lib):
    """A bound above the longest sequence changes nothing."""
    for seqs in ([(2, 300), (1, 40)], [(70, 80), (1, 40)]):
        for max_q in (None, 400, 100000):
            say(f"attn {seqs} max_q={max_q}")
            c = Case(seqs, 4, 2, 64, "q8_0", "q4_0", "bf16", pad=40, seed=61)
            c.check(c.run(lib, max_q=max_q))


def test_attn_splits(lib):
    """A sequence long enough to be split over workgroups, beside short and empty ones; max_kv too small, too large."""
    for dtype in DTYPES:
        c = Case([(1, 5000), (1, 3), (1, 0), (1, 1029)], 8, 2, 128, "q8_0", "q4_0", dtype, page=64, pad=2, seed=11)
        for max_kv in (None, 5000, 900, 0, 10 ** 6):
            say(f"attn splits {dtype} max_kv={max_kv}")
            c.check(c.run(lib, max_kv=max_kv))
        c = Case([(3, 2500), (2, 1), (3, 2)], 8, 2, 64, "q4_0", "q8_0", dtype, page=32, window=1500, seed=12)
        say(f"attn splits {dtype} window")
        c.check(c.run(lib))


def test_attn_bad_pages(lib):
    """Page numbers outside the cache: their cells count as not seen, for decode and for a prompt."""
    for seqs in ([(1, 100), (1, 33), (2, 16)], [(90, 100), (1, 33), (20, 20)], [(1, 2000)]):
        say(f"attn bad pages {seqs}")
        c = Case(seqs, 4, 2, 128, "q8_0", "q8_0", "f32", bad_pages=(0, 3), seed=5)
        c.check(c.run(lib))


@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", DTYPES)
def test_attn_unseen_cells_have_no_effect(lib, head_dim, dtype):
    """NaN and infinite scales in cells that some rows of a tile see and others do not must not reach the others."""
    say(f"attn unseen {head_dim} {dtype}")
    for n, cells in ((4, 60), (100, 130)):
        c = Case([(n, cells)], 4, 2, head_dim, "q8_0", "q4_0", dtype, hurt=[(0, cells - 2)], seed=9)
        out = c.run(lib)
        n = n - 2  # the last two tokens see the hurt cell
        c.start[-1], c.T = n, n
        c.want, c.bound = c.want[:n], c.bound[:n]
        c.check(out[:n])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 80])
def test_attn_ranges_of_values(lib, dtype, n):
    """Tiny and huge values, and peaked rows: V scales near fp16's ends, queries far from one."""
    for q_scale, v_scale in ((1.0, 1e-5), (1.0, 3e4), (30.0, 1.0), (1e-4, 1.0)):
        say(f"attn ranges {dtype} n={n} q {q_scale} v {v_scale}")
        if dtype == "f16" and v_scale > 1e4:
            v_scale = 1e4
        c = Case([(n, 150), (n, 90)], 4, 2, 64, "q8_0", "q8_0", dtype, q_scale=q_scale, v_scale=v_scale, seed=4)
        out = c.run(lib)
        if v_scale < 1e-4 and dtype == "f16":  # outputs among fp16's subnormals: no relative error to speak of
            got = out[:, :c.heads].double().cpu().numpy()
            assert np.all(np.abs(got - c.want) <= c.bound)
        else:
            c.check(out)


def test_attn_same_bits_again_and_in_graphs(lib):
    """The same call twice, and captured and replayed with changed inputs, gives the eager call's bits."""
    import torch
    for seqs, kw in (([(1, 900), (1, 40)], {}), ([(70, 300), (1, 5)], {}), ([(70, 1700)], {})):
        c = Case(seqs, 8, 2, 128, dtype="bf16", seed=21)
        q = c.qt.cuda()[:, 1:1 + c.heads].contiguous()
        kc, vc, table, start, kv_len = dev(c.k), dev(c.v), dev(c.table), dev(c.start), dev(c.kv_len)
        args = (c.k_fmt, c.v_fmt, q, kc, vc, table, start, kv_len, c.kv_heads, c.page)
        out = torch.zeros_like(q)
        call = lambda o: lib.attn(*args, max_q=max(n for n, _ in c.seqs), out=o)  # noqa: E731
        say(f"attn graph {seqs}")
        call(out)
        first = out.clone()
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call(out)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            call(out)
        for i in range(4):
            q.copy_(torch.randn_like(q)) if i else None
            if i == 2:
                kv_len -= 1  # lengths change between replays
            out.fill_(5.0)
            g.replay()
            torch.cuda.synchronize()
            eager = torch.zeros_like(q)
            call(eager)
            torch.cuda.synchronize()
            assert torch.equal(out, eager), f"replay {i}"
            if i == 0:
                assert torch.equal(out, first)


def test_store_attend_load_together(lib):
    """As a serving loop uses them: a prompt stored and attended to, then tokens one at a time, on a side stream."""
    import torch
    rng = np.random.default_rng(31)
    heads, kv_heads, D, page, dim = 8, 2, 64, 16, 128
    pages = 16
    stream = torch.cuda.Stream()
    bias = rng.standard_normal(dim).astype(np.float32)
    prompts = [37, 5]
    total = [45, 13]
    table = rng.permutation(pages)[:2 * 4].reshape(2, 4).astype(np.int32)
    k_all = [rng.standard_normal((t, dim)).astype(np.float32) + bias for t in total]
    v_all = [rng.standard_normal((t, dim)).astype(np.float32) for t in total]
    q_all = [rng.standard_normal((t, heads, D)).astype(np.float32) for t in total]
    # what the cells hold in 64 bits: keys centred (scores move alike: no output changes)
    kd = [oracle.dequant("q8_0", oracle.quantize("q8_0", k - bias), len(k), dim) for k in k_all]
    vd = [oracle.dequant("q4_0", oracle.quantize("q4_0", v), len(v), dim) for v in v_all]
    slot = lambda b, j: int(table[b, j // page]) * page + j % page  # noqa: E731
    with torch.cuda.stream(stream):
        kc = torch.full((pages * page, oracle.row_bytes("q8_0", dim)), 0xFF, dtype=torch.uint8, device="cuda")
        vc = torch.full((pages * page, oracle.row_bytes("q4_0", dim)), 0xFF, dtype=torch.uint8, device="cuda")
        tb, bt = dev(table), dev(bias)
        steps = [[(b, 0, prompts[b]) for b in (0, 1)]]
        steps += [[(b, prompts[b] + i, prompts[b] + i + 1) for b in (0, 1)] for i in range(8)]
        for step in steps:
            say(f"step {step}")
            k, v, q = (np.concatenate([x[b][lo:hi] for b, lo, hi in step]) for x in (k_all, v_all, q_all))
            slots = np.array([slot(b, j) for b, lo, hi in step for j in range(lo, hi)], np.int32)
            lib.kv_store("q8_0", "q4_0", dev(k), dev(v), dev(slots), kc, vc, k_bias=bt)
            start = np.cumsum([0] + [hi - lo for _, lo, hi in step]).astype(np.int32)
            out = lib.attn("q8_0", "q4_0", dev(q), kc, vc, tb, dev(start),
                           dev(np.array([hi for _, _, hi in step], np.int32)), kv_heads, page)
            for x, (b, lo, hi) in enumerate(step):
                want, _ = ref.attention(q_all[b][lo:hi].astype(np.float64), kd[b], vd[b], np.arange(hi), kv_heads, hi - lo,
                                        hi, D ** -0.5, True, 0)
                got = out[start[x]:start[x + 1]].double().cpu().numpy()
                assert np.linalg.norm(got - want) <= ref.l2_bound("f32") * np.linalg.norm(want)
        for b in (0, 1):
            slots = dev(np.array([slot(b, j) for j in range(total[b])], np.int32))
            k, v = lib.kv_load("q8_0", "q4_0", kc, vc, slots, dim, k_bias=bt)
            assert np.array_equal(k.cpu().numpy(), kd[b].astype(np.float32) + bias)
            assert np.array_equal(v.cpu().numpy(), vd[b].astype(np.float32))


def test_cells_past_32_bit_offsets(lib):
    """A cache of more than 4 GiB: its last cells are stored, attended to and loaded."""
    import torch
    dim, heads, kv_heads, D, page = 4096, 32, 32, 128, 64
    rb = oracle.row_bytes("q8_0", dim)
    cells = (2 ** 32 // rb // page + 40) * page
    say(f"cache of {cells * rb / 2 ** 30:.2f} GiB")
    kc = torch.zeros((cells, rb), dtype=torch.uint8, device="cuda")
    vc = torch.zeros((cells, rb), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    n = 100
    k, v = (rng.standard_normal((n, dim)).astype(np.float32) for _ in range(2))
    last = cells // page - 1
    table = np.array([[last, last - 1]], np.int32)
    slots = np.array([table[0, j // page] * page + j % page for j in range(n)], np.int32)
    lib.kv_store("q8_0", "q8_0", dev(k), dev(v), dev(slots), kc, vc)
    k2, v2 = lib.kv_load("q8_0", "q8_0", kc, vc, dev(slots), dim)
    kd, vd = (oracle.dequant("q8_0", oracle.quantize("q8_0", x), n, dim) for x in (k, v))
    assert np.array_equal(k2.cpu().numpy(), kd.astype(np.float32))
    assert np.array_equal(v2.cpu().numpy(), vd.astype(np.float32))
    small = (table[0][:, None] * 4 + np.arange(4)).reshape(1, 8).astype(np.int32)  # the same cells in pages of 16
    for tokens, size in ((1, page), (1, 16), (40, page), (70, page), (70, 16)):
        say(f"attn {tokens} tokens, pages of {size}")
        q = rng.standard_normal((tokens, heads, D)).astype(np.float32)
        out = lib.attn("q8_0", "q8_0", dev(q), kc, vc, dev(table if size == page else small),
                       dev(np.array([0, tokens], np.int32)), dev(np.array([n], np.int32)), kv_heads, size)
        want, _ = ref.attention(q.astype(np.float64), kd, vd, np.arange(n), kv_heads, tokens, n, D ** -0.5, True, 0)
        got = out.double().cpu().numpy()
        assert np.linalg.norm(got - want) <= ref.l2_bound("f32") * np.linalg.norm(want)
