"""A step of many requests through half of a decoder layer, as a serving program
runs it: pages and slots, embedding rows, norm into Q8_0, the fused projection
with the requests' adapters, rotary positions with normed heads, keys and
values into the cache, attention, and the output projection with its adapters
and the next norm.

Every stage is held to its own definition, computed in 64 bits from what the
stage before it gave: bytes and whole numbers exactly, the products to the stated
2e-3 of qmat_gemm (relative L2), adapters, positions and attention to the bounds
derived in their own tests."""
import numpy as np
import pytest

import kv_reference as ref
import oracle
import test_gpu_pages as pages
import test_gpu_rope as rope

pytestmark = pytest.mark.gpu

VOCAB, HIDDEN, HEADS, KV_HEADS, D, PAGE, WIDE, RANK = 300, 256, 4, 2, 64, 16, 8, 16
QKV = (HEADS + 2 * KV_HEADS) * D


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_qmat_amd as qmat
    qmat.library_path()
    return qmat


class Layer:
    def __init__(self, lib, seqs, free):
        import torch
        r = np.random.default_rng(3)
        g = torch.Generator().manual_seed(4)
        self.lib, self.seqs = lib, seqs
        draw = lambda *shape: (r.standard_normal(shape) / np.sqrt(shape[-1])).astype(np.float32)  # noqa: E731
        self.host = {"embed": oracle.quantize("q6_k", draw(VOCAB, HIDDEN)), "qkv": oracle.quantize("q4_k", draw(QKV, HIDDEN)),
                     "out": oracle.quantize("q4_0", draw(HIDDEN, HEADS * D))}
        self.dev = {k: torch.from_numpy(v).cuda() for k, v in self.host.items()}
        adapters = 3
        self.lora = {k: ((torch.randn(adapters, RANK, i, generator=g) / i ** 0.5).half(), (torch.randn(adapters, o, RANK, generator=g) / 4).half())
                     for k, i, o in (("qkv", HIDDEN, QKV), ("out", HEADS * D, HIDDEN))}
        self.lora_dev = {k: (a.cuda(), b.cuda()) for k, (a, b) in self.lora.items()}
        self.scale = torch.tensor([0.5, 1.0, 0.25])
        self.scale_dev = self.scale.cuda()
        self.adapter = [i % 4 - 1 for i in range(seqs)]
        self.adapter_dev = pages.ints(self.adapter)
        self.norms = [(1 + 0.2 * torch.randn(n, generator=g)).cuda() for n in (HIDDEN, D, D, HIDDEN)]
        self.freq, self.axis = lib.rope_freq(D), lib.rope_axis([16, 8, 8])
        self.pool = pages.Pool(seqs, free, PAGE, WIDE, free)
        self.state = self.pool.tensors()
        self.caches = [torch.zeros((free * PAGE, oracle.row_bytes(f, KV_HEADS * D)), dtype=torch.uint8, device="cuda") for f in ("q8_0", "q4_0")]

    def step(self, add, keep, ids, max_tokens, max_q):
        """One step with the library's calls alone; every stage's result."""
        import torch
        q = self.lib
        s = {}
        s["pages"] = q.page_step(add=add, page_size=PAGE, max_tokens=max_tokens, keep=keep, **self.state)
        q_start, slots, positions = s["pages"][:3]
        s["x"] = q.embed("q6_k", self.dev["embed"], HIDDEN, ids)
        _, s["xq"], _ = q.rms_norm(s["x"], self.norms[0], want="q8")
        s["qkv0"] = q.gemm("q4_k", self.dev["qkv"], s["xq"], QKV, HIDDEN, max_tokens)
        a, b = self.lora_dev["qkv"]
        s["qkv"] = q.lora(s["xq"], a, b, self.adapter_dev, q_start, torch.zeros_like(s["qkv0"]), base=s["qkv0"], scale=self.scale_dev, max_q=max_q)
        heads = s["qkv"].view(max_tokens, HEADS + 2 * KV_HEADS, D)
        s["pos"] = torch.stack((positions, positions // 4, positions % 4)).contiguous()
        s["q"], s["k"] = q.rope(heads[:, :HEADS], heads[:, HEADS:HEADS + KV_HEADS], s["pos"], self.freq, axis=self.axis, q_norm=self.norms[1],
                                k_norm=self.norms[2])
        q.kv_store("q8_0", "q4_0", s["k"], heads[:, HEADS + KV_HEADS:], slots, *self.caches)
        s["o"] = q.attn("q8_0", "q4_0", s["q"], *self.caches, self.state["page_table"], q_start, self.state["kv_len"], KV_HEADS, PAGE, max_q=max_q)
        s["oq"] = q.quantize("q8_0", s["o"].flatten(1))
        s["y0"] = q.gemm("q4_0", self.dev["out"], s["oq"], HIDDEN, HEADS * D, max_tokens)
        a, b = self.lora_dev["out"]
        s["y"] = q.lora(s["oq"], a, b, self.adapter_dev, q_start, s["y0"].clone(), scale=self.scale_dev, max_q=max_q)
        _, s["next"], s["h"] = q.rms_norm(s["y"], self.norms[3], residual=s["x"], want="q8")
        return s

    def check(self, s, add, keep, ids, max_tokens):
        import torch
        host = lambda t: t.double().cpu().numpy()  # noqa: E731
        want = self.pool.step(add, keep, max_tokens)
        pages.compare(s["pages"], want, self.state, self.pool)
        start, slots = want[0], np.array(want[1])
        n = start[-1]
        table = oracle.dequant("q6_k", self.host["embed"], VOCAB, HIDDEN).reshape(VOCAB, HIDDEN)
        there = (ids >= 0) & (ids < VOCAB)
        assert np.array_equal(host(s["x"]), np.where(there[:, None], table[np.where(there, ids, 0)], 0.0))

        def normed(h, w):
            return (h / np.sqrt((h ** 2).mean(1, keepdims=True) + 1e-6) * host(w)).astype(np.float32)
        assert np.array_equal(s["xq"].cpu().numpy(), oracle.quantize("q8_0", normed(host(s["x"]), self.norms[0])))

        def product(name, fmt, xq, y0, y):
            a, b = (host(t) for t in self.lora[name])
            out, inn = b.shape[1], a.shape[2]
            x = oracle.dequant("q8_0", xq.cpu().numpy(), max_tokens, inn).reshape(max_tokens, inn)
            w = oracle.dequant(fmt, self.host[name], out, inn).reshape(out, inn)
            assert np.linalg.norm(host(y0) - x @ w.T) <= 2e-3 * np.linalg.norm(x @ w.T)
            whole, bound = host(y0), np.zeros((max_tokens, out))
            for i, ad in enumerate(self.adapter):
                t = slice(start[i], start[i + 1])
                if ad >= 0:
                    c = float(self.scale[ad])
                    whole[t] += c * (x[t] @ a[ad].T) @ b[ad].T
                    bound[t] = c * ((np.abs(x[t]) @ np.abs(a[ad]).T) @ np.abs(b[ad]).T) * (2.0 ** -18 + (inn / 32 + RANK + 16) * 2.0 ** -24)
            assert np.all(np.abs(host(y) - whole) <= bound + 2.0 ** -24 * np.abs(whole))
        product("qkv", "q4_k", s["xq"], s["qkv0"], s["qkv"])
        heads = host(s["qkv"]).reshape(max_tokens, HEADS + 2 * KV_HEADS, D)
        axis = self.axis.cpu().numpy()
        for name, lo, hi, w in (("q", 0, HEADS, self.norms[1]), ("k", HEADS, HEADS + KV_HEADS, self.norms[2])):
            v, bound = rope.formula(heads[:, lo:hi], s["pos"].cpu().numpy(), self.freq.cpu().numpy(), axis, False, host(w), 1e-6, "f32")
            assert np.all(np.abs(host(s[name]) - v) <= bound)
        live = slots >= 0
        rows = (s["k"].flatten(1).cpu().numpy(), s["qkv"][:, (HEADS + KV_HEADS) * D:].cpu().numpy())
        for cache, fmt, row in zip(self.caches, ("q8_0", "q4_0"), rows):
            assert np.array_equal(cache.cpu().numpy()[slots[live]], oracle.quantize(fmt, np.ascontiguousarray(row[live])))
        cells = self.caches[0].shape[0]
        k, v = (oracle.dequant(f, c.cpu().numpy(), cells, KV_HEADS * D).reshape(cells, -1) for c, f in zip(self.caches, ("q8_0", "q4_0")))
        got, whole = host(s["o"]), np.zeros((max_tokens, HEADS, D))
        for i in range(self.seqs):
            t, kv = slice(start[i], start[i + 1]), self.pool.kv[i]
            cell_of = [self.pool.table[i][j // PAGE] * PAGE + j % PAGE for j in range(kv)]
            whole[t], _ = ref.attention(host(s["q"])[t], k, v, cell_of, KV_HEADS, start[i + 1] - start[i], kv, D ** -0.5, True, 0)
        assert np.linalg.norm(got - whole) <= ref.l2_bound("f32") * max(np.linalg.norm(whole), 1e-30)
        assert not got[n:].any()
        assert np.array_equal(s["oq"].cpu().numpy(), oracle.quantize("q8_0", s["o"].flatten(1).cpu().numpy()))
        product("out", "q4_0", s["oq"], s["y0"], s["y"])
        h = s["y"].cpu() + s["x"].cpu()
        assert torch.equal(s["h"].cpu(), h)
        assert np.array_equal(s["next"].cpu().numpy(), oracle.quantize("q8_0", normed(h.double().numpy(), self.norms[3])))


def plan(seqs, kinds):
    """(add, keep, most tokens of a sequence) of each step; keep takes the lengths before it."""
    r = np.random.default_rng(seqs)
    for kind in kinds:
        if kind == "prompt":
            yield r.integers(0, 40, seqs).tolist(), None
        elif kind == "decode":
            yield [1] * seqs, None
        elif kind == "draft":  # up to three of the last cells turned down, four new ones
            yield [4] * seqs, lambda kv: [max(0, v - int(r.integers(0, 4))) for v in kv]
        else:  # some end, others begin
            yield r.integers(0, 20, seqs).tolist(), lambda kv: [v if r.random() < 0.6 else 0 for v in kv]


def test_steps(lib):
    import torch
    seqs = 5
    layer = Layer(lib, seqs, 26)
    r = np.random.default_rng(9)
    for add, cut in plan(seqs, ("prompt", "decode", "draft", "decode", "mixed", "draft", "prompt")):
        keep = None if cut is None else cut(layer.pool.kv)
        max_tokens = sum(add) + 3
        ids = r.integers(0, VOCAB, max_tokens).astype(np.int32)
        ids[-2:] = -1
        s = layer.step(pages.ints(add), pages.ints(keep), torch.from_numpy(ids).cuda(), max_tokens, max(add))
        layer.check(s, add, keep, ids, max_tokens)


def test_captured_step(lib):
    """One captured decode step replayed over growing lengths, beside eager work; the last pages run out on the way."""
    import torch
    seqs, max_tokens = 5, 8
    layer = Layer(lib, seqs, 8)
    r = np.random.default_rng(2)
    add, ids = pages.ints([0] * seqs), torch.zeros(max_tokens, dtype=torch.int32, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(add, None, ids, max_tokens, 1)
    side.synchronize()
    with torch.cuda.graph(graph):
        s = layer.step(add, None, ids, max_tokens, 1)
    for i in range(40):
        n = [1] * seqs if i % 3 else [1, 0, 1, 1, 0]
        now = r.integers(0, VOCAB, max_tokens).astype(np.int32)
        add.copy_(pages.ints(n))
        ids.copy_(torch.from_numpy(now).cuda())
        graph.replay()
        torch.cuda.synchronize()
        layer.check(s, n, None, now, max_tokens)
    assert 2 in s["pages"][4].tolist()
