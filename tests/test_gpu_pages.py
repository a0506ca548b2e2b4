"""Page tables, slots and positions from request lengths on the GPU, against a
plain sequential reading of the rules, number for number."""
import random

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_quantized_weight_qmat_amd as qmat
    qmat.library_path()
    return qmat


class Pool:
    """The state of a cache's pages, and one step of it in plain Python."""

    def __init__(self, seqs, pages, page, wide, free, table_seed=0):
        r = random.Random(table_seed)
        order = list(range(pages))
        r.shuffle(order)
        self.page, self.pages, self.wide = page, pages, wide
        self.kv = [0] * seqs
        self.table = [[-7] * wide for _ in range(seqs)]
        self.free = order[:free] + [-3] * (pages - free)
        self.count = free
        self.order = order[free:]

    def hold(self, b, cells):
        """Gives sequence b cells from the pages that are not on the stack."""
        need = -(-cells // self.page)
        for j in range(need):
            self.table[b][j] = self.order.pop()
        self.kv[b] = cells

    def release(self):
        """Puts the pages that nobody was given on the stack."""
        self.free[self.count:self.count + len(self.order)] = self.order
        self.count += len(self.order)

    def step(self, add, keep, max_tokens):
        ps = self.page
        cut = lambda v, hi: max(0, min(v, hi))  # noqa: E731
        seqs = len(self.kv)
        held = [cut(v, self.wide * ps) for v in self.kv]
        kept = [h if keep is None else cut(keep[b], h) for b, h in enumerate(held)]
        add = [max(0, v) for v in add]
        count = cut(self.count, self.pages)
        asked, fits = 0, []
        for b in range(seqs):
            asked += add[b]
            fits.append(kept[b] + add[b] <= self.wide * ps and (add[b] == 0 or asked <= max_tokens))
        pages = lambda cells: -(-cells // ps)  # noqa: E731
        back = [(b, j) for b in range(seqs) if fits[b] for j in range(pages(kept[b] + add[b]), pages(held[b]))]
        for r, (b, j) in enumerate(reversed(back)):
            if count + r < self.pages:
                self.free[count + r] = self.table[b][j]
        top = min(count + len(back), self.pages)
        status, start, slots, pos, seq, wanted, taken = [], [0], [], [], [], 0, 0
        for b in range(seqs):
            old, now = pages(held[b]), pages(kept[b] + add[b])
            need = max(0, now - old) if fits[b] else 0
            wanted += need
            status.append(1 if not fits[b] else 2 if need and wanted > top else 0)
            if status[b] == 0:
                for j in range(old, old + need):
                    self.table[b][j] = self.free[top - 1 - taken]
                    taken += 1
                for p in range(kept[b], kept[b] + add[b]):
                    page = self.table[b][p // ps]
                    slots.append(page * ps + p % ps if 0 <= page < self.pages else -1)
                    pos.append(p)
                    seq.append(b)
                self.kv[b] = kept[b] + add[b]
            start.append(len(slots))
        self.count = top - taken
        rest = max_tokens - len(slots)
        return start, slots + [-1] * rest, pos + [0] * rest, seq + [-1] * rest, status

    def tensors(self):
        import torch
        t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"kv_len": t(self.kv), "page_table": t(self.table).reshape(len(self.kv), self.wide), "free_pages": t(self.free),
                "free_count": t([self.count])}


def ints(v):
    import torch
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def compare(got, want, state, pool, sound=True):
    for name, g, w in zip(("q_start", "slots", "positions", "token_seq", "status"), got, want):
        assert np.array_equal(g.cpu().numpy(), np.array(w, dtype=np.int32)), name
    assert state["kv_len"].tolist() == pool.kv
    assert state["free_count"].tolist() == [pool.count]
    assert state["free_pages"].tolist() == pool.free
    assert np.array_equal(state["page_table"].cpu().numpy(), np.array(pool.table, dtype=np.int32).reshape(len(pool.kv), pool.wide))
    if sound:  # every page is on the stack or held, once
        held = [pool.table[b][j] for b in range(len(pool.kv)) for j in range(-(-pool.kv[b] // pool.page))]
        assert sorted(held + pool.free[:pool.count]) == list(range(pool.pages))


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("seqs", [1, 2, 63, 64, 65, 300])
def test_steps(lib, seqs, page):
    """Several steps of one pool: prompts, decode, drafted tokens taken back, ends, with few pages."""
    r = random.Random(seqs * page)
    pool = Pool(seqs, 40 + seqs * max(1, 90 // page), page, max(3, 200 // page), 40 + seqs * max(1, 90 // page), seqs)
    state = pool.tensors()
    for kind in ("prompt", "decode", "draft", "mixed", "decode", "end", "prompt", "mixed"):
        keep = None
        if kind == "prompt":
            add = [r.choice((0, 1, r.randrange(130))) for _ in range(seqs)]
        elif kind == "decode":
            add = [1] * seqs
        elif kind == "draft":
            add, keep = [r.randrange(6) for _ in range(seqs)], [max(0, v - r.randrange(4)) for v in pool.kv]
        elif kind == "end":
            add, keep = [0] * seqs, [v if r.random() < 0.5 else 0 for v in pool.kv]
        else:
            add, keep = [r.randrange(80) for _ in range(seqs)], [r.randrange(v + 1) if r.random() < 0.5 else v for v in pool.kv]
        max_tokens = max(1, int(sum(add) * r.choice((0.6, 1.0, 1.3))))
        got = lib.page_step(add=ints(add), page_size=page, max_tokens=max_tokens, keep=ints(keep), **state)
        compare(got, pool.step(add, keep, max_tokens), state, pool)


@pytest.mark.parametrize("seqs,most", [(1023, 4), (1024, 4), (1025, 4), (2500, 30), (3, 9000), (1024, 40)])
def test_large(lib, seqs, most):
    """More sequences than threads, more tokens than one workgroup writes."""
    r = random.Random(seqs)
    page, wide = 16, max(4, most // 8 + 40)
    pool = Pool(seqs, seqs * 6 + most, page, wide, seqs * 2 + most)
    for b in range(seqs):
        pool.hold(b, r.randrange(50))
    pool.release()
    state = pool.tensors()
    for _ in range(3):
        add = [r.randrange(most + 1) for _ in range(seqs)]
        keep = [v if r.random() < 0.7 else r.randrange(v + 1) for v in pool.kv]
        max_tokens = sum(add) + 5
        got = lib.page_step(add=ints(add), page_size=page, max_tokens=max_tokens, keep=ints(keep), **state)
        compare(got, pool.step(add, keep, max_tokens), state, pool)


@pytest.mark.parametrize("seqs,add", [(5, 40), (5, 2000), (1500, 3)])
def test_taken_back(lib, seqs, add):
    """A step whose tokens are taken back leaves the stack and the lengths as they were."""
    pool = Pool(seqs, seqs * (add // 8 + 4), 16, add // 16 + 4, seqs * (add // 8 + 1))
    for b in range(seqs):
        pool.hold(b, (7 * b) % 33)
    pool.release()
    state = pool.tensors()
    before = {k: v.clone() for k, v in state.items()}
    lib.page_step(add=ints([add] * seqs), page_size=16, max_tokens=add * seqs, **state)
    assert not bool((state["free_count"] == before["free_count"]).item())
    lib.page_step(add=ints([0] * seqs), page_size=16, max_tokens=0, keep=before["kv_len"], **state)
    for k in ("kv_len", "free_count", "free_pages"):
        assert bool((state[k] == before[k]).all().item()), k


def test_refusals_in_order(lib):
    """A sequence that waits for pages is not overtaken by one that needs some, but by one that needs none."""
    pool = Pool(6, 12, 4, 6, 5)
    for b, n in enumerate((4, 3, 2, 4, 8, 1)):
        pool.hold(b, n)
    state = pool.tensors()
    add = [4, 13, 2, 20, 1, 30]  # pages: 1, 3, none, 5 of the last one, 1, more than its row has
    got = lib.page_step(add=ints(add), page_size=4, max_tokens=100, **state)
    assert got[4].tolist() == [0, 0, 0, 2, 2, 1]
    compare(got, pool.step(add, None, 100), state, pool)
    pool = Pool(4, 9, 4, 6, 2)
    for b, n in enumerate((4, 3, 2, 4)):
        pool.hold(b, n)
    state = pool.tensors()
    add = [9, 4, 2, 4]  # three pages of two: waits; one: waits behind it; none: done; one: waits
    got = lib.page_step(add=ints(add), page_size=4, max_tokens=100, **state)
    assert got[4].tolist() == [2, 2, 0, 2] and got[0].tolist() == [0, 0, 0, 2, 2]
    compare(got, pool.step(add, None, 100), state, pool, sound=False)
    got = lib.page_step(add=ints([3, 1, 2, 0]), page_size=4, max_tokens=5, **state)  # tokens: 3, 4, 6 (too many), none
    assert got[4].tolist() == [0, 0, 1, 0]
    compare(got, pool.step([3, 1, 2, 0], None, 5), state, pool, sound=False)


def test_values_out_of_range(lib):
    """Lengths, counts and page numbers outside their range: nothing outside the arrays is touched."""
    import torch
    page, wide, pages = 4, 3, 10
    pool = Pool(5, pages, page, wide, 6)
    pool.kv = [2 ** 31 - 1, -5, 3, 12, 4]
    pool.table = [[1, 99, -2], [0, 0, 0], [2 ** 31 - 1, 3, 3], [4, 5, 6], [-2 ** 31, 1, 1]]
    pool.free = [7, 2 ** 30, -9, 8, 9, 100, 0, 0, 0, 0]
    pool.count = 25
    state = pool.tensors()
    guard = torch.full((64,), 5, dtype=torch.int32, device="cuda")
    outs = {"slots": guard[8:18], "status": guard[30:35]}
    for add, keep in (([0, 3, 2, -4, 2 ** 31 - 1], [2 ** 31 - 1, 1, -3, 5, 4]), ([1, 1, 1, 1, 1], [4, 0, 0, 0, -2 ** 31]),
                      ([2 ** 31 - 1] * 5, None)):
        got = lib.page_step(add=ints(add), page_size=page, max_tokens=10, keep=ints(keep), **outs, **state)
        compare(got, pool.step(add, keep, 10), state, pool, sound=False)
    g = guard.tolist()
    assert g[:8] == [5] * 8 and g[18:30] == [5] * 12 and g[35:] == [5] * 29


def test_nothing(lib):
    """No sequences, no rows, no pages, no table columns."""
    import torch
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    count = ints([2])
    got = lib.page_step(e, e, e.view(0, 4), ints([5, 3, 0]), count, 16, 3)
    assert [g.tolist() for g in got] == [[0], [-1] * 3, [0] * 3, [-1] * 3, []] and count.tolist() == [2]
    got = lib.page_step(ints([0, 0]), ints([1, 0]), e.view(2, 0), e, ints([0]), 16, 0)
    assert [g.tolist() for g in got] == [[0, 0, 0], [], [], [], [1, 0]]


def test_captured(lib):
    """A captured step follows the lengths that it finds at replay, beside eager work."""
    import torch
    pool = Pool(40, 200, 16, 8, 200)
    state = pool.tensors()
    add = ints([0] * 40)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.page_step(add=add, page_size=16, max_tokens=400, **state)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = lib.page_step(add=add, page_size=16, max_tokens=400, **state)
    r = random.Random(9)
    for _ in range(4):
        n = [r.randrange(12) for _ in range(40)]
        add.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        compare(got, pool.step(n, None, 400), state, pool)
        assert int(add.sum()) == sum(n)


@pytest.mark.parametrize("seqs,rows,each", [(7, 3000, 5), (256, 2000, 5), (256, 60000, 3), (257, 5000, 5), (1024, 5000, 5), (1024, 60000, 3),
                                            (1030, 2100, 5), (2100, 90000, 3)])
def test_refused_and_taken_back_in_large_steps(lib, seqs, rows, each):
    """Steps whose rows a second kernel writes: too long for a table row, for the tokens, for the pages; pages given back and taken again."""
    r = random.Random(seqs)
    page, wide = 8, 12
    pages = each * seqs
    pool = Pool(seqs, pages, page, wide, 0)
    for b in range(seqs):
        pool.hold(b, r.randrange(4 * page))
    pool.release()
    state = pool.tensors()
    seen = set()
    for _ in range(5):
        add = [r.choice((0, 1, 3, r.randrange(wide * page + 20))) if r.random() < (0.3 if each > 3 else 0.8) else r.randrange(2) for _ in range(seqs)]
        keep = None if r.random() < 0.3 else [max(0, n - r.randrange(20)) for n in pool.kv]
        want = pool.step(add, keep, rows)
        got = lib.page_step(add=ints(add), keep=ints(keep), page_size=page, max_tokens=rows, **state)
        compare(got, want, state, pool)
        seen |= set(want[4])
    assert 0 in seen and (seqs < 100 or 1 in seen) and (each > 3 or 2 in seen)  # a few sequences may all fit


def test_large_step_captured(lib):
    """Two kernels and their workspace in a graph, replayed beside eager steps of another pool."""
    import torch
    pool, other = Pool(300, 3000, 16, 32, 3000), Pool(300, 3000, 16, 32, 3000, table_seed=5)
    state, state2 = pool.tensors(), other.tensors()
    add = ints([0] * 300)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.page_step(add=add, page_size=16, max_tokens=6000, **state)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = lib.page_step(add=add, page_size=16, max_tokens=6000, **state)
    r = random.Random(3)
    for _ in range(4):
        n, m = [r.randrange(20) for _ in range(300)], [r.randrange(20) for _ in range(300)]
        add.copy_(ints(n))
        graph.replay()
        eager = lib.page_step(add=ints(m), page_size=16, max_tokens=6000, **state2)
        torch.cuda.synchronize()
        compare(got, pool.step(n, None, 6000), state, pool)
        compare(eager, other.step(m, None, 6000), state2, other)
