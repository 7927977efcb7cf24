"""Operations on the pages of a cache on the GPU against the oracle, integer by integer and byte by byte."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_47_b200 import build
    build.build()
    import exact_tiled_attention_47_b200 as fa
    fa.fa_device_status(clear=True)
    yield
    assert fa.fa_device_status(clear=True) == 0


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


class Both:
    """The state on the device and in numpy, and pools of unlike page sizes (one of 4 bytes, one above a piece)."""

    def __init__(self, seed, S, pps, P, page, sizes=(4, 20, 64, 2048, 40000)):
        rng = np.random.default_rng(seed)
        self.page = page
        self.table, self.lens, self.refs = np.full((S, pps), -1, np.int32), np.zeros(S, np.int32), np.zeros(P, np.int32)
        self.pools = [rng.integers(0, 256, (P, n), dtype=np.uint8) for n in sizes]
        self.dev()

    def dev(self):
        self.gt, self.gl, self.gr = (torch.from_numpy(x.copy()).cuda() for x in (self.table, self.lens, self.refs))
        self.gp = [torch.from_numpy(x.copy()).cuda() for x in self.pools]

    def same(self):
        torch.cuda.synchronize()
        for s in range(len(self.lens)):  # entries in use (the others mean nothing)
            n = -(-int(self.lens[s]) // self.page)
            assert np.array_equal(self.gt[s, :n].cpu().numpy(), self.table[s, :n]), s
        assert np.array_equal(self.gl.cpu().numpy(), self.lens)
        assert np.array_equal(self.gr.cpu().numpy(), self.refs)
        for g, x in zip(self.gp, self.pools):
            assert np.array_equal(g.cpu().numpy(), x)

    def extend(self, slots, add):
        import exact_tiled_attention_47_b200 as fa
        fa.extend_pages(self.gt, self.gl, self.gr, self.page, i32(add), None if slots is None else i32(slots))
        ok = oracle.pages.extend(self.table, self.lens, self.refs, self.page, range(len(add)) if slots is None else slots, add)
        self.same()
        return ok

    def fork(self, src, dst):
        import exact_tiled_attention_47_b200 as fa
        fa.fork_pages(self.gt, self.gl, self.gr, self.page, i32(src), i32(dst), self.gp)
        ok = oracle.pages.fork(self.table, self.lens, self.refs, self.page, src, dst, self.pools)
        self.same()
        return ok

    def free(self, slots):
        import exact_tiled_attention_47_b200 as fa
        fa.free_pages(self.gt, self.gl, self.gr, self.page, i32(slots))
        oracle.pages.free(self.table, self.lens, self.refs, self.page, slots)
        self.same()

    def compact(self, in_place):
        import exact_tiled_attention_47_b200 as fa
        old = self.gt.clone(), self.gr.clone()
        table, refs, remap, n_live = fa.compact_pages(self.gt, self.gl, self.gr, self.page, self.gp, in_place=in_place)
        if in_place:
            assert table is self.gt and refs is self.gr
        else:
            assert torch.equal(self.gt, old[0]) and torch.equal(self.gr, old[1])
        self.table, self.refs, want, n = oracle.pages.compact(self.table, self.lens, self.refs, self.page, self.pools)
        self.gt, self.gr = table, refs
        assert int(n_live) == n and np.array_equal(remap.cpu().numpy(), want)
        self.same()


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("P,page", [(40, 16), (700, 32), (40000, 16)])
def test_random_life(seed, P, page):
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(seed * 10 + P)
    S, pps = 24, 30
    sizes = (4, 20, 64, 2048, 40000) if P <= 700 else (4, 48)
    t = Both(seed, S, pps, P, page, sizes)
    if P == 40000:  # most pages in use from the start, holes among them: the scan passes several steps
        t.refs[rng.random(P) < 0.9] = 1
        t.dev()
    for step in range(14):
        kind = rng.choice(["extend", "extend", "fork", "free", "compact"])
        if kind == "extend":
            slots = rng.permutation(S)[: rng.integers(1, S)]
            ok = t.extend(slots, [int(min(rng.integers(0, 5 * page), pps * page - t.lens[s])) for s in slots])
            want = 0 if ok else fa.FA_ERR_NO_PAGES
        elif kind == "fork":
            empty, live = np.flatnonzero(t.lens == 0), np.flatnonzero(t.lens)
            if not len(empty) or not len(live):
                continue
            dst = rng.permutation(empty)[: rng.integers(1, len(empty) + 1)]
            ok = t.fork([int(s) for s in rng.choice(live, len(dst))], [int(d) for d in dst])
            want = 0 if ok else fa.FA_ERR_NO_PAGES
        elif kind == "free":
            slots = [int(s) for s in rng.integers(0, S, rng.integers(1, 6))]  # empty ones and the same twice among them
            t.free(slots)
            want = 0
        else:
            if P == 40000:
                t.refs[t.refs > 0] = np.where(np.isin(np.flatnonzero(t.refs > 0), t.table), t.refs[t.refs > 0], 1)
            t.compact(bool(rng.integers(2)))
            want = 0
        assert fa.fa_device_status(clear=True) == want, (step, kind)


def test_slots_from_the_first_on():
    t = Both(1, 5, 4, 30, 16)
    assert t.extend(None, [3, 0, 17])
    assert t.extend(None, [13, 16, 15, 1, 1])


def test_exactly_the_last_pages():
    import exact_tiled_attention_47_b200 as fa
    t = Both(2, 3, 8, 8, 16)
    assert t.extend([1], [5 * 16])
    assert not t.extend([0, 2], [16, 3 * 16])  # four pages, three are free: nothing changes
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_NO_PAGES
    assert t.extend([0, 2], [16, 2 * 16])
    assert not t.fork([1], [0]) and fa.fa_device_status(clear=True) == fa.FA_ERR_SLOTS  # not empty
    t.free([0])
    assert t.fork([1], [0])  # whole pages need no new one


def test_refused_requests_change_nothing():
    import exact_tiled_attention_47_b200 as fa
    t = Both(3, 6, 4, 16, 16)
    assert t.extend([0, 1], [20, 64])
    for slots, add, code in (([2, 2], [1, 1], fa.FA_ERR_SLOTS), ([6], [1], fa.FA_ERR_SLOTS), ([-1], [1], fa.FA_ERR_SLOTS),
                             ([2, 1], [1, 1], fa.FA_ERR_CU_SEQLENS), ([0], [-1], fa.FA_ERR_CU_SEQLENS), ([0], [2 ** 31 - 1], fa.FA_ERR_CU_SEQLENS)):
        assert not t.extend(slots, add)
        assert fa.fa_device_status(clear=True) == code, (slots, add)
    for src, dst, code in (([0, 0], [2, 2], fa.FA_ERR_SLOTS), ([0], [1], fa.FA_ERR_SLOTS), ([0, 2], [2, 3], fa.FA_ERR_SLOTS), ([0], [0], fa.FA_ERR_SLOTS),
                           ([6], [2], fa.FA_ERR_SLOTS), ([0], [-2], fa.FA_ERR_SLOTS)):
        assert not t.fork(src, dst)
        assert fa.fa_device_status(clear=True) == code, (src, dst)
    t.gt[0, 1] = 16  # the partial page's entry names no page
    fa.fork_pages(t.gt, t.gl, t.gr, 16, i32([0]), i32([2]), t.gp)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_PAGE_TABLE
    t.gt[0, 1] = int(t.table[0, 1])
    t.same()


def test_corrupt_tables_are_reported_and_touch_nothing_else():
    import exact_tiled_attention_47_b200 as fa
    t = Both(4, 4, 4, 16, 16)
    assert t.extend([0, 1], [40, 32])
    t.gt[0, 1], t.gt[1, 0] = -7, 99
    fa.free_pages(t.gt, t.gl, t.gr, 16, i32([0, 1, 9]))
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) in (fa.FA_ERR_PAGE_TABLE, fa.FA_ERR_SLOTS)
    # pages 0, 2 of slot 0 and the second of slot 1 are given back, the two lost ones stay counted
    assert t.gr.tolist() == [0, 1, 0, 1] + [0] * 12 and t.gl.tolist() == [0] * 4
    t = Both(5, 4, 4, 16, 16)
    assert t.extend([0], [32])
    t.gt[0, 1] = 7  # a free page
    table, refs, remap, n_live = fa.compact_pages(t.gt, t.gl, t.gr, 16, t.gp)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_PAGE_TABLE
    assert table[0, 0] == 0 and table[0, 1] == -1 and int(n_live) == 2


def test_many_pools():
    # more pools than one launch takes
    import exact_tiled_attention_47_b200 as fa
    t = Both(6, 4, 4, 24, 16, sizes=[64 + 4 * i for i in range(150)])
    assert t.extend([0, 1], [20, 50])
    assert t.fork([0, 1, 1], [3, 2, 0]) is False
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_SLOTS
    assert t.fork([0, 1], [3, 2])
    t.free([0])
    t.compact(False)
    t.compact(True)  # nothing left to move


def test_no_pools_and_empty_lists():
    import exact_tiled_attention_47_b200 as fa
    t = Both(7, 4, 4, 24, 16, sizes=[])
    assert t.extend([0], [17])
    assert t.fork([0], [1])
    t.free([0])
    t.compact(False)
    e = i32([])
    fa.extend_pages(t.gt, t.gl, t.gr, 16, e, e)
    fa.fork_pages(t.gt, t.gl, t.gr, 16, e, e, [])
    fa.free_pages(t.gt, t.gl, t.gr, 16, e)
    t.same()


@pytest.mark.parametrize("live", [0, 1, 8192, 20000, 20011])
def test_compact_large(live):
    rng = np.random.default_rng(live)
    P = 20011
    t = Both(8, 3, 4, P, 16, sizes=[16, 12])
    t.refs[rng.permutation(P)[:live]] = rng.integers(1, 5, live)
    own = np.flatnonzero(t.refs)[-6:]
    t.table[0, : len(own[:4])], t.lens[0] = own[:4], 16 * len(own[:4])
    t.dev()
    t.compact(False)
    t.compact(True)


def test_copy_pages():
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(9)
    a = [torch.randint(0, 256, (30, n), dtype=torch.uint8, device="cuda") for n in (4, 2048, 36000)]
    b = [torch.randint(0, 256, (50, n), dtype=torch.uint8, device="cuda") for n in (4, 2048, 36000)]
    src, dst = i32(rng.integers(0, 30, 20)), i32(rng.permutation(50)[:20])
    want = [y.clone() for y in b]
    for x, y in zip(a, want):
        y[dst.long()] = x[src.long()]
    fa.copy_pages(a, b, src, dst)
    assert all(torch.equal(x, y) for x, y in zip(b, want))
    # inside one pool: destinations that are no sources
    want = [x.clone() for x in a]
    for x in want:
        x[torch.tensor([20, 21, 29], device="cuda")] = x[torch.tensor([3, 3, 0], device="cuda")]
    fa.copy_pages(a, a, i32([3, 3, 0]), i32([20, 21, 29]))
    assert all(torch.equal(x, y) for x, y in zip(a, want)) and fa.fa_device_status(clear=True) == 0
    for s, d, code in (([0, 1], [5, 5], fa.FA_ERR_SLOTS), ([0, 5], [5, 6], fa.FA_ERR_SLOTS), ([30], [0], fa.FA_ERR_PAGE_TABLE),
                       ([0], [30], fa.FA_ERR_PAGE_TABLE), ([-1], [0], fa.FA_ERR_PAGE_TABLE)):
        fa.copy_pages(a, a, i32(s), i32(d))
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == code
        assert all(torch.equal(x, y) for x, y in zip(a, want))


def test_in_a_graph():
    # a beam step captured once and replayed on the state as it then is
    import exact_tiled_attention_47_b200 as fa
    t = Both(10, 6, 8, 64, 16)
    assert t.extend([0, 1], [37, 16])
    src, dst, add = i32([0, 1, 0]), i32([2, 3, 4]), i32([1, 20, 5])
    graph = torch.cuda.CUDAGraph()
    warm = Both(10, 6, 8, 64, 16)  # sets up what the first calls on a device set up
    warm.extend([0], [5])
    warm.fork([0], [1])
    with torch.cuda.graph(graph):
        fa.free_pages(t.gt, t.gl, t.gr, 16, dst)
        fa.fork_pages(t.gt, t.gl, t.gr, 16, src, dst, t.gp)
        fa.extend_pages(t.gt, t.gl, t.gr, 16, add, dst)
    for _ in range(3):
        graph.replay()
        oracle.pages.free(t.table, t.lens, t.refs, 16, [2, 3, 4])
        assert oracle.pages.fork(t.table, t.lens, t.refs, 16, [0, 1, 0], [2, 3, 4], t.pools)
        assert oracle.pages.extend(t.table, t.lens, t.refs, 16, [2, 3, 4], [1, 20, 5])
        t.same()
