"""csa_page_plan when pages run out: steps one after another against a plain allocator, as requests that hold places
without a page roll back, end in any order, grow on and begin again.  The pool never gains, loses or doubles a page."""
import random

import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    csa.load()


class Plain:
    """The definition.  A place of the table without a page (-1) is not given back."""

    def __init__(self, batch, P, max_pages, n_pages, seed=0):
        self.P, self.max_pages, self.n_pages = P, max_pages, n_pages
        self.free = list(range(n_pages))
        random.Random(seed).shuffle(self.free)
        self.count = n_pages
        self.table = [[0] * max_pages for _ in range(batch)]
        self.len = [0] * batch

    def held(self, n):
        return min(-(-n // self.P), self.max_pages)

    def step(self, after, maps=()):
        before = self.len
        p0, p1 = [self.held(n) for n in before], [self.held(n) for n in after]
        batch = range(len(before))
        given = [self.table[b][j] for b in batch for j in range(p1[b], p0[b])]
        given = [pg for pg in given if 0 <= pg < self.n_pages]
        taken = [(b, j) for b in batch for j in range(p0[b], p1[b])]
        R, A = len(given), len(taken)
        for i, pg in enumerate(given):
            self.free[self.count + R - 1 - i] = pg
        got = min(A, self.count + R)
        for i, (b, j) in enumerate(taken):
            self.table[b][j] = self.free[self.count + R - 1 - i] if i < got else -1
        self.count += R - got
        self.len = list(after)
        want = sum(max(0, -(-n // self.P) - p) for n, p in zip(after, p0))
        out = []
        for m, cap, sf in maps:
            pe, start, slots, sfs = self.P // m, [0], [], []
            for b in batch:
                for r in range(before[b] // m, max(before[b] // m, after[b] // m)):
                    pg = self.table[b][r // pe] if r // pe < p1[b] else -1
                    slots.append(pg * pe + r % pe if pg >= 0 else -1)
                    pg = self.table[b][r // 128 * 128 // pe] if slots[-1] >= 0 else -1
                    sfs.append(pg * 128 + r % 128 if pg >= 0 else -1)
                start.append(len(slots))
            pad = [-1] * max(0, cap - len(slots))
            out.append((start, (slots + pad)[:cap], (sfs + pad)[:cap] if sf else None))
        return [got, R, want - got, 0], out

    def all_pages(self):
        """Every page that a request holds or the stack has."""
        return sorted([pg for b, n in enumerate(self.len) for pg in self.table[b][:self.held(n)] if pg >= 0] +
                      self.free[:self.count])


class Both:
    """The allocator and its image on the GPU, stepped together."""

    def __init__(self, batch, P, max_pages, n_pages, maps=(), seed=0, graph=False):
        self.plain = Plain(batch, P, max_pages, n_pages, seed)
        self.t = torch.tensor(self.plain.table, dtype=torch.int32, device=DEV).view(batch, max_pages)
        self.f = torch.tensor(self.plain.free, dtype=torch.int32, device=DEV)
        self.c = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
        self.lens = [torch.zeros(batch, dtype=torch.int64, device=DEV) for _ in range(2)]
        self.maps = maps
        self.sm = [csa.slot_map(m, batch, cap, scales=sf) for m, cap, sf in maps]
        self.info = torch.zeros(4, dtype=torch.int32, device=DEV)
        self.graph = None
        if graph:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._call()

    def _call(self):
        csa.page_plan(*self.lens, self.plain.P, self.t, self.f, self.c, maps=self.sm, info=self.info)

    def step(self, after):
        self.lens[0].copy_(torch.tensor(self.plain.len))
        self.lens[1].copy_(torch.tensor(after))
        self._call() if self.graph is None else self.graph.replay()
        info, maps = self.plain.step(after, self.maps)
        torch.cuda.synchronize()
        assert self.info.tolist() == info
        assert int(self.c) == self.plain.count
        n = self.plain.count
        assert self.f[:n].tolist() == self.plain.free[:n], "free pages"
        t = self.t.tolist()
        for b, ln in enumerate(self.plain.len):
            h = self.plain.held(ln)
            assert t[b][:h] == self.plain.table[b][:h], f"request {b}"
        for s, w, (m, _, sf) in zip(self.sm, maps, self.maps):
            got = (s.row_start.tolist(), s.slots.tolist(), s.sf_slots.tolist() if sf else None)
            assert got == w, f"slots, m = {m}"
        assert self.plain.all_pages() == list(range(self.plain.n_pages))
        csa.check_device_status()


def test_growing_short_then_shrinking_restores_the_stack():
    s = Both(3, 128, 9, 17, maps=[(4, 760, True), (128, 30, False)], seed=6)
    before = s.f.tolist()
    s.step([1000, 1000, 1000])
    assert s.plain.count == 0 and s.info.tolist()[2] == 7
    s.step([0, 0, 0])
    assert s.plain.count == 17 and s.f.tolist() == before
    s.step([1000, 1000, 0])
    assert s.info.tolist()[2] == 0


@pytest.mark.parametrize("order", [(2, 0, 1), (1, 2, 0), (2, 1, 0)])
def test_requests_end_in_any_order_after_a_shortage(order):
    s = Both(3, 128, 9, 17, maps=[(4, 760, True)], seed=7)
    s.step([1000, 1000, 1000])
    lens = [1000, 1000, 1000]
    for b in order:
        lens[b] = 0
        s.step(lens)
        grown = [n + 200 if n else 0 for n in lens]  # the others go on
        s.step(grown)
        s.step(lens)
    s.step([1100, 1000, 0])
    assert s.info.tolist()[2] == 0


def test_growth_inside_a_page_that_could_not_be_had():
    """Its rows have no slot, and that is no report of a bad page."""
    s = Both(2, 128, 9, 5, maps=[(4, 64, True), (128, 4, True)], seed=8)
    s.step([600, 100])
    assert s.info.tolist()[:3] == [5, 0, 1]
    s.step([600, 120])
    assert s.sm[0].slots.tolist()[:5] == [-1] * 5
    s.step([0, 124])
    s.step([600, 140])


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("batch,P,max_pages,n_pages,seed", [(1, 128, 6, 2, 3), (7, 64, 9, 12, 2), (40, 128, 12, 70, 3),
                                                            (300, 128, 8, 400, 4), (1100, 3, 5, 900, 5)])
def test_walks_over_an_exhausted_pool(batch, P, max_pages, n_pages, seed, graph):
    rng = random.Random(seed)
    m = 4 if P % 4 == 0 else 3
    s = Both(batch, P, max_pages, n_pages, maps=[(m, max(8, batch * P // m), P == 128), (P, 2 * batch, False)], seed=seed,
             graph=graph)
    most, short = P * max_pages, 0
    for _ in range(12):
        after = [rng.choice([0, n, max(0, n - rng.randint(0, 2 * P)), min(most, n + rng.randint(0, P)),
                             rng.randint(0, most)]) for n in s.plain.len]
        s.step(after)
        short += s.info.tolist()[2]
    assert short > 0
    s.step([0] * batch)
    assert s.plain.count == n_pages


def test_many_pages_given_back_with_holes_between():
    """More pages than a CTA's list of tiles has groups of 32."""
    s = Both(4, 128, 40000, 70000, seed=9)
    s.step([40000 * 128, 0, 0, 128])
    s.step([40000 * 128, 40000 * 128, 3 * 128, 128])       # the second is 1,000 and the third 3 pages short
    s.step([40000 * 128, 40000 * 128, 3 * 128, 0])
    s.step([10 * 128 + 1, 40000 * 128, 3 * 128, 0])
    s.step([10 * 128 + 1, 7, 700 * 128, 5 * 128])
    s.step([0, 0, 0, 0])
    assert s.plain.count == 70000


def test_a_page_outside_the_pool_is_not_given_back():
    s = Both(2, 128, 6, 12, seed=10)
    s.step([500, 300])
    s.t[0, 1] = 77
    s.t[1, 2] = -5
    lens = [torch.tensor(v, dtype=torch.int64, device=DEV) for v in ([500, 300], [0, 0])]
    info = csa.page_plan(*lens, 128, s.t, s.f, s.c)
    torch.cuda.synchronize()
    with pytest.raises(csa.CsaError, match="INVALID_ARG"):
        csa.check_device_status()
    assert info.tolist() == [0, 5, 0, 0] and int(s.c) == 10
    lost = {s.plain.table[0][1], s.plain.table[1][2]}
    assert sorted(s.f[:10].tolist()) == sorted(set(range(12)) - lost)
