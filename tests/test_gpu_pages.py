"""The pages' operators against their definition, one row after another on the host: whole numbers,
which have to be equal."""
import random

import pytest
import torch

import verify_spec_greedy_gb300 as lib
from pages_reference import Pages

pytestmark = pytest.mark.gpu
I32 = torch.int32


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Device:
    """The same description on the GPU."""

    def __init__(self, m):
        self.m = m
        self.table, self.held, self.refs = dev(m.table), dev(m.held), dev(m.refs)
        self.copies = torch.full((len(m.held), 2), 77, dtype=I32, device="cuda")
        self.moves = torch.full((m.N // 2, 2), 77, dtype=I32, device="cuda")
        self.n_moves = torch.full((1,), 77, dtype=I32, device="cuda")
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def same(self):
        assert self.table.tolist() == self.m.table
        assert self.held.tolist() == self.m.held
        assert self.refs.tolist() == self.m.refs

    def resize(self, keep, lens, copy=True):
        copies, short, bad = self.m.resize(keep, lens, copy)
        self.status.zero_()
        lib.mtp_pages_resize(dev(keep), dev(lens), self.table, self.held, self.refs, self.m.P,
                             self.copies if copy else None, status=self.status)
        self.same()
        if copy:
            assert self.copies.tolist() == [list(c) for c in copies]
        assert int(self.status) == lib.STATUS_NO_PAGES * short | lib.STATUS_BAD_PARAM * bad
        return copies

    def fork(self, src, dst):
        bad = self.m.fork(src, dst)
        self.status.zero_()
        lib.mtp_pages_fork(dev(src), dev(dst), self.table, self.held, self.refs, status=self.status)
        self.same()
        assert int(self.status) == lib.STATUS_BAD_PARAM * bad

    def compact(self):
        pairs = self.m.compact()
        self.status.zero_()
        lib.mtp_pages_compact(self.table, self.held, self.refs, self.moves, self.n_moves,
                              status=self.status)
        self.same()
        assert int(self.n_moves) == len(pairs) and int(self.status) == 0
        assert self.moves.tolist() == [list(p) for p in pairs] + [[-1, -1]] * (self.m.N // 2 - len(pairs))
        return pairs


@pytest.mark.parametrize("B,wide,N,P,seed", [(1, 4, 1, 8, 0), (3, 6, 20, 16, 1), (17, 9, 100, 8, 2),
                                             (64, 12, 700, 32, 3), (300, 5, 1100, 16, 4),
                                             (1500, 4, 9000, 64, 5), (40, 30, 20000, 1, 6)])
def test_rounds_of_everything(B, wide, N, P, seed):
    """Many rounds: drafts are cut and grow, rows branch and end, the cache is moved together;
    there are not always enough pages."""
    r = random.Random(seed)
    d = Device(Pages(B, wide, N, P))
    for i in range(12):
        m = d.m
        keep = [r.randint(0, h * P) if h else 0 for h in m.held]
        keep = [k - k % P if r.random() < 0.2 else -1 if r.random() < 0.1 else k for k in keep]
        fair = max(1, N * P // B)
        lens = [min(wide * P, max(k, 0) + r.randint(0, r.choice([1, P, fair]))) for k in keep]
        d.resize(keep, lens)
        assert m.agrees()
        if B > 1:
            rows = r.sample(range(B), r.randint(0, min(B, 60)))
            cut = r.randint(0, max(0, len(rows) - 1))
            src = [r.choice(rows[:cut + 1]) for _ in rows[cut + 1:]]
            if src:
                d.fork(src, rows[cut + 1:])
                assert m.agrees()
        if i % 4 == 3:
            d.compact()
            assert m.agrees()


def test_branches_get_last_pages_of_their_own():
    m = Pages(6, 5, 30, 16)
    m.take(0, 3)
    m.take(1, 2)
    d = Device(m)
    d.fork([0, 0, 1], [2, 3, 4])
    assert m.refs[:5] == [3, 3, 3, 2, 2]
    # rows 0, 2, 3 write into page 2: the lowest stays; rows 1 and 4 are full at 32: none leaves
    copies = d.resize([40, 32, 40, 40, 32, 0], [44, 40, 50, 40, 33, 0])
    assert copies[0] == (-1, -1) and copies[2][0] == copies[3][0] == 2
    # a row that holds a page whole keeps writers from staying
    m = Pages(3, 5, 30, 16)
    m.take(0, 2)
    d = Device(m)
    d.fork([0, 0], [1, 2])
    copies = d.resize([20, 32, 20], [20, 40, 20])
    assert copies[0] == (1, 2) and copies[2][0] == 1


def test_without_copies_shared_pages_stay():
    m = Pages(2, 4, 10, 8)
    m.take(0, 2)
    d = Device(m)
    d.fork([0], [1])
    d.resize([12, 12], [20, 20], copy=False)
    assert m.table[0][:2] == m.table[1][:2]


def test_too_few_pages():
    m = Pages(4, 8, 10, 8)
    m.take(0, 2)
    d = Device(m)
    d.fork([0], [2])
    # row 0 stays on page 1, row 1 takes five, row 2 would leave page 1 and take three: eight are
    # there and five gone, so it and all after it get none, though row 3 needs but one
    d.resize([12, 0, 12, 0], [12, 40, 40, 8])
    assert m.held == [2, 5, 2, 0] and m.refs[1] == 2
    d.resize([12, 0, 12, 0], [12, 0, 16, 8])
    assert m.held == [2, 0, 2, 1]


def test_lengths_that_do_not_fit_leave_a_row_as_it_is():
    m = Pages(6, 3, 20, 8)
    for b in range(6):
        m.take(b, 2)
    d = Device(m)
    d.resize([17, 5, 4, -1, -7, 16], [20, 4, 25, 100, 3, 24])
    assert m.held == [2, 2, 2, 2, 2, 3]


def test_pairs_that_are_passed_over():
    m = Pages(6, 3, 20, 8)
    for b in range(4):
        m.take(b, 1 + b % 3)
    for src, dst in (([0, 1], [4, 4]), ([0, 4], [4, 5]), ([0], [0]), ([6, -1, 0, 0], [1, 2, 6, -2]),
                     ([3, 0, 1], [5, 5, 5])):
        d = Device(m)
        d.fork(src, dst)
        assert m.agrees()


def test_a_full_and_an_empty_cache_stay():
    m = Pages(2, 8, 9, 8)
    assert Device(m).compact() == []
    m.take(0, 8)
    m.take(1, 1)
    assert Device(m).compact() == []
    one = Pages(1, 1, 1, 8)
    assert Device(one).compact() == []
    one.take(0, 1)
    assert Device(one).compact() == []


def test_a_long_row_and_many_pages():
    m = Pages(2, 30000, 70000, 16)
    m.take(1, 5)
    d = Device(m)
    d.resize([0, 70], [30000 * 16, 16 * 16])
    d.fork([0], [1])
    d.resize([0, 29000 * 16 + 3], [0, 29010 * 16])
    d.compact()
    assert m.agrees()


@pytest.mark.parametrize("shape,dtype,pitch", [((40, 16, 2, 64), torch.bfloat16, 0), ((40, 8, 1, 8), torch.float16, 0),
                                               ((40, 64, 8, 128), torch.bfloat16, 64), ((40, 5, 4), torch.float32, 12)])
def test_copies(shape, dtype, pitch):
    g = torch.Generator(device="cuda").manual_seed(1)
    caches = []
    for _ in range(3):
        whole = torch.randn(shape[0], *shape[1:-1], shape[-1], generator=g, device="cuda").to(dtype)
        if pitch:  # pages further apart than they are long
            n = whole[0].numel()
            wide = torch.zeros(shape[0], n + pitch, dtype=dtype, device="cuda")
            wide[:, :n] = whole.reshape(shape[0], n)
            whole = wide[:, :n].unflatten(1, shape[1:])
        caches.append(whole)
    pairs = [(3, 9), (-1, -1), (4, 0), (4, 39), (-1, 5), (8, -2), (10, 11)]
    for n in (None, 0, 3, 7, 100, -5):
        before = [c.clone() for c in caches]
        status = torch.zeros(1, dtype=I32, device="cuda")
        lib.mtp_pages_copy(caches, dev(pairs), n_pairs=None if n is None else dev([n]), status=status)
        for c, old in zip(caches, before):
            for a, b in pairs[:7 if n is None else max(0, min(n, 7))]:
                if a >= 0 and b >= 0:
                    old[b] = old[a]
            assert torch.equal(c, old)
        assert int(status) == 0
    status = torch.zeros(1, dtype=I32, device="cuda")
    before = caches[0].clone()
    lib.mtp_pages_copy(caches[:1], dev([(40, 1), (2, 2 ** 30), (5, 6)]), status=status)
    before[6] = before[5]
    assert torch.equal(caches[0], before) and int(status) == lib.STATUS_BAD_PARAM


def test_a_graph_of_a_round():
    """Resize and copy captured once, replayed with other lengths."""
    m = Pages(4, 6, 40, 8)
    m.take(0, 3)
    m.fork([0, 0], [1, 2])
    d = Device(m)
    keep, lens = dev([20, 20, 20, 0]), dev([24, 24, 24, 0])
    g = torch.cuda.CUDAGraph()
    cache = torch.randn(40, 8, 2, 16, device="cuda").to(torch.bfloat16)
    want = cache.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lib.mtp_pages_resize(keep, lens, d.table, d.held, d.refs, 8, d.copies)
        lib.mtp_pages_copy([cache], d.copies)
    for k, n in (([20, 20, 20, 0], [24, 24, 24, 0]), ([22, 21, 17, 0], [30, 40, 17, 8]),
                 ([0, 40, 1, 3], [1, 48, 9, 8])):
        keep.copy_(dev(k))
        lens.copy_(dev(n))
        g.replay()
        copies, short, bad = m.resize(k, n)
        assert not short and not bad
        for a, b in copies:
            if a >= 0:
                want[b] = want[a]
        d.same()
        assert torch.equal(cache, want)
