"""Page bookkeeping against a plain Python model: tables, counts, lengths and the
pages' bytes are equal after every call."""
import random

import pytest
import torch

from .gpu_util import lib
from .kv_ref import Pages

pytestmark = pytest.mark.gpu


class Both:
    """The library's state and the model's, side by side."""

    def __init__(self, n_seqs, width, n_pages, page=16, n_pools=3, words=(2, 8), seed=0):
        self.L = lib()
        g = torch.Generator().manual_seed(seed)
        pools = torch.randint(-2 ** 31, 2 ** 31 - 1, (n_pools, n_pages, *words), generator=g, dtype=torch.int32)
        table = torch.full((n_seqs, width), -1, dtype=torch.int32)
        kv_len, refs = torch.zeros(n_seqs, dtype=torch.int32), torch.zeros(n_pages, dtype=torch.int32)
        self.model = Pages(table, kv_len, refs, pools, page)
        self.pools, self.table, self.len, self.refs = pools.cuda(), table.cuda(), kv_len.cuda(), refs.cuda()
        self.pool = self.L.tq1_page_pool(self.pools, self.table, self.len, self.refs, page)
        self.ws = torch.full((self.L.tq1_pages_workspace_size(self.pool),), 0xFF, dtype=torch.uint8, device="cuda")

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def resize(self, seqs, lens):
        self.L.tq1_pages_resize(self.pool, self.ints(seqs), self.ints(lens), self.ws)
        self.model.resize(seqs, lens)

    def fork(self, parents, children):
        self.L.tq1_pages_fork(self.pool, self.ints(parents), self.ints(children), self.ws)
        self.model.fork(parents, children)

    def compact(self):
        self.L.tq1_pages_compact(self.pool, self.ws)
        self.model.compact()

    def check(self):
        assert self.L.tq1_sync_status() == (-9 if self.model.lacking else 0)
        self.model.lacking = False
        assert self.table.tolist() == self.model.table
        assert self.refs.tolist() == self.model.refs
        assert self.len.tolist() == self.model.len
        assert torch.equal(self.pools.cpu(), self.model.pools)


def test_grow_shrink_free():
    b = Both(3, 8, 12)
    for seqs, lens in (([0, 2], [16, 1]), ([0], [17]), ([2, 1, 0], [33, 5, 17]), ([0, 1, 2], [0, 5, 16]), ([1], [128]),
                       ([0], [1])):
        b.resize(seqs, lens)
        b.check()


def test_no_pages_left():
    b = Both(4, 8, 10)
    b.resize([0, 1], [16 * 6, 16 * 3])
    b.check()
    b.resize([2, 3, 1], [17, 1, 16 * 3])  # two pages wanted, one there: sequence 3, behind, stays too
    b.check()
    b.resize([1, 3], [0, 16 * 5])  # what shrinking frees is there to grow on
    b.check()
    b.resize([0], [16 * 9])  # past the table's width
    b.check()
    b.resize([0, 2], [-1, 16])
    b.check()


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 16, 2 ** 30 + 1])
def test_lengths_that_no_row_holds(length):
    b = Both(3, 8, 12)
    b.resize([0, 1], [20, 5])
    b.resize([1, 0, 2], [length, 33, 16])
    b.check()


def test_fork_shares_and_copies():
    b = Both(8, 6, 24)
    b.resize([0, 1, 2], [40, 32, 5])
    b.fork([0, 1, 0, 2], [3, 4, 5, 6])
    b.check()
    b.resize([0], [0])  # the children hold its full pages
    b.check()
    b.fork([7], [0])  # of an empty one: nothing
    b.check()


def test_writing_into_a_shared_page_copies_it_first():
    b = Both(4, 6, 16)
    b.resize([0], [48])
    b.fork([0, 0], [1, 2])
    b.resize([1, 2], [20, 25])  # now both end inside a page that all three hold
    b.check()
    b.resize([1, 2], [21, 60])
    b.check()
    b.resize([0], [30])
    b.check()
    b.resize([0], [31])  # the others have left the page: no copy
    b.check()


def test_two_holders_leave_one_page_in_one_call():
    b = Both(3, 6, 9)
    b.resize([0], [32])
    b.fork([0], [1])
    b.resize([0, 1], [20, 20])
    b.check()
    b.resize([0, 1], [40, 24])
    b.check()
    b.resize([2], [16])  # the page both left is the lowest free one
    b.check()


def test_fork_without_room():
    b = Both(6, 4, 5)
    b.resize([0, 1], [17, 16])
    b.fork([0, 0, 1, 0], [2, 3, 4, 5])
    b.check()


def test_compact():
    b = Both(4, 8, 20)
    b.resize([0, 1, 2, 3], [70, 16, 50, 33])
    b.resize([0, 1], [0, 0])
    b.fork([2], [0])
    b.check()
    b.compact()
    b.check()
    b.compact()  # nothing left to move
    b.check()
    b.resize([2, 0, 3], [0, 0, 0])
    b.compact()
    b.check()


@pytest.mark.parametrize("n_pages,width,page,words", [(37, 9, 16, (4,)), (4096, 200, 1, (4,)), (4097, 300, 32, (1, 12)),
                                                     (9001, 2500, 3, (4,)), (300, 40, 256, (4100,))])
def test_random_rounds(n_pages, width, page, words):
    rng = random.Random(n_pages)
    n = 12
    b = Both(n, width, n_pages, page, 2, words, seed=n_pages)
    for _ in range(25):
        what = rng.random()
        if what < 0.6:
            seqs = rng.sample(range(n), rng.randint(1, n))
            top = min(width * page, 2 * n_pages * page // n)
            b.resize(seqs, [0 if rng.random() < 0.25 else rng.randint(0, top) for _ in seqs])
        elif what < 0.85:
            empty = [s for s in range(n) if b.model.len[s] == 0]
            full = [s for s in range(n) if b.model.len[s] > 0]
            if empty and full:
                b.fork([rng.choice(full) for _ in empty], empty)
        else:
            b.compact()
        b.check()


def test_many_sequences_in_one_call():
    n = 2500
    b = Both(n, 5, 9000, 16, 1, (4,))
    b.resize(list(range(n)), [(i * 13) % 70 for i in range(n)])
    b.check()
    order = list(range(n))
    random.Random(1).shuffle(order)
    b.resize(order, [(i * 29) % 80 for i in order])
    b.check()
    b.compact()
    b.check()


def test_copy():
    L = lib()
    for words in ((4,), (3, 20), (4096, 3)):
        b = Both(1, 1, 30, 16, 4, words)
        src, dst = [3, 5, 3, 29], [0, 1, 28, 7]
        L.tq1_pages_copy(b.pool, b.ints(src), b.ints(dst))
        b.model._copy(list(zip(src, dst)))
        b.check()
        L.tq1_pages_copy(b.pool, b.ints([3, 30, -1, 2]), b.ints([9, 4, 4, 30]))
        assert L.tq1_sync_status() == -8
        b.model._copy([(3, 9)])
        b.check()


def test_pools_apart_and_past_32_bits():
    # Two pools 5 GB apart: pages far behind the first 2^32 bytes.
    L = lib()
    room = torch.empty(2, 5 * 2 ** 30 // 65536, 65536, dtype=torch.uint8, device="cuda")
    n = room.shape[1]
    room[:, n - 1] = 7
    room[:, 5] = 0
    table, ln = torch.full((1, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = L.tq1_page_pool(room, table, ln, torch.zeros(n, dtype=torch.int32, device="cuda"), 16)
    L.tq1_pages_copy(pool, torch.tensor([n - 1], dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda"))
    assert L.tq1_sync_status() == 0
    assert (room[:, 5] == 7).all()


def test_bad_ids_are_skipped_and_reported():
    b = Both(3, 6, 12)
    b.resize([0, 1], [20, 40])
    b.check()
    b.L.tq1_pages_resize(b.pool, b.ints([-1, 3, 0]), b.ints([5, 5, 50]), b.ws)
    assert b.L.tq1_sync_status() == -8
    b.model.resize([0], [50])
    b.check()
    b.L.tq1_pages_fork(b.pool, b.ints([0, 3, 1]), b.ints([1, 2, -1]), b.ws)  # a full child, a bad parent, a bad child
    assert b.L.tq1_sync_status() == -8
    b.check()
