"""Page bookkeeping of more sequences than one round of a call's threads takes, and
of pools of more pages than one kernel counts, against the plain Python model."""
import random

import pytest
import torch

from .gpu_util import lib
from .kv_ref import Pages

pytestmark = pytest.mark.gpu


class Both:
    """The library's state and the model's, side by side; pages of 16 bytes."""

    def __init__(self, n_seqs, width, n_pages, page=16):
        self.L = lib()
        pools = torch.arange(4 * n_pages, dtype=torch.int32).view(1, n_pages, 1, 4)
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
        self.check()

    def fork(self, parents, children):
        self.L.tq1_pages_fork(self.pool, self.ints(parents), self.ints(children), self.ws)
        self.model.fork(parents, children)
        self.check()

    def compact(self):
        self.L.tq1_pages_compact(self.pool, self.ws)
        self.model.compact()
        self.check()

    def check(self):
        assert self.L.tq1_sync_status() == (-9 if self.model.lacking else 0)
        self.model.lacking = False
        assert self.table.tolist() == self.model.table
        assert self.refs.tolist() == self.model.refs
        assert self.len.tolist() == self.model.len
        assert torch.equal(self.pools.cpu(), self.model.pools)


@pytest.mark.parametrize("n_pages", [65536, 65537, 70000, 17 * 4096])
@pytest.mark.parametrize("stay", [8 * 4096, 8 * 4096 + 1, 30001, 5])
def test_compact_large_pools(n_pages, stay):
    # The pages that stay lie behind those of a sequence that leaves, in two
    # runs with a hole between them; `stay` pages: within a chunk of the count
    # and on its boundary.
    b = Both(5, n_pages, n_pages, page=1)
    half = stay // 2
    room = n_pages - stay
    b.resize([0, 1, 2, 3], [room // 2, half, room - room // 2 - 3, stay - half])
    b.compact()  # nothing to move
    b.resize([0, 2], [0, 0])
    b.compact()
    b.resize([4], [n_pages - stay])  # the whole pool
    b.compact()
    b.resize([1], [0])
    b.compact()
    b.resize([3, 4], [0, 0])
    b.compact()  # none in use


def test_fork_more_children_than_threads():
    n = 2600
    b = Both(5 + n, 4, 3200)
    b.resize([0, 1, 2, 3], [40, 32, 5, 17])
    rng = random.Random(7)
    children = list(range(5, 5 + n))
    rng.shuffle(children)
    parents = [rng.choice([0, 0, 1, 2, 2, 3, 4]) for _ in children]
    b.fork(parents, children)
    b.resize([0, 2], [0, 0])
    b.resize(children, [rng.choice([0, 3, 16, 30]) for _ in children])
    b.compact()


@pytest.mark.parametrize("n_pages", [700, 1100, 2300])
def test_fork_more_children_than_pages(n_pages):
    n = 2500
    b = Both(3 + n, 4, n_pages)
    b.resize([0, 1, 2], [40, 32, 5])
    b.fork([i % 3 for i in range(n)], list(range(3, 3 + n)))


@pytest.mark.parametrize("n,n_pages", [(1500, 4000), (1500, 900), (2300, 2100), (1025, 1026)])
def test_more_sequences_than_threads_leave_shared_pages(n, n_pages):
    # All children end inside a page that they share, then grow: each takes a
    # copy of its own (as far as there are pages), the page they leave is free
    # afterwards only when all of them have left it.
    b = Both(1 + n, 6, n_pages)
    b.resize([0], [48])
    b.fork([0] * n, list(range(1, n + 1)))
    rng = random.Random(n)
    order = list(range(n + 1))
    rng.shuffle(order)
    b.resize(order, [20] * (n + 1))
    rng.shuffle(order)
    b.resize(order, [rng.choice([19, 20, 21, 30, 33, 70]) for _ in order])
    rng.shuffle(order)
    b.resize(order, [rng.choice([0, 5, 22, 40]) for _ in order])
    b.compact()
