"""The block table's operations on the GPU against the oracle on Python lists: tables, lengths, counts, status and every
byte of the pools have to be equal."""

import random

import numpy as np
import pytest
import torch

from oracle import pages
from rotated_bit_kv_iq_b200 import binding as B
from tests._helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_bit_kv_iq_b200 import build

    build.build()
    B.lib()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """A table with a 3-bit and an 8-bit cache on the GPU, and the oracle's with copies of their pools."""

    def __init__(self, seqs, per, ps, n_pages, seed=0, hkv=2, layers=2):
        self.pt = B.PageTable(seqs, per, ps, n_pages)
        g = torch.Generator().manual_seed(seed)
        self.guards, shapes = [], []
        for tb in (3200, 8224):
            n = layers * n_pages * hkv * (ps // 32) * tb
            gd = Guarded((n,), torch.uint8)
            gd.t.copy_(torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8))
            self.guards.append(gd)
            shapes.append((layers, n_pages, hkv, ps // 32, tb))
        caches = [B.PagedCache(layers, hkv, ps, n_pages, block_table=self.pt.block_table),
                  B.PagedCache8(layers, hkv, ps, n_pages, block_table=self.pt.block_table, pool=self.guards[1].t)]
        caches[0].pool = self.guards[0].t
        self.pools = B.PagePool.of(*caches)
        self.o = pages.Pages(seqs, per, ps, n_pages,
                             [gd.t.cpu().numpy().reshape(s).copy() for gd, s in zip(self.guards, shapes)])

    def check(self):
        torch.cuda.synchronize()
        assert self.pt.block_table.tolist() == self.o.table
        assert self.pt.seq_len.tolist() == self.o.len
        assert self.pt.ref.tolist() == self.o.ref
        assert self.pt.status.item() == self.o.status
        for gd, want in zip(self.guards, self.o.pools):
            gd.check("pool")
            np.testing.assert_array_equal(gd.t.cpu().numpy().reshape(want.shape), want)

    def extend(self, ids, lens):
        B.iq_pages_extend(self.pt, _i32(ids), _i32(lens))
        self.o.extend(ids, lens)

    def free(self, ids):
        B.iq_pages_free(self.pt, _i32(ids))
        self.o.free(ids)

    def fork(self, p, c):
        B.iq_pages_fork(self.pt, self.pools, _i32(p), _i32(c))
        self.o.fork(p, c)

    def compact(self):
        n = torch.zeros(1, dtype=torch.int32, device=DEV)
        B.iq_pages_compact(self.pt, self.pools, n)
        assert n.item() == self.o.compact()

    def copy(self, s, d):
        B.iq_pages_copy(self.pt, self.pools, _i32(s), _i32(d))
        self.o.copy(s, d)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("ps", [32, 96])
def test_random_schedules(seed, ps):
    """Sequences come, grow, fork, end and are compacted in a random order, with calls that must be refused in between."""
    r = random.Random(seed)
    t = Both(9, 5, ps, 24, seed)
    for step in range(14):
        op = r.choice(["extend", "extend", "fork", "free", "compact", "copy"])
        n = r.randint(0, 5)
        ids = [r.randint(-1, 9) for _ in range(n)]
        if op == "extend":
            t.extend(ids, [r.choice([0, 1, r.randint(0, 5 * ps), 5 * ps, 5 * ps + 1]) for _ in ids])
        elif op == "fork":
            t.fork(ids, [r.randint(-1, 9) for _ in ids])
        elif op == "free":
            t.free(ids)
        elif op == "copy":
            t.copy([r.randint(-1, 24) for _ in ids], [r.randint(-1, 24) for _ in ids])
        else:
            t.compact()
        t.check()


def test_running_out_of_pages():
    t = Both(6, 4, 64, 7)
    t.extend([0, 1, 2, 3], [200, 150, 10, 1])  # 4 + 3 pages: 2 and 3 are refused
    t.check()
    assert t.o.status == pages.NOPAGE and t.o.len[:4] == [200, 150, 0, 0]
    t.fork([0, 1], [4, 5])  # part-filled tails and no page for them
    t.check()
    t.free([1, 1, 17])
    t.fork([0, 0], [4, 4])
    t.check()
    assert t.o.ref[:3] == [2, 2, 2]
    t.extend([0], [256])  # within its last page
    t.extend([4, 0], [256, 256])
    t.check()


def test_requests_whose_sum_passes_32_bits():
    """2048 sequences of up to 2^20 pages each ask for 2^31 of a pool's 8: all but the first few are refused."""
    n, per = 2050, 1 << 20
    t = B.PageTable(n, per, 32, 8)
    lens = [33] + [per * 32] * (n - 2) + [1]
    B.iq_pages_extend(t, _i32(list(range(n))), _i32(lens))
    assert t.status.item() == B.IQ_DEVERR_NOPAGE
    assert t.seq_len.tolist() == [33] + [0] * (n - 1)
    assert t.ref.tolist() == [1, 1] + [0] * 6
    assert t.block_table[0, :3].tolist() == [0, 1, -1] and int((t.block_table >= 0).sum()) == 2


def test_forks_of_forks_share_pages_and_a_whole_page_needs_none():
    t = Both(8, 3, 32, 16)
    t.extend([0, 1], [64, 65])
    t.fork([0, 1, 0], [2, 3, 4])
    t.check()
    t.fork([2, 3, 5, 2], [5, 6, 7, 2])  # 5 was empty before the call: so is 7; 2 cannot be its own child
    t.check()
    t.free([0, 2, 4, 5])
    t.check()
    assert sum(x > 0 for x in t.o.ref) == 5
    t.compact()
    t.compact()
    t.check()


def test_many_sequences_and_pages():
    """Lists and pools of more than one pass of the planning kernels."""
    seqs, n_pages = 3000, 20000
    pt = B.PageTable(seqs, 8, 32, n_pages)
    o = pages.Pages(seqs, 8, 32, n_pages)
    r = random.Random(1)
    ids = list(range(seqs))
    r.shuffle(ids)
    lens = [r.randint(0, 256) for _ in ids]
    B.iq_pages_extend(pt, _i32(ids), _i32(lens))
    o.extend(ids, lens)
    gone = r.sample(range(seqs), 1700)
    B.iq_pages_free(pt, _i32(gone))
    o.free(gone)
    B.iq_pages_compact(pt, None)
    o.compact()
    alive = [i for i in range(seqs) if o.len[i]]
    par = [r.choice(alive) for _ in gone]
    B.iq_pages_fork(pt, None, _i32(par), _i32(gone))
    o.fork(par, gone)
    torch.cuda.synchronize()
    assert pt.block_table.tolist() == o.table and pt.ref.tolist() == o.ref and pt.seq_len.tolist() == o.len
    assert pt.status.item() == o.status


def test_empty_lists_and_graph_capture():
    t = Both(4, 3, 64, 9)
    t.extend([], [])
    t.free([])
    t.fork([], [])
    t.copy([], [])
    t.compact()
    t.check()
    ids, lens, kids = _i32([0, 1]), _i32([100, 64]), _i32([2, 3])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.iq_pages_extend(t.pt, ids, lens)
        B.iq_pages_fork(t.pt, t.pools, ids, kids)
        B.iq_pages_free(t.pt, ids)
        B.iq_pages_compact(t.pt, t.pools)
        B.iq_pages_free(t.pt, kids)
    for _ in range(2):
        g.replay()
        t.o.extend([0, 1], [100, 64])
        t.o.fork([0, 1], [2, 3])
        t.o.free([0, 1])
        t.o.compact()
        t.o.free([2, 3])
        t.check()


def test_binding_refusals():
    t = Both(4, 3, 64, 9)
    other = Both(4, 3, 64, 8)
    with pytest.raises(ValueError):
        B.iq_pages_fork(t.pt, other.pools, _i32([0]), _i32([1]))
    with pytest.raises(ValueError):
        B.iq_pages_fork(t.pt, t.pools, _i32([0]), _i32([1, 2]))
    with pytest.raises(ValueError):
        B.iq_pages_extend(t.pt, _i32([0]), torch.tensor([1], device=DEV))
    with pytest.raises(B.IqError):
        B.iq_pages_free(t.pt, _i32([0] * 4097))
    t.check()
