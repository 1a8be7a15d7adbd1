"""Rows of the cache on the GPU: copy, fork, free and compaction against plain lists
(oracle/tree.py).  Every result is exact."""
import numpy as np
import pytest
import torch

from oracle import tree as OT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_sparse_attention_gb300.build import build
    build()


class Dev:
    """Counts, tables, lengths and a pool of random bytes on the GPU, and the plain copy."""

    def __init__(self, rows, lens, bs=64, seed=0, stride=None, used=None, extra=0, row_pad=0):
        import dsa_sparse_attention_gb300 as dsa
        rng = np.random.default_rng(seed)
        nb = [-(-L // bs) for L in lens]
        stride = stride or max(nb + [1]) + 1
        perm = rng.permutation(rows)
        table = np.full((len(lens), stride), -1, np.int32)
        at = 0
        for r, n in enumerate(nb):
            table[r, :n] = perm[at:at + n]
            at += n
        ref = np.zeros(rows, np.int32)
        ref[perm[:at + extra]] = 1                  # `extra` rows held elsewhere
        self.rb = bs * 708 + row_pad
        self.pool = torch.from_numpy(rng.integers(0, 256, (rows, self.rb), dtype=np.uint8)).cuda()
        cu = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
        self.ref, self.table, self.ctx = cu(ref), cu(table), cu(lens)
        self.layout = dsa.make_layout(self.pool, rows, self.rb, 0, bs * 132, bs)
        self.pages = dsa.make_pages(self.ref, self.table, self.ctx)
        self.ws = dsa.alloc_cache_workspace(self.layout, len(lens))
        self.plain = OT.Pages(ref, table, lens, bs)
        self.dsa = dsa

    def check(self, st=0):
        torch.cuda.synchronize()
        assert self.dsa.dsa_check(self.ws) == st
        assert self.ref.cpu().tolist() == self.plain.ref
        assert self.table.cpu().tolist() == self.plain.table
        assert self.ctx.cpu().tolist() == self.plain.ctx

    def fork(self, parent, child):
        cu = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        src, dst = torch.full((2, len(parent)), -9, dtype=torch.int32, device="cuda")
        self.dsa.dsa_cache_fork(self.layout, self.pages, cu(parent), cu(child), src, dst, ws=self.ws)
        pairs, bad = self.plain.fork(parent, child)
        self.check(-6 if bad else 0)
        assert list(zip(src.cpu().tolist(), dst.cpu().tolist())) == pairs
        return src, dst

    def free(self, reqs):
        self.dsa.dsa_cache_free(self.layout, self.pages, torch.tensor(reqs, dtype=torch.int32, device="cuda"), ws=self.ws)
        bad = self.plain.free(reqs)
        self.check(-6 if bad else 0)

    def copy(self, src, dst, count=None):
        want = self.pool.cpu().numpy().copy()
        n = src.numel() if count is None else max(0, min(src.numel(), int(count)))
        rows = want.copy()
        for s, d in zip(src.cpu().tolist()[:n], dst.cpu().tolist()[:n]):
            if 0 <= s < len(rows) and 0 <= d < len(rows):
                want[d] = rows[s]
        self.dsa.dsa_cache_copy(self.layout, src, dst, count, ws=self.ws)
        torch.cuda.synchronize()
        assert np.array_equal(self.pool.cpu().numpy(), want)


@pytest.mark.parametrize("bs,row_pad", [(16, 0), (64, 16), (256, 4096)])
def test_copy(bs, row_pad):
    d = Dev(70, [1], bs=bs, seed=bs, row_pad=row_pad)
    cu = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    d.copy(cu([3, 3, -1, 9, 12, 69]), cu([5, 0, -1, 9, 68, 1]))       # a repeated source, a skipped pair, in place
    d.copy(cu([1, 2, 3]), cu([10, 11, 12]), cu([2]))
    d.copy(cu([1, 2, 3]), cu([10, 11, 12]), cu([0]))
    d.copy(cu([7, 8]), cu([20, 21]), cu([99]))
    d.copy(cu([]), cu([]))
    assert d.dsa.dsa_check(d.ws) == 0
    for s, t in (([4, -1], [30, 31]), ([4, 70], [32, 33]), ([4, 5], [34, 1 << 30])):
        d.copy(cu(s), cu(t))
        assert d.dsa.dsa_check(d.ws) == -6


def test_copy_past_32_bits():
    # a row whose byte offset needs 33 bits
    import dsa_sparse_attention_gb300 as dsa
    rb = 256 * 708
    rows = (1 << 33) // rb + 3
    pool = torch.empty((rows, rb), dtype=torch.uint8, device="cuda")
    pool[5] = torch.randint(0, 256, (rb,), dtype=torch.uint8, device="cuda")
    layout = dsa.make_layout(pool, rows, rb, 0, 256 * 132, 256)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cu = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_copy(layout, cu([5]), cu([rows - 1]), ws=ws)
    dsa.dsa_cache_copy(layout, cu([rows - 1]), cu([6]), ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(pool[6], pool[5]) and torch.equal(pool[rows - 1], pool[5])


@pytest.mark.parametrize("bs", [16, 64])
def test_fork_free(bs):
    d = Dev(400, [100, bs * 5, 1, 0, bs * 7 + 1] + [0] * 12, bs=bs, seed=1)
    src, dst = d.fork([0, 0, 1, 2, -1, 3, 4, 4], [5, 6, 7, 8, 9, 10, 11, 12])
    d.copy(src, dst)
    d.fork([5, 11], [13, 14])                     # forks of forks
    d.free([5, 6, 6, -1, 12])                     # named twice: freed once
    d.fork([0, 4, 4], [12, 5, 6])                 # the lowest free rows are reused
    d.free([0, 1, 2, 3, 4])                       # parents first: the children keep what they share
    d.free(list(range(17)))
    assert sum(d.plain.ref) == 0


def test_fork_refusals():
    d = Dev(60, [100, 128, 70] + [0] * 6, seed=2)
    d.fork([0, 0, 1], [3, 3, 4])                  # a child named twice: neither is made
    d.fork([0, 1, 2], [2, 5, 6])                  # a child that holds something and is a parent
    d.fork([9, 0, 0, 1], [5, 9, -1, 1])           # ids outside the table, a fork of itself
    d.free([99, 4])
    d.fork([0], [4])


def test_fork_out_of_rows():
    # 8 rows, 5 held: three forks get a row, in order, the rest are left out; full blocks need none
    d = Dev(8, [65, 128, 1] + [0] * 8, seed=3)
    d.fork([0, 2, 1, 0, 0, 1, 2], [3, 4, 5, 6, 7, 8, 9])


def test_fork_many_rows_and_forks():
    # more rows and forks than one round of the scan takes; free rows lie late
    n = 1500
    rows = 40000
    d = Dev(rows, [70, 64, 1] + [0] * n, seed=4, bs=16, extra=rows - 2000)
    d.fork([i % 3 for i in range(n)], [3 + i for i in range(n)])
    d.free([3 + i for i in range(0, n, 2)])
    d.fork([2] * 700, [3 + 2 * i for i in range(700)])


def test_free_records_bad_state():
    d = Dev(40, [200, 300], seed=5)
    d.table[0, 1] = 4000
    d.plain.table[0][1] = 4000
    d.free([0])
    b = d.plain.table[1][2]
    d.ref[b] = 0
    d.plain.ref[b] = 0
    d.free([1])


def _compact(d, alias, copy=True):
    dsa = d.dsa
    cap = max(1, d.ref.numel() // 2)
    src, dst = torch.full((2, cap), -9, dtype=torch.int32, device="cuda")
    counts = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    ref, table = (d.ref, d.table) if alias else (torch.full_like(d.ref, -9), torch.full_like(d.table, -9))
    to = dsa.make_pages(ref, table, d.ctx)
    before = d.pool.cpu().numpy().copy()
    old = [r[:] for r in d.plain.table]
    dsa.dsa_cache_compact(d.layout, d.pages, to, src, dst, counts, ws=d.ws)
    dsa.dsa_cache_copy(d.layout, src, dst, counts[1:], ws=d.ws)
    L, moves = d.plain.compact()
    d.ref, d.table = ref, table
    d.pages = to
    torch.cuda.synchronize()
    assert counts.cpu().tolist() == [L, len(moves)]
    pad = [(-1, -1)] * (cap - len(moves))
    assert list(zip(src.cpu().tolist(), dst.cpu().tolist())) == moves + pad
    after = d.pool.cpu().numpy()
    for r, row in enumerate(d.plain.table):      # every request still finds its content
        for e, b in enumerate(row):
            if b >= 0:
                assert np.array_equal(after[b], before[old[r][e]])


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("rows", [1, 2, 37, 300, 9001])
def test_compact(rows, alias):
    bs = 16
    lens = [0, 1] if rows < 30 else [rows // 6 * bs, 100, 0, rows // 5 * bs + 3]
    lens = [min(L, (rows // 2) * bs) for L in lens]
    d = Dev(rows, lens + [0], bs=bs, seed=rows)
    if rows > 30:
        d.fork([3], [4])
        d.free([1])
    _compact(d, alias)
    d.check()
    _compact(d, alias)                           # nothing left to move
    d.check()


def test_compact_extremes():
    d = Dev(64, [0, 0], seed=6)                  # nothing used
    _compact(d, False)
    d.check()
    d = Dev(20, [64 * 20], seed=7)               # everything used
    _compact(d, True)
    d.check()
    d = Dev(30, [64 * 4, 64 * 2], seed=8)        # an entry that names a free row
    b = d.plain.table[0][1]
    d.ref[b] = 0
    d.plain.ref[b] = 0
    _compact(d, False)
    d.check(-6)


def test_cache_calls_in_a_graph():
    # free, fork and copy captured once and replayed: the replays give the same state
    dsa = __import__("dsa_sparse_attention_gb300")
    d = Dev(300, [1000, 777] + [0] * 6, seed=9)
    cu = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    parent, child = cu([0, 1, 0, 1, 0, 1]), cu([2, 3, 4, 5, 6, 7])
    src, dst = torch.empty((2, 6), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_cache_free(d.layout, d.pages, child, ws=d.ws)
        dsa.dsa_cache_fork(d.layout, d.pages, parent, child, src, dst, ws=d.ws)
        dsa.dsa_cache_copy(d.layout, src, dst, ws=d.ws)
    pairs, _ = d.plain.fork([0, 1, 0, 1, 0, 1], [2, 3, 4, 5, 6, 7])
    for _ in range(3):
        g.replay()
        d.check()
        assert list(zip(src.cpu().tolist(), dst.cpu().tolist())) == pairs
        for s, t in pairs:
            assert torch.equal(d.pool[s], d.pool[t])


@pytest.mark.parametrize("alias", [False, True])
def test_compact_in_a_cluster(alias):
    # more rows than one CTA plans, and tables that take a launch of their own
    bs, rows = 16, 20011
    d = Dev(rows, [rows // 3 * bs, 100, 0, rows // 4 * bs + 5, 0], bs=bs, seed=31, stride=20000, extra=500)
    d.fork([3], [4])
    d.free([1])
    _compact(d, alias)
    d.check()
    _compact(d, alias)
    d.check()


def test_cache_calls_behind_a_memset_in_a_graph():
    # what a memset or a copy writes in front of a call in the same graph is seen by it
    dsa = __import__("dsa_sparse_attention_gb300")
    d = Dev(300, [1000, 777] + [0] * 2, seed=32)
    cu = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    parent, child = cu([0, 1]), cu([2, 3])
    table, ref, ctx = d.table.clone(), d.ref.clone(), d.ctx.clone()
    src, dst = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for x, y in ((d.table, table), (d.ref, ref), (d.ctx, ctx)):
            x.zero_()
            x.copy_(y)
        dsa.dsa_cache_fork(d.layout, d.pages, parent, child, src, dst, ws=d.ws)
        dsa.dsa_cache_copy(d.layout, src, dst, ws=d.ws)
    pairs, _ = d.plain.fork([0, 1], [2, 3])
    for _ in range(5):
        d.table.fill_(-1)
        g.replay()
        d.check()
        assert list(zip(src.cpu().tolist(), dst.cpu().tolist())) == pairs
    for s, t in pairs:
        assert torch.equal(d.pool[s], d.pool[t])
