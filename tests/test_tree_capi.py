"""Trees and cache rows without a GPU: the oracle's definitions on hand-worked cases,
host-side refusals of the calls (nothing is launched), and the structures' layout."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import dsa_sparse_attention_gb300 as dsa
from dsa_sparse_attention_gb300.build import build
from oracle import dsa_oracle as O
from oracle import tree as OT

INC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include")


@pytest.fixture(scope="module")
def lib():
    build()
    return dsa.library()


# ------------------------------------------------------------------- the oracle

def test_visible_by_hand():
    #      0
    #    1   2
    #   3 4
    m = OT.ancestor_masks([-1, 0, 0, 1, 1], 1)
    assert m[:, 0].tolist() == [1, 3, 5, 11, 19]
    assert OT.visible(10, 14, m[4]).tolist() == list(range(10)) + [10, 11, 14]
    assert OT.visible(0, 2, m[2]).tolist() == [0, 2]
    assert OT.visible(5, 3, m[2]).tolist() == [0, 1, 2, 3]
    wide = OT.ancestor_masks(list(range(-1, 39)), 2)
    assert wide[39].tolist() == [0xFFFFFFFF, 0xFF] and OT.visible(7, 46, wide[39]).size == 47


def test_dense_mla_matches_the_sparse_oracle():
    rng = np.random.default_rng(0)
    lat = rng.standard_normal((9, 576))
    q = (rng.standard_normal((96, 576)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    o, l, a = OT.dense_mla(q, lat, 1 / 24)
    ro, rl = O.sparse_mla(q, lat, 1 / 24)
    assert np.allclose(o, ro) and np.allclose(l, rl) and np.all(a >= np.abs(o) - 1e-12)
    o, l, _ = OT.dense_mla(q, lat[:0], 1 / 24)
    assert not o.any() and np.all(np.isneginf(l))


def test_topk_by_hand():
    s = np.asarray([1.0, 5.0, 3.0, 5.0, np.nan, 2.0])
    assert OT.tree_topk(s, np.asarray([0, 1, 2, 3, 5]), 2).tolist() == [1, 3]
    assert OT.tree_topk(s, np.asarray([0, 2, 5]), 4).tolist() == [0, 2, 5, -1]
    assert OT.tree_topk(s, np.asarray([], dtype=np.int64), 2).tolist() == [-1, -1]


def test_pages_by_hand():
    p = OT.Pages([1, 1, 0, 0, 0], [[1, 0, -1], [-1] * 3, [-1] * 3], [5, 0, 0], 4)
    assert p.fork([0, 0], [1, 2]) == ([(0, 2), (0, 3)], False)
    assert p.ref == [1, 3, 1, 1, 0] and p.table[1] == [1, 2, -1] and p.ctx == [5, 5, 5]
    assert not p.free([0, 0])
    assert p.ref == [0, 2, 1, 1, 0]
    assert p.compact() == (3, [(3, 0)])
    assert p.ref == [1, 2, 1, 0, 0] and p.table == [[-1] * 3, [1, 2, -1], [1, 0, -1]]


# -------------------------------------------------------------------- refusals

WS = (0x100000, 1 << 32)


def _layout(**kw):
    args = dict(pool=0x10000, num_rows=100, row_stride=45312, idx_page_offset=0, lat_page_offset=8448)
    args.update(kw)
    return dsa.make_layout(args.pop("pool"), **args)


def _batch(T=2, B=2, max_ctx=1000, bt_stride=16, flags=0):
    return dsa.dsa_batch(T, B, 0x20000, 0x30000, 0x40000, 0x50000, bt_stride, flags, max_ctx)


def _tree(base=0x60000, mask=0x70000, words=2, reserved=0):
    return dsa.dsa_tree(base, mask, words, reserved)


def _pages(**kw):
    a = dict(ref_count=0x20000, block_table=0x30000, ctx_lens=0x40000, num_reqs=4, bt_stride=8)
    a.update(kw)
    return dsa.dsa_pages(*a.values())


def _r(x):
    return None if x is None else ctypes.byref(x)


BAD_TREES = [None, _tree(base=None), _tree(mask=None), _tree(words=0), _tree(words=33), _tree(reserved=1),
             _tree(mask=0x70002), _tree(base=0x60001)]


def test_tree_mla_refusals(lib):
    def call(lay=_layout(), bat=_batch(), tree=_tree(), q=0x80000, scale=0.04, out=0x90000, lse=0xA0000, ws=WS):
        return lib.dsa_tree_mla(_r(lay), _r(bat), _r(tree), q, scale, out, lse, *ws, None)
    for t in BAD_TREES:
        assert call(tree=t) == -1
    assert call(lay=None) == -1 and call(bat=None) == -1
    assert call(lay=_layout(block_size=48)) == -2 and call(lay=_layout(pool=0x10008)) == -1
    assert call(bat=_batch(max_ctx=16 * 64 + 1)) == -1 and call(bat=_batch(flags=8)) == -1
    assert call(bat=_batch(T=65536)) == -2
    for bad in (dict(q=None), dict(q=0x80008), dict(out=None), dict(out=0x90002), dict(lse=0xA0002),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == -1
    need = dsa.dsa_tree_workspace_size(_layout(), _batch())
    assert need > 0 and need % 256 == 0
    for ws in ((None, need), (0x100010, need), (0x100000, need - 1)):
        assert call(ws=ws) == -4
    assert call(bat=_batch(T=0), tree=_tree(base=None, mask=None), q=None, out=None) == 0   # nothing to do
    assert dsa.dsa_tree_workspace_size(_layout(block_size=48), _batch()) == 0


def test_tree_topk_refusals(lib):
    def call(lay=_layout(), bat=_batch(), tree=_tree(), scores=0x80000, ld=1000, k=2048, idx=0x90000, phys=None, ws=WS):
        return lib.dsa_tree_topk(_r(lay), _r(bat), _r(tree), scores, ld, k, idx, phys, *ws, None)
    for t in BAD_TREES:
        assert call(tree=t) == -1
    for bad in (dict(bat=None), dict(k=0), dict(k=2049), dict(ld=999), dict(ld=1002), dict(scores=None),
                dict(scores=0x80008), dict(idx=None), dict(lay=None, phys=0x1000)):
        assert call(**bad) == -1
    assert call(idx=0x90002) == -1 and call(phys=0x90001) == -1
    assert call(bat=_batch(T=65536)) == -2
    assert call(ws=(0x100000, 256)) == -4
    assert call(bat=_batch(T=0)) == 0


def test_tree_commit_refusals(lib):
    def call(lay=_layout(), bat=_batch(T=0), base=0x60000, acc=0x70000, m=4, new=None, ws=(0x100000, 256)):
        return lib.dsa_tree_commit(_r(lay), _r(bat), base, acc, m, new, *ws, None)
    for bad in (dict(lay=None), dict(bat=None), dict(base=None), dict(acc=None), dict(m=-1), dict(lay=_layout(pool=None)),
                dict(bat=_batch(max_ctx=16 * 64 + 1)), dict(bat=_batch(B=0)), dict(base=0x60002), dict(acc=0x70001),
                dict(new=0x80002)):
        assert call(**bad) == -1
    assert call(ws=(0x100000, 255)) == -4 and call(ws=(None, 256)) == -4


def test_cache_refusals(lib):
    L = _layout()
    need = dsa.dsa_cache_workspace_size(L, 4)
    assert need > 0 and need % 256 == 0
    assert dsa.dsa_cache_workspace_size(L, 0) == 0 and dsa.dsa_cache_workspace_size(_layout(block_size=8), 4) == 0
    ws = (0x100000, need)

    def copy(lay=L, src=0x20000, dst=0x30000, n=3, count=None, w=(0x100000, 256)):
        return lib.dsa_cache_copy(_r(lay), src, dst, n, count, *w, None)
    for bad in (dict(lay=None), dict(src=None), dict(dst=None), dict(n=-1), dict(lay=_layout(pool=None)),
                dict(src=0x20002), dict(dst=0x30001), dict(count=0x40002)):
        assert copy(**bad) == -1
    assert copy(w=(0x100000, 255)) == -4 and copy(n=0) == 0

    def fork(lay=L, pg=_pages(), a=0x50000, c=0x60000, n=4, s=0x70000, d=0x80000, w=ws):
        return lib.dsa_cache_fork(_r(lay), _r(pg), a, c, n, s, d, *w, None)
    bad_pages = [None, _pages(ref_count=None), _pages(block_table=None), _pages(ctx_lens=None), _pages(num_reqs=0),
                 _pages(bt_stride=0), _pages(ref_count=0x20001)]
    for pg in bad_pages:
        assert fork(pg=pg) == -1
        assert lib.dsa_cache_free(_r(L), _r(pg), 0x50000, 2, *ws, None) == -1
        assert lib.dsa_cache_compact(_r(L), _r(pg), _r(_pages()), 0x50000, 0x60000, 0x70000, *ws, None) == -1
        assert lib.dsa_cache_compact(_r(L), _r(_pages()), _r(pg), 0x50000, 0x60000, 0x70000, *ws, None) == -1
    for bad in (dict(a=None), dict(c=None), dict(s=None), dict(d=None), dict(n=-1), dict(n=5), dict(lay=None),
                dict(a=0x50001), dict(d=0x80002)):
        assert fork(**bad) == -1
    assert fork(w=(0x100000, need - 1)) == -4 and fork(n=0) == 0
    assert fork(lay=_layout(pool=None), n=0) == 0                     # the pool is not touched
    assert lib.dsa_cache_free(_r(L), _r(_pages()), None, 2, *ws, None) == -1
    assert lib.dsa_cache_free(_r(L), _r(_pages()), 0x50000, -1, *ws, None) == -1
    assert lib.dsa_cache_free(_r(L), _r(_pages()), 0x50000, 2, 0x100000, 255, None) == -4
    assert lib.dsa_cache_free(_r(L), _r(_pages()), None, 0, *ws, None) == 0
    comp = lambda to=_pages(), s=0x50000, d=0x60000, c=0x70000, w=ws: lib.dsa_cache_compact(
        _r(L), _r(_pages()), _r(to), s, d, c, *w, None)
    assert comp(s=None) == comp(d=None) == comp(c=None) == comp(to=_pages(num_reqs=3)) == comp(to=_pages(bt_stride=9)) == -1
    assert comp(w=(0x100000, need - 1)) == -4


def test_binding_refuses_what_the_abi_cannot_see():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    for base, mask in ((i(2), i(3)), (i(2), i(3, 2).long()), (i(2), i(3, 4)[:, ::2]), (i(2, 1), i(3, 2))):
        with pytest.raises(ValueError):
            dsa.make_tree(base, mask)
    for r, b, c in ((i(5), i(3, 4)[:, :2], i(3)), (i(5), i(3, 4), i(2)), (i(5).float(), i(3, 4), i(3))):
        with pytest.raises(ValueError):
            dsa.make_pages(r, b, c)
    lay, ws = _layout(), torch.zeros(1 << 12, dtype=torch.uint8)
    with pytest.raises(ValueError):
        dsa.dsa_cache_copy(lay, i(3), i(2), ws=ws)
    with pytest.raises(ValueError):
        dsa.dsa_cache_fork(lay, _pages(), i(3), i(3), i(2), i(3), ws=ws)
    with pytest.raises(ValueError):
        dsa.dsa_cache_compact(lay, _pages(), _pages(), i(49), i(50), i(2), ws=ws)
    with pytest.raises(ValueError):
        dsa.dsa_tree_commit(lay, _batch(), i(2), i(2, 8)[:, ::2], ws=ws)
    with pytest.raises(ValueError):
        dsa.dsa_tree_commit(lay, _batch(), i(2), i(1, 8), ws=ws)       # a row short
    for count in (i(1).long(), i(0)):
        with pytest.raises(ValueError):
            dsa.dsa_cache_copy(lay, i(2), i(2), count, ws=ws)


def test_structure_layout(tmp_path):
    gcc = shutil.which("gcc")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "dsa.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu\\n",'
                   'sizeof(dsa_tree),offsetof(dsa_tree,mask_words),sizeof(dsa_pages),offsetof(dsa_pages,ctx_lens),'
                   'offsetof(dsa_pages,num_reqs),offsetof(dsa_pages,bt_stride));return 0;}\n')
    exe = tmp_path / "s"
    subprocess.run([gcc, "-std=c99", "-I", INC, str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(dsa.dsa_tree), dsa.dsa_tree.mask_words.offset, ctypes.sizeof(dsa.dsa_pages),
                   dsa.dsa_pages.ctx_lens.offset, dsa.dsa_pages.num_reqs.offset, dsa.dsa_pages.bt_stride.offset]
