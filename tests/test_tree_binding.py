"""The binding's checks of the tree and cache calls' tensors (CPU): lengths, types and places that the
C ABI cannot see, each refused before the library is called, and the forms that are allowed."""
import pytest
import torch

import dsa_sparse_attention_gb300 as dsa


class OnDevice:
    """Looks like a device tensor and has a host tensor's shape, strides and address."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def i32(*shape):
    return OnDevice(torch.zeros(shape, dtype=torch.int32))


def arr(dtype, *shape):
    return OnDevice(torch.zeros(shape, dtype=dtype))


class Library:
    """Notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture()
def lib(monkeypatch):
    r = Library()
    monkeypatch.setattr(dsa, "library", lambda: r)
    monkeypatch.setattr(dsa, "_handle", lambda stream: 77)
    return r


def refused(lib, call, *args, **kw):
    before = len(lib.calls)
    with pytest.raises(ValueError):
        call(*args, **kw)
    assert len(lib.calls) == before


T, B, BF, F32 = 3, 2, torch.bfloat16, torch.float32
LAY = dsa.make_layout(None, 100, 45312, 0, 8448)


def batch():
    return dsa.dsa_batch(T, B, 0x20000, 0x30000, 0x40000, 0x50000, 16, 0, 1000)


def ws():
    return arr(torch.uint8, 4096)


def test_tree_mla(lib):
    tree = dsa.make_tree(i32(B), i32(T, 2))
    q, out, lse = arr(BF, T, 96, 576), arr(BF, T, 96, 512), arr(F32, T, 96)
    dsa.dsa_tree_mla(LAY, batch(), tree, q, 0.04, out, lse, ws=ws())
    dsa.dsa_tree_mla(LAY, batch(), tree, q, 0.04, out, ws=ws())
    dsa.dsa_tree_mla(LAY, batch(), tree, arr(BF, (T + 4) * 96 * 576), 0.04, arr(BF, T + 1, 96, 512), ws=ws())   # longer
    dsa.dsa_tree_mla(LAY, batch(), dsa.make_tree(i32(B + 3), i32(T + 1, 1)), q, 0.04, out, ws=ws())
    dsa.dsa_tree_mla(LAY, batch(), dsa.dsa_tree(1, 2, 1, 0), 0x1000, 0.04, 0x2000, ws=ws())      # addresses
    assert len(lib.calls) == 5 and lib.calls[0][1][3] == q.data_ptr() and lib.calls[0][1][-1] == 77
    for t in (dsa.make_tree(i32(B - 1), i32(T, 2)), dsa.make_tree(i32(B), i32(T - 1, 2))):
        refused(lib, dsa.dsa_tree_mla, LAY, batch(), t, q, 0.04, out, ws=ws())
    wrong = [dict(q=arr(BF, T - 1, 96, 576)), dict(q=arr(torch.float16, T, 96, 576)), dict(q=OnDevice(arr(BF, T, 576, 96).t.transpose(1, 2))),
             dict(q=q.t), dict(out=arr(BF, T, 96, 511)), dict(out=arr(F32, T, 96, 512)), dict(out=out.t),
             dict(lse=arr(F32, T, 95)), dict(lse=arr(BF, T, 96)), dict(lse=lse.t), dict(ws=ws().t)]
    for w in wrong:
        a = dict(q=q, out=out, lse=lse, ws=ws())
        a.update(w)
        refused(lib, dsa.dsa_tree_mla, LAY, batch(), tree, a["q"], 0.04, a["out"], a["lse"], ws=a["ws"])


def test_tree_topk(lib):
    tree, ld, k = dsa.make_tree(i32(B), i32(T, 2)), 1000, 64
    scores, idx = arr(F32, T, ld), i32(T, k)
    wide = torch.zeros(T, ld + 24, dtype=F32)
    ok = lambda s, l=ld, **kw: dsa.dsa_tree_topk(LAY, batch(), tree, s, l, k, kw.pop("idx", idx), ws=ws(), **kw)
    ok(scores)
    ok(scores, phys_slots=i32(T, k))
    ok(OnDevice(wide[:, :ld]), ld + 24)                       # a view of the first columns
    refused(lib, ok, OnDevice(wide[:, 24:]), ld + 24)         # of the last ones: the last row would end behind the array
    one = dsa.dsa_batch(1, B, 1, 2, 3, 4, 16, 0, 1000)
    dsa.dsa_tree_topk(LAY, one, tree, OnDevice(wide[:1, :ld]), ld + 24, k, idx, ws=ws())
    assert len(lib.calls) == 4
    for s, l in ((arr(F32, T - 1, ld), ld), (arr(torch.float64, T, ld), ld), (scores.t, ld), (OnDevice(wide[:, :ld]), ld),
                 (OnDevice(wide.t()), T), (scores, ld + 4), (OnDevice(wide[:2, :ld]), ld + 24)):
        refused(lib, ok, s, l)
    for j in (i32(T, k - 1), arr(torch.int64, T, k), i32(T, k).t, OnDevice(i32(T, 2 * k).t[:, ::2])):
        refused(lib, ok, scores, idx=j)
        refused(lib, ok, scores, phys_slots=j)
    refused(lib, dsa.dsa_tree_topk, LAY, batch(), dsa.make_tree(i32(B), i32(T - 1, 2)), scores, ld, k, idx, ws=ws())


def test_tree_commit(lib):
    dsa.dsa_tree_commit(LAY, batch(), i32(B), i32(B, 4), i32(B), ws=ws())
    dsa.dsa_tree_commit(LAY, batch(), i32(B + 1), i32(B, 4), ws=ws())
    assert len(lib.calls) == 2
    refused(lib, dsa.dsa_tree_commit, LAY, batch(), i32(B - 1), i32(B, 4), i32(B), ws=ws())
    refused(lib, dsa.dsa_tree_commit, LAY, batch(), i32(B), i32(B, 4), i32(B - 1), ws=ws())
    refused(lib, dsa.dsa_tree_commit, LAY, batch(), i32(B), i32(B - 1, 4), i32(B), ws=ws())
    for bad in (dict(base=i32(B).t), dict(acc=i32(B, 4).t), dict(new=i32(B).t), dict(w=ws().t)):
        a = dict(base=i32(B), acc=i32(B, 4), new=i32(B), w=ws())
        a.update(bad)
        refused(lib, dsa.dsa_tree_commit, LAY, batch(), a["base"], a["acc"], a["new"], ws=a["w"])


def test_pages(lib):
    good = dsa.make_pages(i32(100), i32(4, 8), i32(4))
    short = dsa.make_pages(i32(99), i32(4, 8), i32(4))
    host = lambda *s: torch.zeros(s, dtype=torch.int32)
    for r, t, c in ((host(100), i32(4, 8), i32(4)), (i32(100), host(4, 8), i32(4)), (i32(100), i32(4, 8), host(4))):
        with pytest.raises(ValueError):
            dsa.make_pages(r, t, c)
    dsa.dsa_cache_fork(LAY, good, i32(2), i32(2), i32(2), i32(2), ws=ws())
    dsa.dsa_cache_free(LAY, good, i32(2), ws=ws())
    dsa.dsa_cache_compact(LAY, good, good, i32(50), i32(50), i32(2), ws=ws())
    dsa.dsa_cache_copy(LAY, i32(2), i32(2), i32(1), ws=ws())
    assert [c[0] for c in lib.calls] == ["dsa_cache_fork", "dsa_cache_free", "dsa_cache_compact", "dsa_cache_copy"]
    refused(lib, dsa.dsa_cache_fork, LAY, short, i32(2), i32(2), i32(2), i32(2), ws=ws())
    refused(lib, dsa.dsa_cache_free, LAY, short, i32(2), ws=ws())
    refused(lib, dsa.dsa_cache_compact, LAY, short, good, i32(50), i32(50), i32(2), ws=ws())
    refused(lib, dsa.dsa_cache_compact, LAY, good, short, i32(50), i32(50), i32(2), ws=ws())
    refused(lib, dsa.dsa_cache_copy, LAY, i32(2), i32(2), host(1), ws=ws())
    refused(lib, dsa.dsa_cache_copy, LAY, host(2), i32(2), ws=ws())
    refused(lib, dsa.dsa_cache_copy, LAY, i32(2), i32(2), ws=ws().t)
    refused(lib, dsa.dsa_cache_free, LAY, good, host(2), ws=ws())
