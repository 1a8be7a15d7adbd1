"""Prompt calls without a GPU: the oracle on hand-worked cases, refusals of the C ABI (nothing is launched)
and of the binding, and the structures' layout."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import dsa_sparse_attention_gb300 as dsa
from dsa_sparse_attention_gb300.build import build
from oracle import prompt as P
from tests.test_tree_binding import OnDevice, Library, refused   # noqa: F401

INC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include")


@pytest.fixture(scope="module")
def lib():
    build()
    return dsa.library()


# ------------------------------------------------------------------- the oracle

def test_attention_by_hand():
    q = np.zeros((2, 2, 1))
    k, v = np.zeros((3, 1, 1)), np.asarray([1.0, 3.0, 8.0]).reshape(3, 1, 1)
    out, lse, A, big = P.attention(q, k, v, 1.0, True)          # query 0 sits at position 1
    assert np.allclose(out[:, :, 0], [[2, 2], [4, 4]]) and np.allclose(lse, np.log([[2, 2], [3, 3]]))
    assert np.allclose(A, out) and not big.any()
    out, lse, _, _ = P.attention(q, k[:1], v[:1], 1.0, True)    # query 0 sees nothing
    assert np.isneginf(lse[0]).all() and not out[0].any() and np.allclose(out[1], 1.0) and not lse[1].any()
    q[:, 0], k[2] = np.log(3.0), 1.0                            # head 0 weighs the last key three times
    out, lse, _, big = P.attention(q, k, v, 1.0, False)
    assert np.allclose(out[0, :, 0], [28 / 5, 4]) and np.allclose(lse[0], np.log([5, 3])) and np.allclose(big[0], [np.log(3), 0])
    shared = P.attention(q, np.zeros((3, 1, 0)), np.zeros((3, 1, 0)), 1.0, False, k[:, 0])
    assert np.allclose(shared[1], lse)


def test_attention_is_softmax_attention():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    q, k, v, ks = r(5, 4, 12), r(9, 2, 8), r(9, 2, 8), r(9, 4)
    full = torch.cat((k, ks[:, None].expand(9, 2, 4)), 2).repeat_interleave(2, 1)
    mask = torch.ones(5, 9, dtype=torch.bool).tril(4)
    ref = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), full.transpose(0, 1),
                                                           v.repeat_interleave(2, 1).transpose(0, 1), mask, scale=0.3)
    out = P.attention(q.numpy(), k.numpy(), v.numpy(), 0.3, True, ks.numpy())[0]
    assert np.allclose(out, ref.transpose(0, 1).numpy())


def test_join_is_attention_over_both():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    a, b, c = (P.attention(q, k[s], v[s], 0.5, False)[:2] for s in (slice(0, 4), slice(4, 7), slice(0, 7)))
    out, lse, _, _ = P.join(*a, *b)
    assert np.allclose(out, c[0]) and np.allclose(lse, c[1])
    nan, none = np.full_like(a[0], np.nan), np.full_like(a[1], -np.inf)
    out, lse, _, _ = P.join(nan, none, *b)
    assert np.allclose(out, b[0]) and np.allclose(lse, b[1])
    out, lse, _, _ = P.join(nan, none, np.zeros_like(nan), none)
    assert not out.any() and np.isneginf(lse).all()


# --------------------------------------------------------------- host refusals

def _prompt(**kw):
    a = dict(num_seqs=2, heads=8, kv_heads=4, dim=128, shared_dim=64, dtype=0, flags=1, reserved=0, total_q=100, total_k=900,
             max_q=90, max_k=800, cu_q=0x10000, cu_k=0x20000, q_token_stride=8 * 192, q_head_stride=192, k_token_stride=1024,
             k_head_stride=256, v_token_stride=1024, v_head_stride=256, shared_stride=576)
    a.update(kw)
    return dsa.dsa_prompt(*a.values())


def test_prompt_refusals(lib):
    def call(p=None, q=0x30000, k=0x40000, ks=0x50000, v=0x60000, scale=0.1, po=None, pl=None, out=0x70000, lse=0x80000,
             ws=(0x100000, 1 << 40)):
        return lib.dsa_prompt_attn(ctypes.byref(p or _prompt()), q, k, ks, v, scale, po, pl, out, lse, *ws, None)
    bad = [dict(num_seqs=0), dict(cu_q=None), dict(cu_k=0x20002), dict(heads=0), dict(kv_heads=3), dict(flags=4), dict(dtype=2),
           dict(reserved=1), dict(total_q=-1), dict(total_k=1 << 31), dict(max_q=-1), dict(max_k=1 << 31),
           dict(q_token_stride=184), dict(q_head_stride=193), dict(k_token_stride=120), dict(k_head_stride=0),
           dict(v_token_stride=-1024), dict(v_head_stride=1 << 40), dict(shared_stride=56)]
    for b in bad:
        assert call(_prompt(**b)) == -1, b
        assert dsa.dsa_prompt_workspace_size(_prompt(**b)) == 0
    for b in (dict(dim=96), dict(shared_dim=32), dict(heads=129, kv_heads=1), dict(heads=256, kv_heads=4, total_q=1 << 30)):
        assert call(_prompt(**b)) == -2 and dsa.dsa_prompt_workspace_size(_prompt(**b)) == 0
    for b in (dict(q=None), dict(k=None), dict(ks=None), dict(v=None), dict(out=None), dict(q=0x30008), dict(k=0x40002),
              dict(ks=0x50004), dict(v=0x60001), dict(out=0x70008), dict(lse=0x80002), dict(scale=0.0), dict(scale=-1.0),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(po=0x90000), dict(pl=0x90000),
              dict(po=0x90008, pl=0xA0000), dict(po=0x90000, pl=0xA0002)):
        assert call(**b) == -1, b
    assert call(_prompt(shared_dim=0, q_token_stride=1024, q_head_stride=128)) == -1      # k_shared without shared dims
    assert lib.dsa_prompt_attn(None, 1, 1, 1, 1, 1.0, None, None, 1, None, 0, 0, None) == -1
    need = dsa.dsa_prompt_workspace_size(_prompt())
    assert need >= 256 and need % 256 == 0
    for ws in ((None, need), (0x100010, need), (0x100000, need - 1)):
        assert call(ws=ws) == -4
    assert dsa.dsa_prompt_workspace_size(_prompt(flags=3)) == 256                         # never split
    for nothing in (dict(total_q=0), dict(max_q=0)):
        assert call(_prompt(**nothing)) == 0                                              # nothing to do


def test_token_refusals(lib):
    lay = lambda **kw: dsa.dsa_kv_layout(*dict(dict(pool=0x10000, num_rows=100, row_stride_bytes=45312, idx_page_offset=0,
                                                    lat_page_offset=8448, block_size=64, idx_fmt=0, lat_fmt=0, reserved=0), **kw).values())
    bat = lambda **kw: dsa.dsa_batch(*dict(dict(T=2, B=2, q_req=0x20000, q_pos=0x30000, ctx=0x40000, bt=0x50000, stride=16, flags=0,
                                                max_ctx=1000), **kw).values())
    r = ctypes.byref
    write = lambda L=None, b=None, k=0x60000, lat=0x70000, ws=(0x100000, 256): lib.dsa_write_tokens(
        r(L or lay()), r(b or bat()), k, lat, *ws, None)
    for x in (dict(L=lay(pool=None)), dict(b=bat(B=0)), dict(b=bat(q_req=None)), dict(b=bat(max_ctx=1025)), dict(k=0x60008),
              dict(lat=0x70002)):
        assert write(**x) == -1
    assert write(L=lay(block_size=48)) == -2
    for ws in ((None, 256), (0x100000, 255), (0x100020, 256)):
        assert write(ws=ws) == -4
    assert write(k=None, lat=None) == 0 and write(b=bat(T=0)) == 0
    spans = lambda cu=0x80000, start=0x90000, rows=10: dsa.dsa_spans(cu, start, rows)
    read = lambda L=None, b=None, s=None, k=0x60000, lat=0x70000, ws=(0x100000, 256): lib.dsa_read_tokens(
        r(L or lay()), r(b or bat()), r(s or spans()), k, lat, *ws, None)
    for x in (dict(L=lay(pool=None)), dict(b=bat(B=0)), dict(b=bat(ctx=None)), dict(b=bat(max_ctx=1025)), dict(s=spans(cu=None)),
              dict(s=spans(cu=0x80002)), dict(s=spans(start=0x90002)), dict(s=spans(rows=-1)), dict(s=spans(rows=1 << 31)),
              dict(k=0x60008), dict(lat=0x70002)):
        assert read(**x) == -1
    for ws in ((None, 256), (0x100000, 255), (0x100020, 256)):
        assert read(ws=ws) == -4
    assert read(k=None, lat=None) == 0 and read(s=spans(rows=0)) == 0
    assert lib.dsa_read_tokens(r(lay()), r(bat()), None, 0x60000, None, 0x100000, 256, None) == -1


# ------------------------------------------------------------------ the binding

@pytest.fixture()
def fake(monkeypatch):
    x = Library()
    monkeypatch.setattr(dsa, "library", lambda: x)
    monkeypatch.setattr(dsa, "_handle", lambda stream: 77)
    return x


def dev(dtype, *shape):
    return OnDevice(torch.zeros(shape, dtype=dtype))


def test_prompt_binding(fake):
    BF, F32, I = torch.bfloat16, torch.float32, torch.int32
    q, k, v, ks = dev(BF, 5, 4, 192), dev(BF, 9, 2, 128), dev(BF, 9, 2, 128), dev(BF, 9, 64)
    cu = (dev(I, 3), dev(I, 3))
    p = dsa.make_prompt(*cu, q, k, v, ks, flags=1)
    assert [getattr(p, n) for n, _ in p._fields_[:12]] == [2, 4, 2, 128, 64, 0, 1, 0, 5, 9, 5, 9]
    assert (p.q_token_stride, p.q_head_stride, p.k_token_stride, p.v_head_stride, p.shared_stride) == (768, 192, 256, 128, 64)
    for bad in (dict(q=dev(F32, 5, 4, 192)), dict(q=dev(BF, 5, 4, 128)), dict(q=q.t), dict(k=dev(torch.float16, 9, 2, 128)),
                dict(v=dev(BF, 8, 2, 128)), dict(ks=dev(BF, 8, 64)), dict(ks=dev(BF, 9, 1, 64)), dict(ks=None),
                dict(k=OnDevice(torch.zeros(9, 128, 2, dtype=BF).transpose(1, 2)))):
        a = dict(dict(q=q, k=k, v=v, ks=ks), **bad)
        with pytest.raises(ValueError):
            dsa.make_prompt(*cu, a["q"], a["k"], a["v"], a["ks"])
    for c in ((dev(I, 3), dev(I, 4)), (dev(torch.int64, 3), cu[1]), (cu[0].t, cu[1])):
        with pytest.raises(ValueError):
            dsa.make_prompt(*c, q, k, v, ks)
    ws, out, lse = dev(torch.uint8, 256), dev(BF, 5, 4, 128), dev(F32, 5, 4)
    dsa.dsa_prompt_attn(p, q, k, v, 0.1, out, lse, k_shared=ks, ws=ws)
    dsa.dsa_prompt_attn(p, q, k, v, 0.1, out, None, k_shared=ks, prev_out=out, prev_lse=lse, ws=ws)
    assert len(fake.calls) == 2 and fake.calls[0][1][1] == q.data_ptr() and fake.calls[0][1][-1] == 77
    wide = OnDevice(torch.zeros(9, 2, 256, dtype=BF)[..., :128])
    for bad in (dict(q=dev(BF, 6, 4, 192)), dict(k=wide), dict(v=wide), dict(v=v.t), dict(ks=OnDevice(torch.zeros(9, 576, dtype=BF)[:, 512:])),
                dict(ks=None), dict(out=dev(BF, 5, 4, 127)), dict(out=dev(F32, 5, 4, 128)), dict(lse=dev(F32, 5, 3)), dict(lse=lse.t),
                dict(po=dev(F32, 5, 4, 128)), dict(pl=dev(F32, 4, 4)), dict(ws=ws.t)):
        a = dict(dict(q=q, k=k, v=v, ks=ks, out=out, lse=lse, po=None, pl=None, ws=ws), **bad)
        refused(fake, dsa.dsa_prompt_attn, p, a["q"], a["k"], a["v"], 0.1, a["out"], a["lse"], k_shared=a["ks"],
                prev_out=a["po"], prev_lse=a["pl"], ws=a["ws"])
    one = dsa.make_prompt(*cu, dev(BF, 1, 1, 64), dev(BF, 0, 1, 64), dev(BF, 0, 1, 64))   # dimensions of one element, no keys
    assert one.total_k == 0 and one.q_token_stride >= 64 and one.k_head_stride >= 64


def test_token_binding(fake):
    BF, I = torch.bfloat16, torch.int32
    lay, bat = dsa.make_layout(None, 100, 45312, 0, 8448), dsa.dsa_batch(3, 2, 1, 2, 3, 4, 16, 0, 1000)
    ws = dev(torch.uint8, 256)
    dsa.dsa_write_tokens(lay, bat, dev(BF, 3, 128), dev(BF, 3, 576), ws=ws)
    dsa.dsa_write_tokens(lay, bat, latent=dev(BF, 4, 576), ws=ws)
    for a in ((dev(BF, 2, 128), None), (dev(torch.float32, 3, 128), None), (None, dev(BF, 2, 576)), (None, dev(BF, 3, 576).t)):
        refused(fake, dsa.dsa_write_tokens, lay, bat, *a, ws=ws)
    spans = dsa.make_spans(dev(I, 3), dev(I, 2), 7)
    dsa.dsa_read_tokens(lay, bat, spans, dev(BF, 7, 128), dev(BF, 7, 576), ws=ws)
    dsa.dsa_read_tokens(lay, bat, dsa.make_spans(dev(I, 4), None, 7), None, dev(BF, 7, 576), ws=ws)
    assert [c[0] for c in fake.calls] == ["dsa_write_tokens"] * 2 + ["dsa_read_tokens"] * 2
    for a in ((dev(BF, 6, 128), None), (None, dev(BF, 6, 576)), (None, dev(torch.float16, 7, 576)), (None, dev(BF, 7, 576).t)):
        refused(fake, dsa.dsa_read_tokens, lay, bat, spans, *a, ws=ws)
    for s in (dsa.make_spans(dev(I, 2), dev(I, 2), 7), dsa.make_spans(dev(I, 3), dev(I, 1), 7)):
        refused(fake, dsa.dsa_read_tokens, lay, bat, s, None, dev(BF, 7, 576), ws=ws)
    with pytest.raises(ValueError):
        dsa.make_spans(torch.zeros(3, dtype=I), None, 7)


def test_structure_layout(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    names = {"dsa_prompt": dsa.dsa_prompt, "dsa_spans": dsa.dsa_spans}
    src = "#include <stddef.h>\n#include <stdio.h>\n#include \"dsa.h\"\nint main(void){\n"
    want = []
    for n, cls in names.items():
        src += f'printf("%zu\\n", sizeof({n}));\n'
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            src += f'printf("%zu\\n", offsetof({n}, {f}));\n'
            want.append(getattr(cls, f).offset)
    c = tmp_path / "s.c"
    c.write_text(src + "return 0;}\n")
    subprocess.run([cc, "-std=c99", "-I", INC, str(c), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == want
