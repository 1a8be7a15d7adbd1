"""New tokens' records into the pages and cached positions' values out of them, byte by byte against the
oracle: the same fp32 quotients and roundings on both sides, so no tolerance."""
import numpy as np
import pytest
import torch

from dsa_sparse_attention_gb300 import workloads as W
from oracle import front as F
from oracle import prompt as P
from oracle.formats import decode_bf16
from tests.parity import oracle_layout

pytestmark = pytest.mark.gpu
FORMATS = [(0, 0), (1, 1), (0, 1), (1, 0)]   # (index keys, latents)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_sparse_attention_gb300.build import build
    build()


def _bits(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.float32))).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _dev(u16):
    return torch.from_numpy(u16.view(np.int16)).cuda().view(torch.bfloat16)


def _work(lens, new, fmt, bs, seed):
    from dsa_sparse_attention_gb300.harness import DeviceWorkload
    wl = W.make_workload(lens, new, seed=seed, permute=True, idx_fmt=fmt[0], lat_fmt=fmt[1], block_size=bs)
    return wl, DeviceWorkload(wl)


def _values(rng, T):
    """N(0, 1) rows, and in the first ones what is special: zeros, tiny and huge values, one value alone."""
    k, lat = rng.standard_normal((T, 128)), rng.standard_normal((T, 576))
    scales = 2.0 ** rng.integers(-20, 20, (T, 1))
    k *= scales
    lat *= np.clip(scales, 2.0 ** -12, 64.0)
    for i, v in enumerate([0.0, 2.0 ** -133, 2.0 ** -126, 1e-30, 2.0 ** 127, 448.0, 1e30]):
        if i < T:
            k[i], lat[i] = 0.0, 0.0
            k[i, 5], lat[i, 7] = v, v
            if i % 2:
                k[i, 64:] = -v
                lat[i, 300:] = -v / 3
    if T > 9:
        k[8, ::2] = 0.0                                    # alternating zeros of both signs
        k[8, 1::4] = -0.0
        lat[9] = np.repeat(np.arange(36) / 3.0, 16)        # constant groups
    return _bits(k), _bits(lat)


def _write(wl, pool, k, lat, tokens):
    """The oracle's writes into a copy of the pool."""
    bs = wl.block_size
    for t in tokens:
        row, slot = wl.block_table[wl.q_req[t], wl.q_pos[t] // bs], int(wl.q_pos[t]) % bs
        if k is not None:
            if wl.idx_fmt == 0:
                F.write_index_key(pool, wl.row_stride, wl.idx_page_offset, bs, row, slot, *F.index_key_fp8(k[t]))
            else:
                F.write_index_key_mxfp4(pool, wl.row_stride, wl.idx_page_offset, bs, row, slot, *F.index_key_mxfp4(k[t]))
        if lat is not None:
            F.write_latent(pool, wl.row_stride, wl.lat_page_offset, row, slot, F.latent_record(lat[t], wl.lat_fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,new,bs", [([1], [1], 16), ([100, 33, 64], [35, 33, 1], 64), ([300, 7], [290, 7], 256),
                                         ([17, 49], [17, 3], 32)])
def test_written_bytes(lens, new, bs, fmt):
    import dsa_sparse_attention_gb300 as dsa
    wl, dw = _work(lens, new, fmt, bs, 3)
    k, lat = _values(np.random.default_rng(sum(lens)), sum(new))
    T = sum(new)
    for keys, lats in ((k, lat), (k, None), (None, lat), (None, None)):
        dw.pool.copy_(torch.from_numpy(wl.pool))
        want = wl.pool.copy()
        _write(wl, want, keys, lats, range(T))
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        dsa.dsa_write_tokens(dw.layout, dw.batch, None if keys is None else _dev(keys), None if lats is None else _dev(lats), ws=ws)
        assert dsa.dsa_check(ws) == 0
        got = dw.pool.cpu().numpy()
        assert np.array_equal(got, want), f"{np.count_nonzero(got != want)} bytes differ"


@pytest.mark.parametrize("fmt", FORMATS[:2])
def test_padding_and_places_out_of_range(fmt):
    import dsa_sparse_attention_gb300 as dsa
    wl, dw = _work([200, 90, 64], [20, 20, 20], fmt, 64, 5)
    k, lat = _values(np.random.default_rng(1), 60)
    dw.q_req[3:9] = -1                                     # padding: nothing is recorded
    want = wl.pool.copy()
    _write(wl, want, k, lat, [t for t in range(60) if not 3 <= t < 9])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dsa.dsa_write_tokens(dw.layout, dw.batch, _dev(k), _dev(lat), ws=ws)
    assert dsa.dsa_check(ws) == 0 and np.array_equal(dw.pool.cpu().numpy(), want)
    dw.pool.copy_(torch.from_numpy(wl.pool))
    dw.q_req[10] = 3                                       # no such request
    dw.q_pos[11], dw.q_pos[12] = -1, 200                   # no such position
    dw.bt[1] = wl.num_rows                                 # no such row
    dw.bt[2] = -1
    want = wl.pool.copy()
    _write(wl, want, k, lat, [0, 1, 2, 9] + list(range(13, 20)))
    dsa.dsa_write_tokens(dw.layout, dw.batch, _dev(k), _dev(lat), ws=ws)
    assert dsa.dsa_check(ws) == -6 and np.array_equal(dw.pool.cpu().numpy(), want)


def _same(got, want):
    got = got.double().cpu().numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{len(bad)} values differ, first {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


def _spans(dsa, start, lens, gap):
    cu = np.concatenate([[0], np.cumsum(lens)]) + gap
    i32 = lambda a: torch.tensor([int(x) for x in a], dtype=torch.int32, device="cuda")
    return cu, dsa.make_spans(i32(cu), None if start is None else i32(start), int(cu[-1]) + gap)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,start,take,bs", [([1], None, [1], 16), ([200, 64, 90], [3, 0, 89], [197, 64, 1], 64),
                                                ([300, 5, 500], [0, 2, 100], [0, 3, 0], 256), ([70, 400], None, [64, 400], 32)])
def test_read_values(lens, start, take, bs, fmt):
    import dsa_sparse_attention_gb300 as dsa
    wl, dw = _work(lens, 1, fmt, bs, 7)
    cu, spans = _spans(dsa, start, take, 2)
    n = spans.rows
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lay = oracle_layout(wl)
    for with_k, with_lat in ((True, True), (True, False), (False, True)):
        k = torch.full((n, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lat = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda")
        dsa.dsa_read_tokens(dw.layout, dw.batch, spans, k if with_k else None, lat if with_lat else None, ws=ws)
        assert dsa.dsa_check(ws) == 0
        want_k, want_l = np.full((n, 128), 7.0), np.full((n, 576), 7.0)
        for r, m in enumerate(take):
            kk, ll = P.token_values(lay, wl.block_table[r], (start[r] if start else 0) + np.arange(m))
            if with_k:      # the product of code and fp32 scale, rounded to fp32 and then to bf16
                want_k[cu[r]:cu[r + 1]] = decode_bf16(_bits(kk.astype(np.float32)))
            if with_lat:
                want_l[cu[r]:cu[r + 1]] = decode_bf16(_bits(ll))
                assert np.array_equal(decode_bf16(_bits(ll)).reshape(ll.shape), ll)   # exact in bf16
        _same(k, want_k)
        _same(lat, want_l)


@pytest.mark.parametrize("fmt", FORMATS[:2])
def test_outputs_that_begin_off_32_bytes(fmt):
    import dsa_sparse_attention_gb300 as dsa
    wl, dw = _work([100], 1, fmt, 64, 7)
    cu, spans = _spans(dsa, [5], [90], 0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    k = torch.full((90 * 128 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    lat = torch.full((90 * 576 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_read_tokens(dw.layout, dw.batch, spans, k[8:-8].view(90, 128), lat[8:-8].view(90, 576), ws=ws)
    assert dsa.dsa_check(ws) == 0
    kk, ll = P.token_values(oracle_layout(wl), wl.block_table[0], 5 + np.arange(90))
    _same(k[8:-8].view(90, 128), decode_bf16(_bits(kk.astype(np.float32))))
    _same(lat[8:-8].view(90, 576), ll)
    assert all(torch.all(x[e] == 7.0) for x in (k, lat) for e in (slice(0, 8), slice(-8, None)))


@pytest.mark.parametrize("rows", [4900, 9000, 20_000, 40_000])
def test_sizes_of_a_cta(rows):
    """As many rows as take 4 to 32 of them a CTA to read, and 8 to 64 to write."""
    import dsa_sparse_attention_gb300 as dsa
    wl, dw = _work([rows], [rows], (0, 1), 64, 7)
    g = torch.Generator(device="cuda").manual_seed(1)
    lat = torch.randn((rows, 576), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((rows, 128), generator=g, device="cuda").to(torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dsa.dsa_write_tokens(dw.layout, dw.batch, k, lat, ws=ws)
    ko, lo = torch.zeros_like(k), torch.zeros_like(lat)
    cu, spans = _spans(dsa, None, [rows], 0)
    dsa.dsa_read_tokens(dw.layout, dw.batch, spans, ko, lo, ws=ws)
    assert dsa.dsa_check(ws) == 0
    at = sorted({0, 1, rows - 1, rows // 2} | {int(x) for x in np.random.default_rng(rows).integers(0, rows, 300)})
    bits = lambda x, t: x[t].view(torch.int16).cpu().numpy().view(np.uint16)
    pool = dw.pool.cpu().numpy()
    wl.pool[:] = pool
    lay = oracle_layout(wl)
    for t in at:
        row, slot = wl.block_table[0, t // 64], t % 64
        base = int(row) * wl.row_stride
        codes, scale = F.index_key_fp8(bits(k, t))
        p = base + wl.idx_page_offset
        assert np.array_equal(pool[p + slot * 128:p + slot * 128 + 128], codes)
        p = base + wl.lat_page_offset + slot * 352
        assert np.array_equal(pool[p:p + 352], F.latent_record(bits(lat, t), 1))
    kk, ll = P.token_values(lay, wl.block_table[0], np.asarray(at))
    _same(ko[at], decode_bf16(_bits(kk.astype(np.float32))))
    _same(lo[at], ll)


def test_many_requests():
    import dsa_sparse_attention_gb300 as dsa
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(1, 20, 700)]
    wl, dw = _work(lens, 1, (0, 0), 16, 9)
    take = [int(rng.integers(0, L + 1)) for L in lens]
    start = [int(rng.integers(0, L - m + 1)) for L, m in zip(lens, take)]
    cu, spans = _spans(dsa, start, take, 1)
    lat = torch.full((spans.rows, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dsa.dsa_read_tokens(dw.layout, dw.batch, spans, None, lat, ws=ws)
    assert dsa.dsa_check(ws) == 0
    want = np.full((spans.rows, 576), 7.0)
    for r, m in enumerate(take):
        want[cu[r]:cu[r + 1]] = P.token_values(oracle_layout(wl), wl.block_table[r], start[r] + np.arange(m))[1]
    _same(lat, want)


def test_rows_out_of_range_are_recorded_and_left():
    import dsa_sparse_attention_gb300 as dsa
    wl, dw = _work([100, 100, 100, 100], 1, (0, 0), 64, 9)
    dw.bt[2, 1] = wl.num_rows + 5
    cu, spans = _spans(dsa, [0, 95, 60, -2], [10, 10, 10, 10], 0)   # past the end, a bad row, before the start
    lat = torch.full((40, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dsa.dsa_read_tokens(dw.layout, dw.batch, spans, None, lat, ws=ws)
    assert dsa.dsa_check(ws) == -6
    want = np.full((40, 576), 7.0)
    ok = {0: (0, 10, 0), 1: (10, 15, 95), 2: (20, 24, 60), 3: (32, 40, 0)}
    for r, (a, b, s) in ok.items():
        want[a:b] = P.token_values(oracle_layout(wl), wl.block_table[r], s + np.arange(b - a))[1]
    _same(lat, want)
    # a list that does not ascend: no row of the array is read twice or out of range
    spans = dsa.make_spans(torch.tensor([0, 30, 5, 50, 20], dtype=torch.int32, device="cuda"), None, 40)
    dsa.dsa_read_tokens(dw.layout, dw.batch, spans, None, lat, ws=ws)
    dsa.dsa_check(ws)


def test_written_then_read_and_scored():
    """The layer step finds what dsa_write_tokens wrote where the front would have written it."""
    import dsa_sparse_attention_gb300 as dsa
    wl, dw = _work([3000, 700], 2, (0, 0), 64, 5)
    rng = np.random.default_rng(1)
    k, lat = _bits(rng.standard_normal((4, 128))), _bits(rng.standard_normal((4, 576)))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dsa.dsa_write_tokens(dw.layout, dw.batch, _dev(k), _dev(lat), ws=ws)
    _write(wl, wl.pool, k, lat, range(4))
    idx, out, lse = dw.layer_step()
    torch.cuda.synchronize()
    assert dsa.dsa_check(ws) == 0 and dsa.dsa_check(dw.ws) == 0
    from tests.parity import OracleCache, check_mla, check_topk
    oc = OracleCache(wl)
    check_topk(oc, idx.cpu().numpy(), [0, 1, 2, 3], dw.topk)
    check_mla(oc, idx.cpu().numpy(), out.float().cpu().numpy(), lse.cpu().numpy(), [0, 1, 2, 3])
