"""Trees of drafted tokens on the GPU: the dense attention, the top-k, the commit, and a
run of them together, against the float64 definitions (oracle/tree.py)."""
import numpy as np
import pytest
import torch

from dsa_sparse_attention_gb300 import workloads as W
from oracle import dsa_oracle as O
from oracle import tree as OT
from tests.tree_cases import DeviceTree, TreeCase, check_mla, make_case, random_parents

pytestmark = pytest.mark.gpu

FMTS = [W.LAT_FP8, W.LAT_NVFP4]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_sparse_attention_gb300.build import build
    build()


def _check(ws):
    import dsa_sparse_attention_gb300 as dsa
    return dsa.dsa_check(ws)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bs", [16, 64, 256])
def test_mla_ragged(fmt, bs):
    # contexts around tile and page borders, one drafted token to forty, an empty context
    case = make_case([0, 1, 127, 128, 129, 700, 2047], [3, 1, 2, 5, 40, 7, 1], seed=3 + bs, lat_fmt=fmt,
                     block_size=bs)
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    print("worst use of the tolerance", check_mla(case, out, lse))


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_one_token_many_ctas(fmt):
    # one drafted token over more tiles than there are CTAs, then over fewer
    for base in (25000, 1000):
        case = make_case([base], [1], seed=base, lat_fmt=fmt)
        d = DeviceTree(case)
        out, lse = d.mla()
        torch.cuda.synchronize()
        assert _check(d.ws) == 0
        check_mla(case, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_many_tiles_a_cta(fmt):
    # more work than CTAs: every CTA walks tiles of several tokens (700 tokens of 5 to 7 tiles),
    # and a long token next to short ones
    case = make_case([800, 600, 12000], [300, 380, 20], seed=77, lat_fmt=fmt)
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    check_mla(case, out, lse, list(range(0, 700, 23)) + [299, 300, 679, 680, 699])


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_same_bits_every_time(fmt):
    # many CTAs at work on many segments, again and again: a copy that lands before the place it goes to
    # has been read shows as a call whose bits differ
    case = make_case([800, 600, 12000], [300, 380, 20], seed=77, lat_fmt=fmt)
    d = DeviceTree(case)
    out, lse = (x.clone() for x in d.mla())
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        d.out.fill_(7.0)
        d.mla()
        differ += (d.out != out).sum() + (d.lse != lse).sum()
    assert int(differ) == 0 and _check(d.ws) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_masks_and_padding(fmt):
    # rows that see nothing, rows that see only others, bits behind the token, a padding token,
    # a committed length equal to the context (causal whatever the mask)
    case = make_case([0, 300, 64, 90], [4, 6, 3, 2], seed=9, lat_fmt=fmt, words=2)
    m = case.mask
    m[0] = 0                                   # nothing at all: an empty context and no bit
    m[1] = [1, 0]                              # only slot 0
    m[5] = [0, 0]                              # the committed context only
    m[6] = [0xFFFFFFFF, 0xFFFFFFFF]            # bits behind its own slot do not count
    case.base[2] = case.wl.ctx_lens[2]
    d = DeviceTree(case)
    pad = 8
    d.q_req[pad] = -1
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    assert bool((out[pad] == 7.0).all()) and bool((lse[pad] == 7.0).all())
    check_mla(case, out, lse, [t for t in range(case.wl.num_tokens) if t != pad])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("flags", [0, 1])
def test_mla_nothing_to_do(fmt, flags):
    # a batch of padding alone: nothing is written, and the next call on the workspace is whole
    import dsa_sparse_attention_gb300 as dsa
    flags *= dsa.DSA_BATCH_INVARIANT
    case = make_case([300, 40], [4, 3], seed=11, lat_fmt=fmt)
    d = DeviceTree(case, flags=flags)
    q_req = d.q_req.clone()
    d.q_req.fill_(-1)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0 and (out == 7.0).all() and (lse == 7.0).all()
    d.q_req.copy_(q_req)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    check_mla(case, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_garbage_in_unseen_places(fmt):
    # NaN codes at drafted positions a token does not see and behind the context's end
    case = make_case([200, 70], [9, 30], seed=21, lat_fmt=fmt)
    wl = case.wl
    hidden = 5                                  # nobody but slot 5 itself sees slot 5 of request 0
    for t in range(9):
        case.mask[t] &= ~np.uint32(1 << hidden)
    rows = wl.pool.reshape(wl.num_rows, wl.row_stride)
    rec = 576 if fmt == W.LAT_FP8 else 352
    bs = wl.block_size
    for r, s in [(0, 205)] + [(0, s) for s in range(209, 256)] + [(1, s) for s in range(100, 128)]:
        at = wl.lat_page_offset + (s % bs) * rec
        rows[wl.block_table[r, s // bs], at:at + rec] = 0x7F
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    check_mla(case, out, lse)


def _put_latents(wl, r, pos, values):
    """Latents (fp32 [n, 576]) written at positions `pos` of request r, in the pool's format."""
    rows = wl.pool.reshape(wl.num_rows, wl.row_stride)
    rec = W.to_e4m3(values) if wl.lat_fmt == W.LAT_FP8 else W.quantize_nvfp4_latent(values)
    for s, v in zip(pos, rec):
        at = wl.lat_page_offset + (s % wl.block_size) * rec.shape[1]
        rows[wl.block_table[r, s // wl.block_size], at:at + rec.shape[1]] = v


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_rising_logits(fmt):
    # logits that grow by hundreds along the context: the running maximum moves in most tiles
    case = make_case([1500], [4], seed=33, lat_fmt=fmt)
    wl = case.wl
    q = O.decode_bf16(wl.q[0]).reshape(96, 576)
    dirs = np.sign(q[:1]).astype(np.float32)     # aligned with head 0 of token 0
    pos = np.arange(0, 1500, 50)
    _put_latents(wl, 0, pos, dirs * np.linspace(0.5, 24, pos.size, dtype=np.float32)[:, None])
    wl.q[1:] = wl.q[:1]
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    check_mla(case, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sink", [0, 5999])
def test_mla_sink_and_tail(fmt, sink):
    # one position carries about half of the weight, thousands of others, 2^-12 of it each,
    # the rest: small weights must not be lost beside a large one
    case = make_case([6000], [2], seed=40 + sink, lat_fmt=fmt)
    wl = case.wl
    q = O.decode_bf16(wl.q[0]).reshape(96, 576)
    wl.q[1:] = wl.q[:1]
    u = np.zeros((1, 576), np.float32)
    u[0] = np.sign(q[0])
    gain = 12.5 * np.log(2.0) * 24.0 / np.abs(q[0]).sum()
    g = np.random.default_rng(1)
    vals = (0.1 * g.standard_normal((6002, 576)) + 0.25).astype(np.float32)
    _put_latents(wl, 0, np.arange(6002), vals)
    _put_latents(wl, 0, [sink], vals[sink:sink + 1] + np.float32(gain) * u)
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    check_mla(case, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_strided_rows_and_words(fmt):
    # a row stride above the row's pages, mask rows of more words than needed
    bs = 32
    need = bs * (132 + (576 if fmt == W.LAT_FP8 else 352))
    case = make_case([333, 65], [6, 33], seed=50, lat_fmt=fmt, block_size=bs, row_stride=need + 4096, words=5,
                     pool_rows=40, bt_stride=19)
    d = DeviceTree(case, max_ctx=19 * bs)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    check_mla(case, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_invariant_flag(fmt):
    # with DSA_BATCH_INVARIANT a token's bits do not depend on the batch
    import dsa_sparse_attention_gb300 as dsa
    case = make_case([900, 4000, 130], [3, 5, 2], seed=60, lat_fmt=fmt)
    d = DeviceTree(case, flags=dsa.DSA_BATCH_INVARIANT)
    out, lse = d.mla()
    torch.cuda.synchronize()
    check_mla(case, out, lse)
    wl = case.wl
    for t in (0, 5, 9):
        one = TreeCase(W.Workload(**{**wl.__dict__, "q_req": wl.q_req[t:t + 1], "q_pos": wl.q_pos[t:t + 1],
                                     "q": wl.q[t:t + 1]}), case.base, case.mask[t:t + 1], [0])
        e = DeviceTree(one, flags=dsa.DSA_BATCH_INVARIANT)
        o1, l1 = e.mla()
        torch.cuda.synchronize()
        assert torch.equal(o1[0], out[t]) and torch.equal(l1[0], lse[t])


def test_mla_repeat_stream_graph():
    # the same bits from a second call, from another stream, and from a replayed graph whose
    # inputs changed in between
    case = make_case([700, 1300], [5, 8], seed=70)
    d = DeviceTree(case)
    out, lse = (x.clone() for x in d.mla())
    d.mla()
    torch.cuda.synchronize()
    assert torch.equal(out, d.out) and torch.equal(lse, d.lse)
    side = torch.cuda.Stream()
    d.out.fill_(7.0)
    torch.cuda.synchronize()
    d.mla(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, d.out) and torch.equal(lse, d.lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.mla(stream=torch.cuda.current_stream())
    d.q_pos[:5] -= 0
    d.base[1] = 900                              # fewer committed, the rest through the mask
    d.ctx[1] = 908
    d.q_pos[5:] = torch.arange(900, 908, dtype=torch.int32, device="cuda")
    g.replay()
    torch.cuda.synchronize()
    case.base[1], case.wl.ctx_lens[1], case.wl.q_pos[5:] = 900, 908, np.arange(900, 908)
    check_mla(case, d.out, d.lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_bad_inputs_are_recorded(fmt):
    # a block id outside the pool, a position outside the context: recorded, nothing read there,
    # the other request's tokens unharmed
    case = make_case([500, 300], [2, 3], seed=80, lat_fmt=fmt)
    for bad in (10 ** 6, -5):
        d = DeviceTree(case)
        d.bt[0, 3] = bad
        out, lse = d.mla()
        torch.cuda.synchronize()
        assert _check(d.ws) == -6
        check_mla(case, out, lse, [2, 3, 4])
    d = DeviceTree(case)
    d.q_pos[0] = 600
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == -6
    check_mla(case, out, lse, [1, 2, 3, 4])


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_more_tokens_than_the_plan_holds_at_once(fmt):
    # 1,500 tokens, padding among them and at both ends: the plan takes them 1,024 at a time
    case = make_case([130, 7, 390], [700, 60, 740], seed=81, lat_fmt=fmt, block_size=16)
    d = DeviceTree(case)
    pad = [0, 1, 1023, 1024, 1025, 1200, 1498, 1499]
    for t in pad:
        d.q_req[t] = -1
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    assert (out[pad] == 7.0).all() and (lse[pad] == 7.0).all()
    check_mla(case, out, lse, [t for t in [2, 500, 699, 700, 759, 760, 1022, 1026, 1199, 1201, 1497]])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [0.0, -0.03])
def test_mla_scales(fmt, scale):
    # a scale of zero gives the mean of the values; a negative one turns the order around
    case = make_case([40, 500], [3, 2], seed=82, lat_fmt=fmt)
    case.wl.sm_scale = scale
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    check_mla(case, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_far_apart_logits(fmt):
    # logits hundreds apart: a few positions take it all, and the others' weights are zeros, not NaN
    case = make_case([300, 900], [4, 3], seed=83, lat_fmt=fmt)
    case.wl.sm_scale *= 64.0
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    check_mla(case, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_calls_behind_a_memset_in_a_graph(fmt):
    # the first kernel of each call may be scheduled early: what a memset or a copy in front of it in the
    # same graph writes has to be seen all the same
    import dsa_sparse_attention_gb300 as dsa
    case = make_case([300, 900], [4, 3], seed=84, lat_fmt=fmt)
    d = DeviceTree(case)
    T, k, ld = 7, 64, 904
    q, base, q_req = d.q.clone(), d.base.clone(), d.q_req.clone()
    scores = torch.from_numpy(np.random.default_rng(3).standard_normal((T, ld)).astype(np.float32)).cuda()
    sc = scores.clone()
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    ws = dsa.alloc_workspace(d.layout, d.batch, k)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        d.q.zero_()
        d.q_req.zero_()
        d.q_req.copy_(q_req)
        d.q.copy_(q)
        d.mla(stream=torch.cuda.current_stream())
        d.q.zero_()                              # only after the attention has read it
        sc.zero_()
        sc.copy_(scores)
        dsa.dsa_tree_topk(d.layout, d.batch, d.tree, sc, ld, k, idx, ws=ws)
        sc.zero_()
    for _ in range(5):
        d.q.fill_(1.0)
        idx.fill_(-7)
        g.replay()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0 and _check(ws) == 0
    check_mla(case, d.out, d.lse)
    _check_topk(case, scores.cpu().numpy(), k, idx.cpu().numpy())


def test_mla_two_streams_at_once():
    # two batches on two streams, each with its workspace, many calls in flight: each gives the bits it
    # gives alone
    cases = [make_case([1500, 40], [6, 9], seed=85), make_case([700, 90, 5], [8, 2, 4], seed=86, lat_fmt=W.LAT_NVFP4)]
    devs = [DeviceTree(c) for c in cases]
    alone = []
    for d in devs:
        d.mla()
        torch.cuda.synchronize()
        alone.append((d.out.clone(), d.lse.clone()))
        d.out.fill_(7.0)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for d, s in zip(devs, streams):
            d.mla(stream=s)
    torch.cuda.synchronize()
    for d, (out, lse) in zip(devs, alone):
        assert _check(d.ws) == 0
        assert torch.equal(d.out, out) and torch.equal(d.lse, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_mla_and_commit_past_32_bits(fmt):
    # the same rows of a pool, moved past 6 GB: the same bits, and the commit moves the same records
    import dsa_sparse_attention_gb300 as dsa
    case = make_case([300, 900], [4, 3], seed=87, lat_fmt=fmt)
    wl = case.wl
    near = DeviceTree(case)
    out, lse = (x.clone() for x in near.mla())
    acc = torch.tensor([[1, 3, -1], [0, 2, -1]], dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    dsa.dsa_tree_commit(near.layout, near.batch, near.base, acc, new, ws=near.ws)
    far = DeviceTree(case)
    shift = 6 * 2 ** 30 // wl.row_stride + 1
    far.pool = torch.empty((shift + wl.num_rows) * wl.row_stride, dtype=torch.uint8, device="cuda")
    far.pool[shift * wl.row_stride:] = torch.from_numpy(wl.pool.reshape(-1)).cuda()
    far.bt = torch.where(far.bt >= 0, far.bt + shift, far.bt)
    far.layout = dsa.make_layout(far.pool, shift + wl.num_rows, wl.row_stride, wl.idx_page_offset, wl.lat_page_offset,
                                 wl.block_size, wl.idx_fmt, wl.lat_fmt)
    far.batch = dsa.make_batch(far.q_req, far.q_pos, far.ctx, far.bt, wl.max_ctx_len)
    far.mla()
    dsa.dsa_tree_commit(far.layout, far.batch, far.base, acc, new, ws=far.ws)
    torch.cuda.synchronize()
    assert _check(near.ws) == 0 and _check(far.ws) == 0
    assert torch.equal(far.out, out) and torch.equal(far.lse, lse)
    assert torch.equal(far.pool[shift * wl.row_stride:], near.pool.reshape(-1))


# ----------------------------------------------------------------------- top-k

def _topk(case, scores, k, phys=False, max_ctx=None, pad=()):
    import dsa_sparse_attention_gb300 as dsa
    d = DeviceTree(case, max_ctx=max_ctx)
    for t in pad:
        d.q_req[t] = -1
    ws = dsa.alloc_workspace(d.layout, d.batch, k)
    sc = torch.from_numpy(scores).cuda()
    idx = torch.full((scores.shape[0], k), -7, dtype=torch.int32, device="cuda")
    ph = torch.full_like(idx, -7) if phys else None
    dsa.dsa_tree_topk(d.layout, d.batch, d.tree, sc, scores.shape[1], k, idx, ph, ws=ws)
    torch.cuda.synchronize()
    assert dsa.dsa_check(ws) == 0
    return idx.cpu().numpy(), ph.cpu().numpy() if phys else None


def _topk_case(bases, drafts, seed, words=None, bs=64):
    """A case without a pool's content (the top-k reads scores and the block table only)."""
    rng = np.random.default_rng(seed)
    ctx = [b + n for b, n in zip(bases, drafts)]
    nblk = [(c + bs - 1) // bs for c in ctx]
    bt = np.full((len(ctx), max(nblk)), -1, np.int32)
    perm = rng.permutation(sum(nblk)).astype(np.int32)
    at = 0
    for r, n in enumerate(nblk):
        bt[r, :n] = perm[at:at + n]
        at += n
    T = sum(drafts)
    words = words or max(1, (max(drafts) + 31) // 32)
    mask = np.concatenate([OT.ancestor_masks(random_parents(rng, n), words) for n in drafts if n])
    wl = W.Workload("scores", np.zeros(16, np.uint8), max(1, perm.size), bs * 708, 0, bs * 132, bs, 0, 0, bt,
                    np.asarray(ctx, np.int32), np.concatenate([np.full(n, r, np.int32) for r, n in enumerate(drafts)]),
                    np.concatenate([np.arange(b, b + n, dtype=np.int32) for b, n in zip(bases, drafts)]),
                    np.zeros((T, 1), np.uint8), np.zeros((T, 1), np.float32), np.zeros((T, 1), np.uint16))
    ld = (max(ctx) + 3) // 4 * 4
    return TreeCase(wl, np.asarray(bases, np.int32), mask, []), rng.standard_normal((T, ld)).astype(np.float32)


def _check_topk(case, scores, k, idx, phys=None, skip=()):
    bs = case.wl.block_size
    for t in range(scores.shape[0]):
        if t in skip:
            assert np.all(idx[t] == -7)
            continue
        ref = OT.tree_topk(scores[t], case.seen(t), k)
        assert np.array_equal(idx[t], ref), f"token {t}"
        if phys is not None:
            row = case.wl.block_table[int(case.wl.q_req[t])]
            want = [-1 if s < 0 else int(row[s // bs]) * bs + s % bs for s in ref]
            assert np.array_equal(phys[t], want), f"token {t}: slots"


@pytest.mark.parametrize("k", [1, 100, 2048])
def test_topk_small_rows(k):
    case, scores = _topk_case([0, 1, 90, 2040, 2047, 2048, 9000], [3, 5, 40, 20, 1, 70, 9], seed=k)
    idx, ph = _topk(case, scores, k, phys=True)
    _check_topk(case, scores, k, idx, ph)


@pytest.mark.parametrize("bases", [[65500, 30000], [65530, 70000, 131000]])
@pytest.mark.parametrize("bs", [16, 64])
def test_topk_long_rows(bases, bs):
    case, scores = _topk_case(bases, [12] * len(bases), seed=5, bs=bs)
    idx, ph = _topk(case, scores, 2048, phys=True)
    _check_topk(case, scores, 2048, idx, ph)


@pytest.mark.parametrize("base", [4090, 14330, 16380, 40000])
@pytest.mark.parametrize("shape", ["normal", "outlier", "tiny", "huge", "tail"])
def test_topk_around_the_rules(base, shape):
    # rows around the length where the sampled bound sets in, scores whose spread the digits handle badly
    case, scores = _topk_case([base, base + 3], [9, 20], seed=base)
    if shape == "outlier":
        scores[:, 77] = np.float32(3e38)
        scores[:, 99] = np.float32(-3e38)
    elif shape == "tiny":
        scores *= np.float32(1e-42)              # subnormal, few distinct values
    elif shape == "huge":
        with np.errstate(over="ignore"):
            scores *= np.float32(1e38)           # infinities among them
    elif shape == "tail":
        scores = np.exp(3 * np.abs(scores)).astype(np.float32)
    idx, ph = _topk(case, scores, 2048, phys=True)
    _check_topk(case, scores, 2048, idx, ph)


@pytest.mark.parametrize("base", [5000, 70000])
def test_topk_unseen_scores_and_ties(base):
    # NaN, infinities and the best scores at unseen positions; thousands of equal scores
    case, scores = _topk_case([base], [64], seed=6)
    for t in range(64):
        unseen = np.setdiff1d(np.arange(base, base + 64), case.seen(t))
        scores[t, unseen] = np.resize([np.nan, np.inf, -np.inf, 50.0], unseen.size).astype(np.float32)
        scores[t, base + 64:] = np.nan
    scores[10:20, ::2] = np.where(np.isfinite(scores[10:20, ::2]), np.float32(1.5), scores[10:20, ::2])
    scores[20, :base] = 0.0
    scores[21, :base] = -0.0
    scores[22, :base:2] = -0.0
    scores[22, 1:base:2] = 0.0
    idx, _ = _topk(case, scores, 2048)
    _check_topk(case, scores, 2048, idx)


@pytest.mark.parametrize("base", [3000, 20000, 100000])
@pytest.mark.parametrize("shape", ["equal", "two", "falling", "rising", "lowest", "heavy"])
def test_topk_distributions(base, shape):
    # scores that a sampled bound serves badly: all equal, two values, sorted rows, infinities,
    # a few large ones in one place
    case, scores = _topk_case([base], [6], seed=8)
    n = scores.shape[1]
    g = np.random.default_rng(base)
    if shape == "equal":
        scores[:] = -2.5
    elif shape == "two":
        scores[:] = np.where(g.random(scores.shape) < 0.3, np.float32(1), np.float32(-1))
    elif shape == "falling":
        scores[:] = -np.arange(n, dtype=np.float32)
    elif shape == "rising":
        scores[:] = np.arange(n, dtype=np.float32) * np.float32(1e-3)
    elif shape == "lowest":
        scores[:] = np.float32(-3.4028235e38)
        scores[:, 5:base:7] = -np.inf
        scores[:, base // 2] = np.inf
    else:
        scores[:, 100:2300] += 50
    idx, _ = _topk(case, scores, 2048)
    _check_topk(case, scores, 2048, idx)


@pytest.mark.parametrize("max_ctx", [None, 80 * 1024])
def test_topk_empty_padding_and_mask_edges(max_ctx):
    case, scores = _topk_case([0, 2040, 3000], [4, 64, 40], seed=7, words=3)
    case.mask[0] = 0                            # sees nothing
    case.mask[4 + 63] = 0xFFFFFFFF              # every slot up to its own, and bits behind it
    case.mask[4 + 20] = 0                       # the committed context only
    case.base[2] = case.wl.ctx_lens[2]          # causal
    if max_ctx:                                 # the passes for long rows
        bt = np.full((3, max_ctx // 64), -1, np.int32)
        bt[:, :case.wl.block_table.shape[1]] = case.wl.block_table
        case.wl.block_table = bt
        scores = np.pad(scores, ((0, 0), (0, max_ctx - scores.shape[1])))
    idx, _ = _topk(case, scores, 2048, max_ctx=max_ctx, pad=(2, 70))
    _check_topk(case, scores, 2048, idx, skip=(2, 70))


@pytest.mark.parametrize("base", [3000, 70000])
def test_topk_infinities_and_signed_zeros(base):
    # infinities are scores like any other; 0 and -0 are equal, so the lower position wins
    case, scores = _topk_case([base], [4], 88)
    rng = np.random.default_rng(88)
    scores[0] = rng.choice(np.asarray([np.inf, -np.inf, 0.0, -0.0], np.float32), scores.shape[1])
    scores[1] = -np.inf
    scores[2] = np.where(rng.random(scores.shape[1]) < 0.5, np.float32(0.0), np.float32(-0.0))
    scores[3, ::3] = np.inf
    idx, _ = _topk(case, scores, 700)
    _check_topk(case, scores, 700, idx)


# ---------------------------------------------------------------------- commit

def _commit(wl, base, accept, alias=False):
    import dsa_sparse_attention_gb300 as dsa
    cu = lambda a, dt=None: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    pool, bt, ctx = cu(wl.pool), cu(wl.block_table), cu(wl.ctx_lens)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    layout = dsa.make_layout(pool, wl.num_rows, wl.row_stride, wl.idx_page_offset, wl.lat_page_offset, wl.block_size,
                             wl.idx_fmt, wl.lat_fmt)
    batch = dsa.make_batch(none, none, ctx, bt, wl.max_ctx_len)
    ws = dsa.alloc_cache_workspace(layout, len(base))
    new = ctx if alias else torch.full((len(base),), -1, dtype=torch.int32, device="cuda")
    dsa.dsa_tree_commit(layout, batch, cu(np.asarray(base, np.int32)), cu(np.asarray(accept, np.int32)), new, ws=ws)
    torch.cuda.synchronize()
    return pool.cpu().numpy().reshape(wl.num_rows, wl.row_stride), new.cpu().tolist(), dsa.dsa_check(ws)


def _cache_layout(wl):
    return OT.CacheLayout(wl.block_size, wl.idx_page_offset, wl.lat_page_offset, wl.idx_fmt, wl.lat_fmt)


@pytest.mark.parametrize("idx_fmt", [W.IDX_FP8, W.IDX_MXFP4])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bs", [16, 128])
def test_commit(idx_fmt, fmt, bs):
    # nothing, one, all, a path whose sources are overwritten by earlier moves, more than one round
    base = [0, 15, 16, 100, 250]
    drafts = [5, 20, 33, 40, 9]
    wl = W.make_workload([b + n for b, n in zip(base, drafts)], 1, seed=bs, idx_fmt=idx_fmt, lat_fmt=fmt, block_size=bs)
    wl.pool[:] = np.random.default_rng(2).integers(0, 256, wl.pool.size, dtype=np.uint8)
    acc = np.full((5, 33), -1, np.int32)
    acc[0, :5] = range(5)
    acc[1, :3] = [1, 2, 3]
    acc[2, :32] = range(1, 33)
    acc[3, :20] = np.sort(np.random.default_rng(3).permutation(40)[:20])
    acc[4, 1] = 3                                # behind a negative entry: not read
    got, lens, st = _commit(wl, base, acc)
    want, wl_lens = OT.commit(wl.pool.reshape(wl.num_rows, wl.row_stride), _cache_layout(wl), wl.block_table, base,
                              wl.ctx_lens, acc)
    assert st == 0 and lens == wl_lens and np.array_equal(got, want)
    got, lens, st = _commit(wl, base, acc, alias=True)
    assert st == 0 and lens == wl_lens and np.array_equal(got, want)


def test_commit_refuses_a_request():
    # rows that do not ascend, leave the draft, or lie on a missing block: that request is left alone
    base = [40, 40, 40, 40, 40]
    wl = W.make_workload([60] * 5, 1, seed=4)
    wl.pool[:] = np.random.default_rng(5).integers(0, 256, wl.pool.size, dtype=np.uint8)
    acc = np.asarray([[3, 3, -1], [5, 2, -1], [4, 20, -1], [2, 7, 9], [1, 3, 4]], np.int32)
    wl.block_table[3, 0] = wl.num_rows
    got, lens, st = _commit(wl, base, acc)
    bt = wl.block_table.copy()
    bt[3, 0] = 0
    want, want_lens = OT.commit(wl.pool.reshape(wl.num_rows, wl.row_stride), _cache_layout(wl), bt, base,
                                wl.ctx_lens, np.where(np.arange(5)[:, None] == 3, [[3, 3, -1]], acc))
    assert st == -6 and lens == want_lens == [-1, -1, -1, -1, 43] and np.array_equal(got, want)


# ------------------------------------------------------------ a run of them all

def test_draft_score_attend_commit():
    """A tree is written into the cache, scored, selected, attended (sparse, and dense
    where the selection holds everything), its accepted path committed, and the next
    token decoded: the same as decoding on a cache that never held the tree."""
    import dsa_sparse_attention_gb300 as dsa
    base, n = [150, 515], [7, 9]
    case = make_case(base, n, seed=90)
    wl = case.wl
    d = DeviceTree(case)
    T = wl.num_tokens
    rng = np.random.default_rng(91)
    lat = torch.from_numpy(rng.standard_normal((T, 576)).astype(np.float32)).cuda().to(torch.bfloat16)
    dsa.dsa_write_latent(d.layout, d.batch, lat, ws=d.ws)
    ws = dsa.alloc_workspace(d.layout, d.batch, 2048)
    ld = (wl.max_ctx_len + 3) // 4 * 4
    scores = torch.full((T, ld), float("nan"), device="cuda")
    q_idx, w = torch.from_numpy(wl.q_idx).cuda(), torch.from_numpy(wl.w).cuda()
    dsa.dsa_indexer_score(d.layout, d.batch, q_idx, w, scores, ld, ws)
    idx = torch.empty((T, 2048), dtype=torch.int32, device="cuda")
    dsa.dsa_tree_topk(d.layout, d.batch, d.tree, scores, ld, 2048, idx, ws=ws)
    out, lse = torch.empty_like(d.out), torch.empty_like(d.lse)
    dsa.dsa_sparse_mla(d.layout, d.batch, d.q, idx, 2048, wl.sm_scale, out, lse, ws=ws)
    dense, dlse = d.mla()
    torch.cuda.synchronize()
    assert dsa.dsa_check(ws) == 0 and dsa.dsa_check(d.ws) == 0
    wl.pool[:] = d.pool.cpu().numpy()            # the oracle reads the pool as written
    check_mla(case, dense, dlse)
    check_mla(case, out, lse)
    k = 100                                      # a real selection, too
    idx2 = torch.empty((T, k), dtype=torch.int32, device="cuda")
    dsa.dsa_tree_topk(d.layout, d.batch, d.tree, scores, ld, k, idx2, ws=ws)
    sc = scores.cpu().numpy()
    for t in range(T):
        assert np.array_equal(idx2[t].cpu().numpy(), OT.tree_topk(sc[t], case.seen(t), k))
    # the deepest path of each tree is accepted
    acc = np.full((2, 9), -1, np.int32)
    for r in range(2):
        deep = max(range(case.first[r], case.first[r] + n[r]), key=lambda t: case.seen(t).size)
        path = [int(s) - base[r] for s in case.seen(deep) if s >= base[r]]
        acc[r, :len(path)] = path
    before = wl.pool.reshape(wl.num_rows, wl.row_stride).copy()
    new_lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    dsa.dsa_tree_commit(d.layout, d.batch, d.base, torch.from_numpy(acc).cuda(), new_lens, ws=d.ws)
    torch.cuda.synchronize()
    want, lens = OT.commit(before, _cache_layout(wl), wl.block_table, base, wl.ctx_lens, acc)
    assert np.array_equal(d.pool.cpu().numpy().reshape(want.shape), want) and new_lens.cpu().tolist() == lens
    # one more token for each request on the committed cache: its ancestors' latents, in order
    for r in range(2):
        L = lens[r]
        wl.pool[:] = want.reshape(-1)
        one = TreeCase(W.Workload(**{**wl.__dict__, "ctx_lens": np.asarray([L], np.int32),
                                     "block_table": wl.block_table[r:r + 1], "q_req": np.zeros(1, np.int32),
                                     "q_pos": np.asarray([L - 1], np.int32), "q": wl.q[:1]}),
                       np.asarray([L], np.int32), np.zeros((1, 1), np.uint32), [0])
        e = DeviceTree(one)
        o, l = e.mla()
        torch.cuda.synchronize()
        check_mla(one, o, l)
