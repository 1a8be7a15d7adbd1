"""Trees of drafted tokens where tests at ordinary sizes do not look: rows on which a token
sees little, rows of millions of scores, errors that a worst-case bound would hide, and
logits far beyond a softmax's usual range."""
import numpy as np
import pytest
import torch

from dsa_sparse_attention_gb300 import workloads as W
from oracle import dsa_oracle as O
from oracle import tree as OT
from tests.parity import oracle_layout
from tests.test_gpu_tree import _check, _check_topk, _topk, _topk_case
from tests.tree_cases import DeviceTree, check_mla, make_case

FMTS = [W.LAT_FP8, W.LAT_NVFP4]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_sparse_attention_gb300.build import build
    build()


# ------------------------------------------------ errors of a few values, not of all

def rms_use(case, out, t):
    """Largest share that the rms error of any head's 64 dims (a chunk) takes of its bound.

    The roundings of a token's result, independent of each other: the output to bf16, uniform
    within half a step, so at most 2^-8 / sqrt(3) of the value in the mean square; every weight,
    to 9 significant bits or more, so a dim moves by at most (2^-9 / sqrt(3)) sqrt(sum p^2 v^2), and
    with it the fp16 partials (2^-11); the logits, off by at most e of check_mla each.  The bound is
    twice the root of the sum of squares: the error of a chunk's 64 dims scatters by 9 % around its
    mean square, and where one weight carries the result its rounding is at most sqrt(3) times its mean.
    Where check_mla's bound stays at 2^-8 of sum p |v|, this one shrinks with the number of positions,
    as the result does, so wrong values at a few positions show."""
    wl = case.wl
    lat = O.gather_latents(oracle_layout(wl), wl.block_table[int(wl.q_req[t])], case.seen(t))
    ref, lse, _ = OT.dense_mla(wl.q[t], lat, wl.sm_scale)
    q = O.decode_bf16(wl.q[t]).reshape(96, 576)
    p = np.exp(wl.sm_scale * (q @ lat.T) - lse[:, None])
    spread = (p * p) @ (lat[:, :512] ** 2)
    e = 2.0 ** -18 * abs(wl.sm_scale) * (np.abs(q) @ np.abs(lat).T).max(axis=1)
    chunks = lambda x: x.reshape(96, 8, 64).mean(axis=2)
    bound = 2 * np.sqrt(2.0 ** -16 / 3 * chunks(ref ** 2) + (2.0 ** -18 / 3 + e[:, None] ** 2) * chunks(spread))
    err = out[t].astype(np.float64) - ref
    return float((np.sqrt(chunks(err ** 2)) / bound).max())


@pytest.mark.parametrize("fmt", FMTS)
def test_rms_bound_sees_one_wrong_warp(fmt):
    # (no GPU) the exact result, rounded, passes; with 32 positions' values of 64 dims exchanged for
    # others', which the worst-case bound lets pass, it does not
    case = make_case([25000], [1], seed=301, lat_fmt=fmt)
    wl = case.wl
    lat = O.gather_latents(oracle_layout(wl), wl.block_table[0], case.seen(0))
    ref, _, _ = OT.dense_mla(wl.q[0], lat, wl.sm_scale)
    bf16 = lambda x: torch.from_numpy(x).to(torch.bfloat16).float().numpy()[None]
    assert rms_use(case, bf16(ref), 0) < 1.0
    bad = lat.copy()
    bad[1312:1344, 192:256] = lat[2312:2344, 192:256]
    q = O.decode_bf16(wl.q[0]).reshape(96, 576)
    logits = wl.sm_scale * (q @ lat.T)
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    out = (p / p.sum(axis=1, keepdims=True)) @ bad[:, :512]
    assert rms_use(case, bf16(out), 0) > 2.0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("flags", [0, 1])
def test_mla_rms(fmt, flags):
    # a token over 196 tiles, alone (more tiles than CTAs) and among others, and with the fixed order
    import dsa_sparse_attention_gb300 as dsa
    case = make_case([25000, 800, 3000], [1, 40, 9], seed=302, lat_fmt=fmt)
    d = DeviceTree(case, flags=flags * dsa.DSA_BATCH_INVARIANT)
    out, _ = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    out = out.float().cpu().numpy()
    for t in [0, 1, 2, 7, 20, 39, 40, 41, 45, 49]:
        use = rms_use(case, out, t)
        assert use < 1.0, f"token {t}: rms error {use:.3g} of its bound"


# ------------------------------------------------------------------- very long rows

@pytest.mark.gpu
@pytest.mark.parametrize("shape", ["normal", "late"])
def test_topk_row_of_millions(shape):
    # more than 1,024 chunks of 4,096 scores: the selection places its entries in more than one round
    case, scores = _topk_case([4300000], [3], seed=304)
    if shape == "late":
        scores[:, 4194304 - 700:4194304 + 900] += 20
    idx, _ = _topk(case, scores, 2048)
    _check_topk(case, scores, 2048, idx)


# --------------------------------------------------------------- few seen positions

def _samples_seen(n, base, bits, samples=4096):
    """How many of the top-k's sampled positions (one of each of as many equal stretches, at a place
    hashed from its number) a token at position n - 1 sees."""
    q = np.arange(samples, dtype=np.uint64)
    a, b = n * q // samples, n * (q + 1) // samples
    h = (q * 2654435761) & 0xFFFFFFFF
    h ^= h >> 15
    at = a + h % (b - a)
    d = at.astype(np.int64) - base
    return int(np.sum((d < 0) | np.isin(d, np.flatnonzero(bits))))


def _rank(n, k, samples=4096):
    m = np.float32(samples) * np.float32(k) / np.float32(n)
    return min(int(m + np.float32(6) * np.sqrt(m)) + 8, samples)


# positions of the context, committed, k, mask words, and whether fewer samples are seen than the bound's rank
# where that is taken from all samples (it is above the 256 groups')
FEW = [(20000, 2100, 2048, 1, True), (19996, 1100, 1024, 1, True), (16000, 0, 900, 32, True), (15000, 300, 1200, 32, True),
       (40000, 2060, 2048, 2, True), (60000, 2100, 2048, 1, False), (200000, 2100, 2048, 1, False),
       (30000, 1, 20, 1, False)]


def _few_case(n, base, k, words, tokens=4):
    rng = np.random.default_rng(n + base)
    case, scores = _topk_case([n - tokens], [tokens], seed=n, words=words)
    case.base[0] = base
    bits = rng.random((tokens, words * 32)) < 0.97
    bits[:, 0] = True
    case.mask[:] = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)
    unseen = np.ones(scores.shape, bool)
    for t in range(tokens):
        unseen[t, case.seen(t)] = False
    scores[unseen] = np.where(rng.random(int(unseen.sum())) < 0.5, np.float32(np.nan), np.float32(9.0))
    return case, scores, bits


def test_few_seen_cases_are_what_they_say():
    # (no GPU) the cases do have more positions seen than k, and fewer samples seen than the rank where they say so
    for n, base, k, words, fewer in FEW:
        case, _, bits = _few_case(n, base, k, words)
        for t in range(4):
            pos = int(case.wl.q_pos[t])
            assert case.seen(t).size > k
            rank = _rank(pos + 1, k)
            assert (rank > 256 and _samples_seen(pos + 1, base, bits[t]) < rank) == fewer


@pytest.mark.gpu
@pytest.mark.parametrize("n,base,k,words,fewer", FEW)
def test_topk_few_seen_on_long_rows(n, base, k, words, fewer):
    # a small committed context, a narrow mask and a position far behind both: most of the row is not
    # seen, and what lies there, NaN and larger scores, is not compared
    case, scores, _ = _few_case(n, base, k, words)
    idx, ph = _topk(case, scores, k, phys=True)
    _check_topk(case, scores, k, idx, ph)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
def test_mla_few_seen_in_a_long_context(fmt):
    # whole tiles that nobody sees between the committed context and the token
    case = make_case([4990, 3000], [4, 2], seed=303, lat_fmt=fmt)
    case.base[:] = [300, 0]
    case.mask[:4, 0] = [0xFFFFFFFF, 0x80000001, 0, 0x00F0F0F0]
    case.mask[4:, 0] = [0x80000000, 0]          # one position of 3,000; nothing
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    check_mla(case, out, lse)


# ------------------------------------------------------------------ far-out logits

@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [1e3, 1e5, 1e6, 1.7e6])
def test_mla_logits_of_hundred_millions(fmt, scale):
    # Logits up to 2^28 in log2 units, where an fp32 logit is 16 apart from the next: one position takes
    # a head's weight, and its latent, exact in bf16 (6 significant bits at most), is the result, but for
    # the others' weights: each is at most exp(2 e - gap) < exp(-40), 702 of them times the largest latent.
    # Heads whose two largest logits lie nearer than four times their error e have no such answer.
    # (Without the weights' cap 4 and 7 of the 192 heads were not finite at 1e6, 175 and 179 at 1.7e6.)
    case = make_case([700], [2], seed=305, lat_fmt=fmt)
    wl = case.wl
    wl.sm_scale = scale
    d = DeviceTree(case)
    out, lse = d.mla()
    torch.cuda.synchronize()
    assert _check(d.ws) == 0
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    clear = 0
    for t in range(2):
        lat = O.gather_latents(oracle_layout(wl), wl.block_table[0], case.seen(t))
        q = O.decode_bf16(wl.q[t]).reshape(96, 576)
        logits = scale * (q @ lat.T)
        assert np.abs(logits).max() * 1.4427 < 2.0 ** 28
        e = 2.0 ** -18 * scale * (np.abs(q) @ np.abs(lat).T).max(axis=1)
        best = logits.argmax(axis=1)
        two = np.sort(logits, axis=1)[:, -2:]
        for h in np.flatnonzero(two[:, 1] - two[:, 0] > 4 * e + 40):
            off = np.abs(out[t, h] - lat[best[h], :512]).max()
            assert off <= 702 * np.exp(-40.0) * np.abs(lat).max(), f"token {t}, head {h}: {off}"
            assert abs(lse[t, h] - two[h, 1]) <= e[h] + 1e-6 * abs(two[h, 1])
            clear += 1
    assert clear > 150
