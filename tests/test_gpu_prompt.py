"""Prompt attention on the GPU against the float64 oracle (tolerances: tests/prompt_cases.py)."""
import numpy as np
import pytest
import torch

from tests.prompt_cases import PromptCase

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_sparse_attention_gb300.build import build
    build()


def _run(case):
    import dsa_sparse_attention_gb300 as dsa
    case.to_device().run()
    assert dsa.dsa_check(case.ws) == 0
    return case.check()


SHAPES = [(4, 4, 128, 64), (4, 4, 128, 0), (3, 3, 64, 0), (2, 2, 64, 64)]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens", [[(1, 1)], [(33, 33)], [(128, 128)], [(300, 300)]])
def test_one_sequence(lens, shape, dt):
    h, g, d, e = shape
    _run(PromptCase(lens, h, g, d, e, dt, seed=len(lens) + d + e))


RAGGED = [(127, 127), (1, 300), (0, 5), (129, 129), (5, 0), (64, 200), (40, 17), (256, 256), (0, 0), (257, 400), (1, 1)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES + [(8, 1, 128, 0), (28, 4, 128, 0), (10, 2, 64, 0), (128, 1, 64, 64), (6, 2, 128, 64),
                                            (96, 2, 128, 0)])
def test_ragged(shape, causal):
    h, g, d, e = shape
    _run(PromptCase(RAGGED, h, g, d, e, BF if h % 4 else FP, causal, seed=h + d, gap=3))


@pytest.mark.parametrize("layout", ["kv", "heads", "wide"])
@pytest.mark.parametrize("dim,shared", [(128, 64), (64, 0)])
def test_strides(layout, dim, shared):
    _run(PromptCase([(70, 70), (1, 90), (200, 333)], 6, 3, dim, shared, BF, True, seed=5, gap=2, layout=layout))


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("causal,prev", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("shape", [(4, 4, 128, 64), (16, 2, 128, 0), (5, 1, 64, 0), (2, 2, 64, 64)])
def test_few_rows_split_over_the_keys(shape, causal, prev, dt):
    h, g, d, e = shape
    case = PromptCase([(1, 5000), (3, 700), (2, 1), (4, 0), (1, 512), (1, 513), (7, 4095), (0, 9)], h, g, d, e, dt, causal,
                      seed=17, gap=1, prev=prev)
    case.to_device()
    assert case.ws.numel() > 256        # parts
    _run(case)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [RAGGED, [(1, 5000), (2, 700)], [(3, 0), (100, 90)]])
@pytest.mark.parametrize("dim,shared", [(128, 64), (64, 0)])
def test_joined_with_an_earlier_result(lens, dim, shared, causal):
    _run(PromptCase(lens, 4, 2, dim, shared, BF, causal, seed=3, prev=True))
    # and in its place
    case = PromptCase(lens, 4, 2, dim, shared, FP, causal, seed=4, prev=True).to_device()
    rows = slice(int(case.cu_q[0]), int(case.cu_q[-1]))
    case.out[rows], case.lse[rows] = case.d_prev[0][rows], case.d_prev[1][rows]
    case.d_prev = (case.out, case.lse)
    case.run()
    case.check()


def test_outputs_that_begin_off_32_bytes():
    for lens in ([(300, 300)], [(1, 900)], [(40, 300)]):
        case = PromptCase(lens, 4, 2, 128, 0, BF, True, seed=3).to_device()
        t = case.out.shape[0]
        room = torch.full((t * 4 * 128 + 16,), 7.0, dtype=BF, device="cuda")
        case.out = room[8:8 + t * 4 * 128].view(t, 4, 128)
        assert case.out.data_ptr() % 32 == 16
        case.run()
        case.check()
        assert torch.all(room[:8] == 7.0) and torch.all(room[-8:] == 7.0)


@pytest.mark.parametrize("shape", [(8, 8, 128, 64), (64, 8, 128, 0), (4, 2, 64, 0), (3, 3, 64, 64)])
def test_items_of_a_tile_or_none(shape):
    """Many single tokens whose keys, or whose last part's keys, are one tile or none: CTAs go from item to
    item with one S or neither in use."""
    import dsa_sparse_attention_gb300 as dsa
    h, g, d, e = shape
    lens = [(1, n) for n in (1, 513, 128, 129, 0, 640, 600, 1, 1025, 90, 1100, 0, 0, 16, 1537, 2)] * 6
    case = PromptCase(lens, h, g, d, e, BF, True, seed=21).to_device()
    case.run()
    assert dsa.dsa_check(case.ws) == 0
    case.check()
    first, fl = case.out.clone(), case.lse.clone()
    for _ in range(200):
        case.run()
    assert dsa.dsa_check(case.ws) == 0 and torch.equal(case.out, first) and torch.equal(case.lse, fl)


def test_runs_longer_than_one_accumulator_sums():
    """150,000 keys whose values have one sign, in fp16: runs of 65,536 keys merged in fp32, and with the
    invariant flag the same bits alone and beside a longer sequence."""
    import dsa_sparse_attention_gb300 as dsa
    kw = dict(heads=2, kv=1, dim=64, dt=FP, causal=True, flags=dsa.DSA_PROMPT_INVARIANT)
    long = PromptCase([(3, 150_000), (5, 700), (2, 66_000)], seed=31, **kw)
    long.v = long.v.abs() + 0.5
    long.to_device().run()
    assert dsa.dsa_check(long.ws) == 0
    long.check()
    a, b = int(long.cu_q[1]), int(long.cu_k[1])
    one = PromptCase([(5, 700)], seed=0, **kw)
    one.q, one.k, one.v, one.ks = long.q[a:a + 5], long.k[b:b + 700], long.v[b:b + 700], long.ks[b:b + 700]
    one.to_device().run()
    assert torch.equal(one.out, long.out[a:a + 5]) and torch.equal(one.lse, long.lse[a:a + 5])


def test_joining_chunks_is_one_call_over_both():
    import dsa_sparse_attention_gb300 as dsa
    whole = PromptCase([(150, 900), (20, 333)], 4, 4, 128, 64, FP, True, seed=8)
    whole.to_device()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    # the first part of every context (no row's own tokens among it), then the rest on top, in place
    cut = [500, 256]
    rows = [torch.arange(0, 500), torch.arange(900, 900 + 256)]
    rest = [torch.arange(500, 900), torch.arange(900 + 256, 1233)]
    out, lse = torch.empty_like(whole.out), torch.empty_like(whole.lse)
    for n, (part, cu, flags) in enumerate([(rows, (0, 500, 756), 0), (rest, (0, 400, 477), dsa.DSA_PROMPT_CAUSAL)]):
        at = torch.cat(part).cuda()
        k, v, ks = whole.dk[at], whole.dv[at], whole.dks[at]
        cu_k = i32(*cu)
        pr = dsa.make_prompt(whole.d_cu_q, cu_k, whole.dq, k, v, ks, 150, 500, flags)
        prev = dict(prev_out=out, prev_lse=lse) if n else {}
        ws = dsa.alloc_prompt_workspace(pr)
        dsa.dsa_prompt_attn(pr, whole.dq, k, v, whole.scale, out, lse, k_shared=ks, ws=ws, **prev)
        assert dsa.dsa_check(ws) == 0
    assert sum(cut) == 756
    whole.run()
    # the earlier result's rounding to fp16 comes on top: half a step of a value of at most sum p |v|
    assert (out.double() - whole.out.double()).abs().max().item() <= 4 * 2.0 ** -11 * whole.v.abs().max().item()
    assert (lse - whole.lse).abs().max().item() <= 1e-4


def test_earlier_results_that_weigh_nothing_are_not_read():
    case = PromptCase([(5, 40), (3, 0)], 4, 4, 64, 0, BF, False, seed=2, prev=True)
    case.prev_lse[:] = float("-inf")
    case.prev_out[:] = float("nan")
    _run(case)


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("lens", [[(600, 1500), (130, 130)], [(1, 2000)], [(100, 1500)]])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("top", [12.0, 300.0])
def test_growing_logits_move_the_reference(dt, lens, dim, top):
    # Keys grow along the sequence and point where the queries do: every tile's logits pass the last's by far
    # (by 3,400 at most, which is more than a bf16 weight holds).
    case = PromptCase(lens, 2, 2, dim, 0, dt, True, seed=4)
    q = torch.sign(torch.randn(1, 2, dim, generator=torch.Generator().manual_seed(1)))
    n = case.k.shape[0]
    case.q = (q + 0.01 * case.q.float()).to(dt)
    case.k = (q * torch.linspace(0.0, top, n)[:, None, None] + 0.05 * case.k.float()).to(dt)
    _run(case)


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("lens", [[(600, 1500)], [(1, 2000)]])
@pytest.mark.parametrize("dt", [BF, FP])
def test_single_logits_far_above_the_others(dt, lens, dim):
    # One key in each of some tiles, in every half of them, passes all before it; between them the weights are small.
    case = PromptCase(lens, 2, 1, dim, 0, dt, False, seed=4)
    q = torch.sign(torch.randn(1, 1, dim, generator=torch.Generator().manual_seed(1)))
    case.q = (q + 0.1 * case.q.float()).to(dt)
    k = 0.1 * case.k.float()
    for n, at in enumerate((3, 70, 200, 383, 384, 700, 1279, 1499)):
        k[at] = q * (0.5 * (n + 1))
    case.k = k.to(dt)
    _run(case)


def test_falling_logits_underflow():
    case = PromptCase([(130, 1500)], 2, 2, 128, 0, FP, False, seed=6)
    q = torch.sign(torch.randn(1, 2, 128, generator=torch.Generator().manual_seed(1)))
    case.q = (q + 0.01 * case.q.float()).to(FP)
    case.k = (q * torch.linspace(12.0, -12.0, 1500)[:, None, None]).to(FP)
    _run(case)


@pytest.mark.parametrize("dim,shared", [(128, 64), (128, 0), (64, 0)])
@pytest.mark.parametrize("lens", [[(600, 1500)], [(1, 2000)], [(100, 330)]])
@pytest.mark.parametrize("dt", [BF, FP])
def test_keys_whose_logits_are_minus_infinity(dt, lens, dim, shared):
    # They weigh nothing, though the first tiles hold no other: the result is that over the keys behind.
    case = PromptCase(lens, 2, 1, dim, shared, dt, False, seed=8)
    case.q[..., 0] = 0.5
    case.k[:300, :, 0] = float("-inf")
    case.to_device().run()
    (lq, lk), = lens
    case.lens, case.cu_k = [(lq, lk - 300)], np.asarray([300, lk])
    case.check()


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("lens", [[(600, 700)], [(1, 2000)]])
@pytest.mark.parametrize("dt", [BF, FP])
def test_logits_of_a_hundred_million_are_finite(dt, lens, dim):
    # fp32 holds them to 16 at best: a weight may be 2^8 too large, which either type holds (0.86 * 2^27)
    case = PromptCase(lens, 2, 2, dim, 0, dt, True, seed=4, scale=2.5 * 128 / dim)
    sign = torch.sign(torch.randn(1, 2, dim, generator=torch.Generator().manual_seed(1)))
    case.q = (sign * 600.0 + case.q.float()).to(dt)
    case.k = (sign * 600.0 + case.k.float()).to(dt)
    case.to_device().run()
    # Logits known to 2^-18 of 10^8 leave the weights of keys within 400 of the largest open (the tolerance of
    # other cases is of first order in that error, which must be below 1): any mean of the values is right, up to
    # a rounding of a weight and of the result.
    u = torch.finfo(dt).eps / 2
    most = case.v.abs().amax(0).cuda().double() * (1 + 4 * u)
    assert torch.isfinite(case.out).all() and (case.out.double().abs() <= most).all()
    assert torch.isfinite(case.lse).all() and (case.lse > 0.9e8).all() and (case.lse < 1.5e8).all()


@pytest.mark.parametrize("dim,shared", [(128, 64), (128, 0), (64, 0)])
@pytest.mark.parametrize("lens,prev", [([(600, 1500)], False), ([(1, 2000)], True), ([(100, 330)], True), ([(600, 700)], True)])
def test_nan_stays_in_the_rows_that_see_it(lens, prev, dim, shared):
    case = PromptCase(lens, 2, 1, dim, shared, BF, True, seed=8, prev=prev).to_device()
    out, lse = (x.clone() for x in case.run())
    (lq, lk), = lens
    row, key = lq // 2, lk - lq // 3 - 1      # a query, and a key that the last third sees
    case.dq[row, 1, 0] = float("nan")
    case.dk[key, 0, 5] = float("nan")
    if prev:
        case.d_prev[1][0] = float("-inf")     # the first row sees keys alone
    case.run()
    nan = torch.zeros(lq, 2, dtype=torch.bool, device="cuda")
    nan[key - (lk - lq):] = True
    nan[row, 1] = True
    assert torch.equal(torch.isnan(case.lse), nan)
    assert torch.equal(torch.isnan(case.out), nan[..., None].expand(case.out.shape))
    rest = ~nan
    rest[0] = False
    assert torch.equal(case.out[rest], out[rest]) and torch.equal(case.lse[rest], lse[rest])


@pytest.mark.parametrize("dim,shared", [(128, 64), (64, 0)])
def test_invariant_rows_do_not_depend_on_the_bound(dim, shared):
    import dsa_sparse_attention_gb300 as dsa
    got = []
    for max_k in (900, 70000):                # one run of keys, or two of which one is empty
        case = PromptCase([(300, 900), (1, 40), (3, 0)], 2, 1, dim, shared, BF, True, seed=8, prev=True,
                          flags=dsa.DSA_PROMPT_INVARIANT, max_k=max_k)
        _run(case)
        got.append((case.out, case.lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_many_short_sequences():
    rng = np.random.default_rng(0)
    lens = [(int(a), int(b)) for a, b in rng.integers(0, 4, (1500, 2))]
    _run(PromptCase(lens, 2, 1, 64, 0, BF, True, seed=9))


def test_all_empty():
    import dsa_sparse_attention_gb300 as dsa
    _run(PromptCase([(7, 0), (130, 0)], 4, 4, 128, 64, BF, True, seed=1))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 4, 128, dtype=BF, device="cuda")
    k = torch.zeros(9, 4, 128, dtype=BF, device="cuda")
    pr = dsa.make_prompt(i32(0, 0), i32(0, 9), q, k, k)
    dsa.dsa_prompt_attn(pr, q, k, k, 1.0, q, ws=dsa.alloc_prompt_workspace(pr))


@pytest.mark.parametrize("lens", [[(300, 300)], [(1, 3000)]])
def test_without_lse(lens):
    import dsa_sparse_attention_gb300 as dsa
    case = PromptCase(lens, 4, 2, 64, 0, BF, True, seed=1).to_device()
    case.run()
    out = torch.empty_like(case.out)
    dsa.dsa_prompt_attn(case.prompt, case.dq, case.dk, case.dv, case.scale, out, ws=case.ws)
    assert torch.equal(out, case.out)


def test_arrays_that_go_up_and_down():
    """Overlapping sequences between descending ones: recorded, and nothing is written out of range."""
    import dsa_sparse_attention_gb300 as dsa
    case = PromptCase([(90, 90)] + [(0, 0)] * 40, 4, 4, 64, 0, BF, True, seed=3, max_q=90, max_k=90).to_device()
    room = torch.full((3 * case.out.numel(),), 7.0, dtype=BF, device="cuda")
    case.out = room[case.out.numel():2 * case.out.numel()].view(case.out.shape)
    up_down = torch.tensor([0, 90] * 20 + [0], dtype=torch.int32)
    case.d_cu_q[:41].copy_(up_down)
    case.d_cu_k[:41].copy_(up_down)
    case.run()
    assert dsa.dsa_check(case.ws) == -6
    n = case.out.numel()
    assert torch.all(room[:n] == 7.0) and torch.all(room[2 * n:] == 7.0)


def test_lengths_that_break_the_rules_are_recorded_and_left():
    import dsa_sparse_attention_gb300 as dsa
    good = PromptCase([(9, 30), (20, 20), (11, 40)], 4, 4, 64, 0, BF, True, seed=3)
    for cu_q, cu_k, left in [((0, 9, 29, 41), (0, 30, 50, 90), (2,)), ((-1, 9, 29, 40), (0, 30, 50, 90), (0,)),
                             ((0, 9, 8, 40), (0, 30, 50, 90), (1, 2)), ((0, 9, 29, 40), (0, 30, 50, 91), (2,)),
                             ((0, 9, 29, 40), (0, 30, 29, 90), (1, 2))]:
        good.to_device()
        good.d_cu_q.copy_(torch.tensor(cu_q, dtype=torch.int32))
        good.d_cu_k.copy_(torch.tensor(cu_k, dtype=torch.int32))
        good.run()
        assert dsa.dsa_check(good.ws) == -6
        assert dsa.dsa_check(good.ws) == 0
        out = good.out.cpu()
        for i in left:
            a, b = (0, 9, 29, 40)[i], (9, 29, 40)[i]
            if (cu_q[i], cu_q[i + 1]) == (8, 40):
                continue   # longer than max_q: nothing of it is written, and its rows are others' too
            assert torch.all(out[a:b] == 7.0)
        keep = [i for i in range(3) if i not in left]
        good.check(seqs=keep)


def test_bounds_that_are_too_small_are_recorded():
    import dsa_sparse_attention_gb300 as dsa
    case = PromptCase([(9, 30), (20, 700)], 4, 4, 64, 0, BF, True, seed=3, max_q=20, max_k=600)
    case.to_device().run()
    assert dsa.dsa_check(case.ws) == -6
    assert torch.all(case.out[9:] == 7.0)
    case.check(seqs=[0])


def test_a_row_is_the_same_alone_and_in_a_batch():
    import dsa_sparse_attention_gb300 as dsa
    kw = dict(heads=6, kv=3, dim=128, shared=64, dt=BF, causal=True, flags=dsa.DSA_PROMPT_INVARIANT)
    many = PromptCase([(30, 700), (257, 999), (1, 1), (3, 3000)], seed=11, **kw).to_device()
    many.run()
    for i, (a, b) in enumerate(zip(many.cu_q, many.cu_k)):
        if i == 4:
            break
        lq, lk = many.lens[i]
        for part in (lq, 1):             # the whole sequence, and its last token alone
            one = PromptCase([(part, lk)], seed=0, **kw)
            one.q, one.k, one.v, one.ks = (x[a + lq - part:a + lq] if x is many.q else x[b:b + lk]
                                           for x in (many.q, many.k, many.v, many.ks))
            one.to_device().run()
            assert torch.equal(one.out, many.out[a + lq - part:a + lq])
            assert torch.equal(one.lse, many.lse[a + lq - part:a + lq])


def test_replayed_graphs_and_streams():
    import dsa_sparse_attention_gb300 as dsa
    cases = [PromptCase([(200, 200), (3, 2100)], 4, 4, 128, 64, BF, True, seed=s).to_device() for s in (1, 2)]
    few = PromptCase([(1, 3000), (1, 100)], 4, 2, 64, 0, FP, True, seed=3).to_device()
    want = []
    for c in cases + [few]:
        c.run()
        want.append((c.out.clone(), c.lse.clone()))
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for c, s in zip(cases + [few], streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, (o, l) in zip(cases + [few], want):
        assert torch.equal(c.out, o) and torch.equal(c.lse, l)
        c.out.fill_(7.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        few.run()
        cases[0].run()
        few.run()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(few.out, want[2][0]) and torch.equal(cases[0].out, want[0][0])
    # new lengths in the same arrays: the graph reads them on the device
    few.d_cu_k.copy_(torch.tensor([0, 40, 100], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    few.lens, few.cu_k = [(1, 40), (1, 60)], np.asarray([0, 40, 100])
    few.check()
    assert all(dsa.dsa_check(c.ws) == 0 for c in cases + [few])


def test_the_same_bits_from_every_call():
    case = PromptCase([(700, 700), (90, 2500)], 8, 8, 128, 64, BF, True, seed=13).to_device()
    case.run()
    first, fl = case.out.clone(), case.lse.clone()
    for _ in range(60):
        case.out.fill_(0.0)
        case.run()
        assert torch.equal(case.out, first) and torch.equal(case.lse, fl)


def test_far_rows():
    # rows 16 KB apart: offsets of keys and values pass 2^31 elements
    import dsa_sparse_attention_gb300 as dsa
    n, dt = 300_000, BF
    buf = torch.empty(n * 8192, dtype=dt, device="cuda")
    k, v = buf.as_strided((n, 1, 64), (8192, 64, 1)), buf.as_strided((n, 1, 64), (8192, 64, 1), 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
    v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
    q = torch.randn((2, 1, 64), generator=g, device="cuda").to(dt)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu_q, cu_k = i32(0, 1, 2), i32(0, 290_000, n)
    case = PromptCase([(1, 290_000), (1, 10_000)], 1, 1, 64, 0, dt, True)
    case.q, case.k, case.v = q.cpu(), k.cpu(), v.cpu()
    for flags in (dsa.DSA_PROMPT_CAUSAL, dsa.DSA_PROMPT_CAUSAL | dsa.DSA_PROMPT_INVARIANT):
        pr = dsa.make_prompt(cu_q, cu_k, q, k, v, flags=flags)
        ws = dsa.alloc_prompt_workspace(pr)
        out, lse = torch.empty_like(q), torch.empty(2, 1, device="cuda")
        dsa.dsa_prompt_attn(pr, q, k, v, case.scale, out, lse, ws=ws)
        assert dsa.dsa_check(ws) == 0
        case.check(out, lse)


def test_prompt_over_the_cache():
    """Write a chunk, read the whole context back, expand it per head, attend: the same as the absorbed
    attention over the latents themselves (the values' projection applied to its result)."""
    import dsa_sparse_attention_gb300 as dsa
    from dsa_sparse_attention_gb300 import workloads as W
    from dsa_sparse_attention_gb300.harness import DeviceWorkload
    new, ctx = [37, 130], [700, 45]
    wl = W.make_workload([a + b for a, b in zip(new, ctx)], new, seed=3, permute=True, pool_rows=60)
    dw = DeviceWorkload(wl)
    T, N = sum(new), sum(new) + sum(ctx)
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dsa.dsa_write_tokens(dw.layout, dw.batch, randn(T, 128).to(BF), randn(T, 576).to(BF), ws=ws)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu_q, cu_k = i32(0, 37, 167), i32(0, 737, 912)
    lat = torch.empty(N, 576, dtype=BF, device="cuda")
    dsa.dsa_read_tokens(dw.layout, dw.batch, dsa.make_spans(cu_k, None, N), None, lat, ws=ws)
    w_uk, w_uv = (randn(512, 96, 128) * 512 ** -0.5 for _ in range(2))
    # one projection for keys and values of a head, side by side
    kv = torch.einsum("nc,chd->nhd", lat[:, :512].float(), torch.cat((w_uk, w_uv), 2)).to(BF)
    k, v, ks = kv[..., :128], kv[..., 128:], lat[:, 512:]
    q = randn(T, 96, 192).to(BF)
    scale = 192 ** -0.5
    pr = dsa.make_prompt(cu_q, cu_k, q, k, v, ks, 130, 737, dsa.DSA_PROMPT_CAUSAL)
    pws = dsa.alloc_prompt_workspace(pr)
    out, lse = torch.empty(T, 96, 128, dtype=BF, device="cuda"), torch.empty(T, 96, device="cuda")
    dsa.dsa_prompt_attn(pr, q, k, v, scale, out, lse, k_shared=ks, ws=pws)
    # absorbed: q . (W_uk c) = (W_uk^T q) . c, over the pages as they are
    qa = torch.cat((torch.einsum("thd,chd->thc", q[..., :128].float(), w_uk), q[..., 128:].float()), 2).to(BF)
    tree = dsa.make_tree(dw.ctx, torch.zeros(T, 1, dtype=torch.int32, device="cuda"))
    tws = dsa.alloc_tree_workspace(dw.layout, dw.batch)
    o2, l2 = torch.empty(T, 96, 512, dtype=BF, device="cuda"), torch.empty(T, 96, device="cuda")
    dsa.dsa_tree_mla(dw.layout, dw.batch, tree, qa, scale, o2, l2, ws=tws)
    assert dsa.dsa_check(ws) == 0 and dsa.dsa_check(pws) == 0 and dsa.dsa_check(tws) == 0
    want = torch.einsum("thc,chd->thd", o2.float(), w_uv)
    # Both sides round keys or absorbed queries, values and results to bf16 once each: logits of about
    # N(0, 1) move by 2^-8 / sqrt(12) * sqrt(2), the results by a few half steps of their rms.
    rel = (out.float() - want).norm() / want.norm()
    assert rel.item() <= 4 * 2.0 ** -8, rel.item()
    assert (lse - l2).abs().max().item() <= 0.05
