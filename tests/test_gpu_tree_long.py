"""The dense attention of drafted tokens over contexts of hundreds of thousands of positions, where a
CTA sums many tiles of one token, against float64 sums on the GPU (elementary torch operations).

The tensor core adds to its accumulator by truncation: sums of one sign come out small by a share that
grows with the tiles summed in one run.  A run is 512 tiles long at most and loses 2^-11 of its sum at
most; the runs' sums are added in fp32."""
import pytest
import torch

import dsa_sparse_attention_gb300 as dsa
from dsa_sparse_attention_gb300 import workloads as W

pytestmark = pytest.mark.gpu

FMTS = [W.LAT_FP8, W.LAT_NVFP4]
BS = 64
RUN = 2.0 ** -11          # what a run may lose of its sum
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_sparse_attention_gb300.build import build
    build()


class Long:
    """One request with a context of n positions: random latents, drafted tokens at the last positions."""

    def __init__(self, fmt, n, tokens, seed, base=None, mask=None, flags=0, positive=False, slope=0.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.fmt, self.n, self.T = fmt, n, tokens
        blocks = -(-n // BS)
        rec = 576 if fmt == W.LAT_FP8 else 352
        rb = BS * (132 + rec)
        x = torch.randn((blocks * BS, 576), generator=g, device="cuda")
        if positive:
            x = x.abs()
        if slope:   # the last dim, which the values do not have, moves along the context
            x[:, 560:] = 0
            x[:, 575] = torch.linspace(-slope, slope, blocks * BS, device="cuda")
        lat = (x.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == W.LAT_FP8 else self.nvfp4(x)).view(blocks, -1)
        del x
        perm = torch.randperm(blocks + 2, generator=g, device="cuda")[:blocks]
        self.pool = torch.zeros((blocks + 2, rb), dtype=torch.uint8, device="cuda")
        self.pool[perm, BS * 132:] = lat
        self.lat = lat.view(blocks * BS, rec)[:n]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.bt, self.ctx = perm.to(torch.int32)[None].contiguous(), i32([n])
        self.pos = list(range(n - tokens, n))
        self.base_host = n if base is None else base
        self.mask_host = [[0]] * tokens if mask is None else mask
        self.q = torch.randn((tokens, 96, 576), generator=g, device="cuda").to(torch.bfloat16)
        if slope:   # heads whose logits rise, fall, or do neither by 2 slope
            self.q[:, :, 560:] = 0
            self.q[:, 0::3, 575] = 24.0
            self.q[:, 1::3, 575] = -24.0
        self.inputs = (i32([0] * tokens), i32(self.pos), i32([self.base_host]), i32(self.mask_host))
        layout = dsa.make_layout(self.pool, blocks + 2, rb, 0, BS * 132, BS, dsa.DSA_IDX_FP8, fmt)
        batch = dsa.make_batch(self.inputs[0], self.inputs[1], self.ctx, self.bt, n, flags)
        tree = dsa.make_tree(self.inputs[2], self.inputs[3])
        ws = dsa.alloc_tree_workspace(layout, batch)
        ws[256:].fill_(0xFF)                       # what an earlier call may have left: NaN where sums lie
        self.out = torch.full((tokens, 96, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((tokens, 96), 7.0, device="cuda")
        dsa.dsa_tree_mla(layout, batch, tree, self.q, 1 / 24, self.out, self.lse, ws=ws)
        torch.cuda.synchronize()
        assert dsa.dsa_check(ws) == 0

    @staticmethod
    def nvfp4(x):
        n = x.shape[0]
        rec = torch.zeros((n, 352), dtype=torch.uint8, device="cuda")
        mid = torch.tensor([(a + b) / 2 for a, b in zip(GRID, GRID[1:])], device="cuda")
        for r in range(0, n, 1 << 17):
            y = x[r:r + (1 << 17)].view(-1, 36, 16)
            sc = (y.abs().amax(2) / 6.0).to(torch.float8_e4m3fn)
            v = y / sc.float().clamp_min(2.0 ** -9)[:, :, None]
            code = (torch.bucketize(v.abs(), mid).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)).view(-1, 288, 2)
            rec[r:r + (1 << 17), :288] = code[:, :, 0] | (code[:, :, 1] << 4)
            rec[r:r + (1 << 17), 288:324] = sc.view(torch.uint8)
        return rec

    def latents(self, seen):
        """float64 [seen, 576]"""
        rec = self.lat[seen]
        if self.fmt == W.LAT_FP8:
            return rec.contiguous().view(torch.float8_e4m3fn).double()
        code = torch.stack((rec[:, :288] & 15, rec[:, :288] >> 4), 2).reshape(-1, 36, 16).int()
        grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device="cuda")
        return (grid[code] * rec[:, 288:324].contiguous().view(torch.float8_e4m3fn).double()[:, :, None]).view(-1, 576)

    def seen(self, t):
        s = list(range(min(self.base_host, self.pos[t] + 1)))
        row = self.mask_host[t]
        return s + [self.base_host + i for i in range(32 * len(row))
                    if (row[i >> 5] >> (i & 31)) & 1 and self.base_host + i <= self.pos[t]]

    def exact(self, t):
        """(out, lse, sum p |v|, sum p^2 v^2, largest error of a logit) in float64."""
        c = self.latents(torch.tensor(self.seen(t), dtype=torch.int64, device="cuda"))
        q = self.q[t].double()
        d = q @ c.t() / 24
        lse = torch.logsumexp(d, 1)
        p = torch.exp(d - lse[:, None])
        del d
        e = 2.0 ** -18 / 24 * (q.abs() @ c.abs().t()).amax(1)
        v = c[:, :512]
        return p @ v, lse, p @ v.abs(), (p * p) @ (v * v), e

    def check(self, t):
        """The worst-case bound of every element, and the root mean square of 64 dims, as for short contexts
        (tests/tree_cases.py, tests/test_gpu_tree_edges.py), with what a run may lose beside them."""
        out, lse = self.out[t].double(), self.lse[t].double()
        if not self.seen(t):
            assert not out.any() and bool((lse == -float("inf")).all())
            return
        ref, ref_l, A, spread, e = self.exact(t)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11 + RUN + 2 * e[:, None]) * (1 + 2.0 ** -7) * A + 2.0 ** -25
        use = float(((out - ref).abs() / tol).max())
        assert use <= 1.0, f"token {t}: {use:.3g} of the tolerance"
        assert bool(((lse - ref_l).abs() <= 2.0 ** -9 + e + 1e-6 * ref_l.abs()).all()), f"token {t}: lse"
        chunks = lambda x: x.view(96, 8, 64).mean(2)
        bound = 2 * torch.sqrt((2.0 ** -16 / 3 + RUN * RUN) * chunks(ref ** 2) + (2.0 ** -18 / 3 + e[:, None] ** 2) * chunks(spread))
        rms = float((torch.sqrt(chunks((out - ref) ** 2)) / bound).max())
        assert rms <= 1.0, f"token {t}: rms error {rms:.3g} of its bound"


@pytest.mark.parametrize("fmt,n", [(W.LAT_FP8, 600000), (W.LAT_NVFP4, 300000)])
def test_sums_of_one_sign(fmt, n):
    # a whole token in one CTA: the mean relative error of 49,152 outputs, whose own roundings to bf16
    # (2^-8 / sqrt(3) each, independent) leave 1e-5 of it
    d = Long(fmt, n, 1, 1, flags=dsa.DSA_BATCH_INVARIANT, positive=True)
    ref, lse, _, _, _ = d.exact(0)
    bias = float(((d.out[0].double() - ref) / ref).mean())
    print(f"mean relative error {bias:.3g}")
    assert abs(bias) <= RUN + 6e-5
    assert float((d.lse[0].double() - lse).abs().max()) < 1e-4


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [65536, 65537, 131072, 140000])
def test_one_token_in_one_cta(fmt, n):
    # 512 tiles, one more, two whole runs, a ragged third
    d = Long(fmt, n, 2, 2, flags=dsa.DSA_BATCH_INVARIANT)
    d.check(0)
    d.check(1)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("flags", [0, 1])
def test_references_move_between_runs(fmt, flags):
    # 170 tokens over 70,000 positions, 600 tiles a CTA; logits that rise or fall by 40 along the context
    d = Long(fmt, 70000, 170, 3, flags=flags * dsa.DSA_BATCH_INVARIANT, slope=20.0)
    for t in (0, 1, 50, 85, 120, 169):
        d.check(t)


@pytest.mark.parametrize("fmt", FMTS)
def test_runs_in_which_nothing_is_seen(fmt):
    # tokens far behind a short committed context, some of which see nothing at all: the tiles that are
    # seen come first, last or in the middle of a CTA's share
    T = 170
    mask = [[0x0F0F00FF if t % 3 else 0] for t in range(T)]
    for base in (300, 0):
        d = Long(fmt, 140000, T, 4, base=base, mask=mask)
        for t in range(T):
            d.check(t)
