"""Seeded packed sequences for the prompt attention, and their comparison with the oracle.

Tolerance, from the roundings the attention makes, u being half a step of the inputs' type
(bf16 2^-8, fp16 2^-11): a weight is rounded once to that type, the sum is of the weights before
that, so the output moves by at most u * A with A = sum p |v|; the output is rounded once, u *
|out|.  Logits are sums of at most 192 exact products in fp32: their error is at most 2^-18 *
scale * sum |q k| (two bits for the order and the truncation of a tensor-core sum), and 2^-21 *
(1 + their size) for the fp32 scaling and the exponential; a weight moves by that error e, the
output by 2 e A, the lse by e.  The tensor core truncates where it adds 16 keys' products to the
accumulator: 2^-23 of the sum's terms for each of the 8 steps of a tile of 128 keys, 2^-20 A a
tile, of which 512 at most are summed in a run.  An fp16 weight is exact to 2^-25 of 2^7 or more that the heaviest weighs: 2^-32 * sum |v|.
A joined result weighs both sides in fp32: 2^-20 of each.
"""
import numpy as np
import torch

from oracle import prompt as P

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class PromptCase:
    """Sequences of (queries, keys), values N(0, 1); rows of no sequence are `gap` long, in front,
    between (at `between`) and behind, and hold NaN."""

    def __init__(self, lens, heads=4, kv=4, dim=128, shared=0, dt=torch.bfloat16, causal=True, seed=0, gap=0, flags=0,
                 prev=False, scale=None, max_q=None, max_k=None, layout="plain"):
        import dsa_sparse_attention_gb300 as dsa
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dt, self.causal = lens, dt, causal
        self.heads, self.kv, self.dim, self.shared = heads, kv, dim, shared
        self.scale = scale or 1.0 / float(np.sqrt(dim + shared))
        lq, lk = [a for a, _ in lens], [b for _, b in lens]
        self.cu_q = np.concatenate([[0], np.cumsum(lq)]) + gap
        self.cu_k = np.concatenate([[0], np.cumsum(lk)]) + gap
        t, n = int(self.cu_q[-1]) + gap, int(self.cu_k[-1]) + gap
        randn = lambda *s: torch.randn(s, generator=g, dtype=torch.float32)
        q, k, v, ks = randn(t, heads, dim + shared) * 1.5, randn(n, kv, dim), randn(n, kv, dim), randn(n, shared)
        for x, cu in ((q, self.cu_q), (k, self.cu_k), (v, self.cu_k), (ks, self.cu_k)):
            x[:cu[0]] = float("nan")
            x[cu[-1]:] = float("nan")
        self.q, self.k, self.v, self.ks = (x.to(dt) for x in (q, k, v, ks))
        self.prev_out = randn(t, heads, dim).to(dt) if prev else None
        self.prev_lse = (randn(t, heads) + 3.0) if prev else None
        self.layout, self.flags = layout, flags | (dsa.DSA_PROMPT_CAUSAL if causal else 0)
        self.max_q, self.max_k = max_q or max(lq + [1]), max_k or max(lk + [1])

    def to_device(self):
        import dsa_sparse_attention_gb300 as dsa
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        self.d_cu_q, self.d_cu_k = i32(self.cu_q), i32(self.cu_k)
        dq, dk, dv = self.q.cuda(), self.k.cuda(), self.v.cuda()
        if self.layout == "kv":             # one projection's output: keys and values of a head side by side
            both = torch.cat((dk, dv), 2)
            dk, dv = both[..., :self.dim], both[..., self.dim:]
        elif self.layout == "heads":        # heads outermost
            dq, dk, dv = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (dq, dk, dv))
        elif self.layout == "wide":         # columns of a wider array
            wide = lambda x: torch.cat((x, x.new_full((*x.shape[:2], 8), float("nan"))), 2)[..., :x.shape[2]]
            dq, dk, dv = wide(dq), wide(dk), wide(dv)
        self.dq, self.dk, self.dv = dq, dk, dv
        self.dks = None
        if self.shared:                     # the last dims of latents
            lat = torch.full((self.ks.shape[0], 576), float("nan"), dtype=self.dt, device="cuda")
            lat[:, 576 - self.shared:] = self.ks.cuda()
            self.dks = lat[:, 576 - self.shared:]
        t = self.q.shape[0]
        self.out = torch.full((t, self.heads, self.dim), 7.0, dtype=self.dt, device="cuda")
        self.lse = torch.full((t, self.heads), 7.0, dtype=torch.float32, device="cuda")
        self.prompt = dsa.make_prompt(self.d_cu_q, self.d_cu_k, dq, dk, dv, self.dks, self.max_q, self.max_k, self.flags)
        self.ws = dsa.alloc_prompt_workspace(self.prompt)
        self.d_prev = (None, None) if self.prev_out is None else (self.prev_out.cuda(), self.prev_lse.cuda())
        return self

    def run(self, stream=None):
        import dsa_sparse_attention_gb300 as dsa
        dsa.dsa_prompt_attn(self.prompt, self.dq, self.dk, self.dv, self.scale, self.out, self.lse, k_shared=self.dks,
                            prev_out=self.d_prev[0], prev_lse=self.d_prev[1], ws=self.ws, stream=stream)
        return self.out, self.lse

    def check(self, out=None, lse=None, seqs=None, prev=None):
        """Every row of every sequence against the oracle; returns the worst use of the tolerance."""
        out = (self.out if out is None else out).double().cpu().numpy()
        lse = (self.lse if lse is None else lse).double().cpu().numpy()
        u, worst = U[self.dt], 0.0
        f = lambda x, a, b: x[a:b].double().numpy()
        prev = prev or (self.prev_out, self.prev_lse)
        for i, (lq, lk) in enumerate(self.lens):
            if (seqs is not None and i not in seqs) or lq == 0:
                continue
            a, c = int(self.cu_q[i]), int(self.cu_k[i])
            v = f(self.v, c, c + lk)
            ref, rl, A, big = P.attention(f(self.q, a, a + lq), f(self.k, c, c + lk), v, self.scale, self.causal,
                                          f(self.ks, c, c + lk) if self.shared else None)
            e = 2.0 ** -18 * big + 2.0 ** -21 * (1 + big)
            vsum = np.repeat(np.abs(v).sum(axis=0), self.heads // self.kv, axis=0)[None]
            part = (u + 2 * e[..., None] + min((lk + 127) // 128, 512) * 2.0 ** -20) * (1 + 2 * u) * A + 2.0 ** -32 * vsum
            tl = e + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(rl), rl, 0.0)))
            if prev[0] is not None:
                po, pl = f(prev[0], a, a + lq), f(prev[1], a, a + lq)
                own = ref
                ref, both, wa, wb = P.join(po, pl, own, rl)
                kept = np.where((wa > 0)[..., None], np.abs(po), 0.0)
                part = wb[..., None] * (part + (2 * e[..., None] + 2.0 ** -20) * np.abs(own)) + wa[..., None] * kept * (2 * e[..., None] + 2.0 ** -20)
                rl = both
                tl = tl + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(rl), rl, 0.0)))
            tol = u * np.abs(ref) + part + 1e-30
            got, gl = out[a:a + lq], lse[a:a + lq]
            none = np.isneginf(rl)
            assert np.all(np.isneginf(gl[none])) and not got[none].any(), f"sequence {i}: rows that see nothing"
            assert np.isfinite(got).all() and np.isfinite(gl[~none]).all(), f"sequence {i}: not finite"
            use = (np.abs(got - ref) / tol).max()
            ul = (np.abs(gl[~none] - rl[~none]) / tl[~none]).max() if (~none).any() else 0.0
            assert use <= 1.0, f"sequence {i}: output {use:.3g} of the tolerance"
            assert ul <= 1.0, f"sequence {i}: lse {ul:.3g} of the tolerance"
            worst = max(worst, use, ul)
        rest = np.ones(out.shape[0], bool)
        rest[self.cu_q[0]:self.cu_q[-1]] = False
        assert np.all(out[rest] == 7.0) and np.all(lse[rest] == 7.0), "rows of no sequence are left as they were"
        return worst
