"""Seeded trees of drafted tokens on top of a synthetic workload, their device side,
and the comparison of the dense attention with the oracle.

Tolerance of the attention, from the roundings it makes (relative to the value a
rounding is off by at most half a step: bf16 2^-8, 9 significant bits 2^-9, fp16 2^-11):
a weight is rounded once, to 9 significant bits or more, and the sum is of the weights
before (or after) that rounding, so the output moves by at most 2 * 2^-9 * A with
A = sum p |v|; a partial is rounded to fp16 (2^-11 of it, and of A at most); the output
to bf16.  Logits are sums of
576 exact products in fp32: their error e is at most 2^-18 * scale * sum |q c| (two bits
for the order and the truncation of a tensor-core sum of 2^-24 terms over 576), a weight
moves by e, the output by 2 e A.  The lse moves by 2^-9 + e.
"""
from dataclasses import dataclass

import numpy as np
import torch

from dsa_sparse_attention_gb300 import workloads as W
from oracle import dsa_oracle as O
from oracle import tree as OT
from tests.parity import oracle_layout


@dataclass
class TreeCase:
    wl: object
    base: np.ndarray       # int32 [B]
    mask: np.ndarray       # uint32 [T, words]
    first: list            # first token of each request

    def seen(self, t):
        r = int(self.wl.q_req[t])
        return OT.visible(int(self.base[r]), int(self.wl.q_pos[t]), self.mask[t])


def random_parents(rng, n):
    return [-1] + [int(rng.integers(0, i)) for i in range(1, n)]


def make_case(bases, drafts, seed, *, words=None, parents=None, **kw):
    """Requests with `bases` committed and `drafts` drafted tokens; random trees."""
    rng = np.random.default_rng(seed)
    wl = W.make_workload([b + n for b, n in zip(bases, drafts)], list(drafts), seed=seed, **kw)
    words = max(1, (max(drafts) + 31) // 32) if words is None else words
    mask, first = [], []
    for i, n in enumerate(drafts):
        first.append(sum(drafts[:i]))
        if n:
            mask.append(OT.ancestor_masks(random_parents(rng, n) if parents is None else parents[i], words))
    return TreeCase(wl, np.asarray(bases, np.int32), np.concatenate(mask), first)


class DeviceTree:
    """A case on the GPU."""

    def __init__(self, case, flags=0, max_ctx=None):
        import dsa_sparse_attention_gb300 as dsa
        wl = case.wl
        self.case, self.wl = case, wl
        cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.pool, self.bt, self.ctx = cu(wl.pool), cu(wl.block_table), cu(wl.ctx_lens)
        self.q_req, self.q_pos = cu(wl.q_req), cu(wl.q_pos)
        self.q = cu(wl.q.view(np.int16)).view(torch.bfloat16)
        self.base, self.mask = cu(case.base), cu(case.mask.view(np.int32))
        self.layout = dsa.make_layout(self.pool, wl.num_rows, wl.row_stride, wl.idx_page_offset, wl.lat_page_offset,
                                      wl.block_size, wl.idx_fmt, wl.lat_fmt)
        self.batch = dsa.make_batch(self.q_req, self.q_pos, self.ctx, self.bt, max_ctx or wl.max_ctx_len, flags)
        self.tree = dsa.make_tree(self.base, self.mask)
        T = wl.num_tokens
        self.ws = dsa.alloc_tree_workspace(self.layout, self.batch)
        self.out = torch.full((T, 96, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, 96), 7.0, dtype=torch.float32, device="cuda")

    def mla(self, stream=None):
        import dsa_sparse_attention_gb300 as dsa
        dsa.dsa_tree_mla(self.layout, self.batch, self.tree, self.q, self.wl.sm_scale, self.out, self.lse, ws=self.ws,
                         stream=stream)
        return self.out, self.lse


def check_mla(case, out, lse, tokens=None):
    """Every element of every token against the oracle; returns the worst use of the tolerance."""
    wl = case.wl
    lay = oracle_layout(wl)
    out = out.float().cpu().numpy().astype(np.float64)
    lse = lse.cpu().numpy().astype(np.float64)
    worst = 0.0
    for t in range(wl.num_tokens) if tokens is None else tokens:
        lat = O.gather_latents(lay, wl.block_table[int(wl.q_req[t])], case.seen(t))
        ref, ref_l, A = OT.dense_mla(wl.q[t], lat, wl.sm_scale)
        if lat.shape[0] == 0:
            assert not out[t].any() and np.all(np.isneginf(lse[t])), f"token {t}: sees nothing"
            continue
        q = np.abs(O.decode_bf16(wl.q[t]).reshape(96, 576))
        e = 2.0 ** -18 * abs(wl.sm_scale) * (q @ np.abs(lat).T).max(axis=1)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -11 + 2 * e[:, None]) * (1 + 2.0 ** -7) * A
        tol += 2.0 ** -25 + 2.0 ** -28 * np.abs(lat[:, :512]).sum(axis=0)
        use = (np.abs(out[t] - ref) / np.maximum(tol, 1e-30)).max()
        ul = (np.abs(lse[t] - ref_l) / (2.0 ** -9 + e + 1e-6 * np.abs(ref_l))).max()
        assert np.isfinite(out[t]).all() and use <= 1.0, f"token {t}: output {use:.3g} of the tolerance"
        assert ul <= 1.0, f"token {t}: lse {ul:.3g} of the tolerance"
        worst = max(worst, use, ul)
    return worst
