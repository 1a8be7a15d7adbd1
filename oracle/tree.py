"""Trees of drafted tokens and the rows of the cache, from their definitions
(float64 / plain lists; shares no code with the CUDA path).

visible(t) = {s <= q_pos : s < base or bit (s - base) of the token's mask}.
"""
import numpy as np

from . import dsa_oracle as O


def ancestor_masks(parents, words):
    """Mask rows (uint32 [n, words]) of a tree given by each slot's parent (-1: root):
    a slot sees itself and its ancestors."""
    out = np.zeros((len(parents), words), dtype=np.uint32)
    for i, p in enumerate(parents):
        if p >= 0:
            out[i] = out[p]
        out[i, i >> 5] |= np.uint32(1 << (i & 31))
    return out


def visible(base, pos, mask_row):
    """Ascending positions that a token at `pos` with this mask row sees."""
    seen = list(range(min(base, pos + 1)))
    for i in range(32 * len(mask_row)):
        if (int(mask_row[i >> 5]) >> (i & 31)) & 1 and base + i <= pos:
            seen.append(base + i)
    return np.asarray(seen, dtype=np.int64)


def dense_mla(q_tok, lat, sm_scale):
    """out [96, 512], lse [96], and A [96, 512] = sum_s p(s) |v(s)|, the scale of the
    error that a relative error of the weights makes.  No latents: zeros, -inf."""
    q = O.decode_bf16(np.asarray(q_tok)).reshape(O.H_MLA, O.D_LAT)
    if lat.shape[0] == 0:
        z = np.zeros((O.H_MLA, O.D_V))
        return z, np.full(O.H_MLA, -np.inf), z
    logits = sm_scale * (q @ lat.T)
    m = logits.max(axis=1, keepdims=True)
    e = np.exp(logits - m)
    l = e.sum(axis=1, keepdims=True)
    p = e / l
    v = lat[:, :O.D_V]
    return p @ v, (m + np.log(l))[:, 0], p @ np.abs(v)


def tree_topk(scores, seen, k):
    """The k best of scores[seen], equal scores by lower position; ascending, -1 behind."""
    out = np.full(k, -1, dtype=np.int64)
    best = seen[np.lexsort((seen, -scores[seen].astype(np.float64)))[:k]]
    out[:best.size] = np.sort(best)
    return out


# ------------------------------------------------------------ rows of the cache

def _record(rows, layout, bt_row, s):
    """The three byte ranges of position s: (row, offset, length)."""
    bs, slot = layout.bs, s % layout.bs
    row = int(bt_row[s // bs])
    codes = 128 if layout.idx_fmt == O.IDX_FP8 else 64
    lat = 576 if layout.lat_fmt == O.LAT_FP8 else 352
    return [(row, layout.idx_off + slot * codes, codes), (row, layout.idx_off + bs * codes + slot * 4, 4),
            (row, layout.lat_off + slot * lat, lat)]


class CacheLayout:
    """Where a position's bytes lie in a row of the packed pool."""

    def __init__(self, bs, idx_off, lat_off, idx_fmt, lat_fmt):
        self.bs, self.idx_off, self.lat_off, self.idx_fmt, self.lat_fmt = bs, idx_off, lat_off, idx_fmt, lat_fmt


def commit(pool2d, layout, block_table, base, ctx, accept):
    """New pool and committed lengths after every request keeps its accepted slots (a
    request whose row is not ascending inside its draft keeps its pool and length -1)."""
    out = pool2d.copy()
    lens = []
    for r in range(len(base)):
        path = []
        for a in accept[r]:
            if a < 0:
                break
            path.append(int(a))
        if any(b <= a for a, b in zip(path, path[1:])) or any(base[r] + a >= ctx[r] for a in path):
            lens.append(-1)
            continue
        for i, a in enumerate(path):
            for (rs, os, n), (rd, od, _) in zip(_record(pool2d, layout, block_table[r], base[r] + a),
                                                _record(pool2d, layout, block_table[r], base[r] + i)):
                out[rd, od:od + n] = pool2d[rs, os:os + n]
        lens.append(int(base[r]) + len(path))
    return out, lens


class Pages:
    """Reference counts, tables and lengths as plain lists."""

    def __init__(self, ref, table, ctx, bs):
        self.ref, self.table, self.ctx, self.bs = [int(v) for v in ref], [[int(v) for v in r] for r in table], \
            [int(v) for v in ctx], bs

    def free(self, reqs):
        bad = False
        for r in reqs:
            if r < 0:
                continue
            if r >= len(self.ctx):
                bad = True
                continue
            for e, b in enumerate(self.table[r]):
                if b < 0:
                    continue
                self.table[r][e] = -1
                if b >= len(self.ref) or self.ref[b] <= 0:
                    bad = True
                else:
                    self.ref[b] -= 1
            self.ctx[r] = 0
        return bad

    def fork(self, parent, child):
        """Pairs (src, dst) and whether any fork was left out."""
        bad = False
        named = [c for p, c in zip(parent, child) if p >= 0]
        parents = {p for p in parent if p >= 0}
        free = [i for i, v in enumerate(self.ref) if v <= 0]
        pairs, made, at = [], [], 0
        for p, c in zip(parent, child):
            pairs.append((-1, -1))
            if p < 0:
                continue
            n = len(self.ctx)
            ok = p < n and 0 <= c < n and named.count(c) == 1 and c not in parents and self.ctx[c] == 0
            if ok and self.ctx[p] % self.bs:
                at += 1
                if at > len(free):
                    ok = False
                else:
                    pairs[-1] = (self.table[p][self.ctx[p] // self.bs], free[at - 1])
            if not ok:
                bad = True
                continue
            made.append((p, c, pairs[-1][1]))
        for p, c, new in made:
            full = self.ctx[p] // self.bs
            for b in self.table[p][:full]:
                self.ref[b] += 1
            row = self.table[p][:full] + ([new] if new >= 0 else [])
            if new >= 0:
                self.ref[new] = 1
            self.table[c] = row + [-1] * (len(self.table[c]) - len(row))
            self.ctx[c] = self.ctx[p]
        return pairs, bad

    def compact(self):
        """(L, moves): the counts and tables follow; moves are (src, dst) pairs."""
        L = sum(1 for v in self.ref if v > 0)
        holes = [i for i in range(L) if self.ref[i] <= 0]
        movers = [i for i in range(L, len(self.ref)) if self.ref[i] > 0]
        to = {i: i for i, v in enumerate(self.ref) if v > 0}
        for s, d in zip(movers, holes):
            to[s] = d
            self.ref[d], self.ref[s] = self.ref[s], 0
        self.ref = [max(v, 0) for v in self.ref]
        self.table = [[to.get(b, -1) if b >= 0 else -1 for b in row] for row in self.table]
        return L, list(zip(movers, holes))
