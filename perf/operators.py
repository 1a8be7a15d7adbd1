"""The operators of speculative decoding over the packed cache, as they are measured.

Five operators, each in its plain form (elementary torch operations) and as the
calls that a program makes of the library:

  tree_mla   attention of a tree of drafted tokens over the paged latents: token t
             sees the committed positions of its request and its ancestors among
             the drafted slots
  tree_topk  the exact top-k of a drafted token's indexer scores over the same
             visible positions (ties to the lower position)
  commit     the accepted path of each tree moved to the positions behind the
             committed context (index key, key scale and latent of every token)
  fork       free the losing branches, fork the winners: full blocks shared by
             reference count, the last partial block copied to a free row
  compact    live rows of a pool moved into the holes below them, block tables and
             reference counts following

Sizes depend on the case alone, values on the seed.  Rows of the pool are
[index page | latent page] with blocks of `bs` tokens: FP8 keys 128 + 4 bytes a
token; FP8 latents 576 bytes, NVFP4 latents 352 bytes a token.
"""
import math

import torch

own = False

HEADS, LAT, VDIM, TOPK = 96, 576, 512, 2048
SCALE = 1.0 / 24.0
MAX_PAIRS = 7.0e6           # largest sum of (drafted tokens x context) of a drawn attention case


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the first drafted token of one short conversation: latency alone
        dict(name="tree_mla_b1_n1_1k", op="tree_mla", reqs=1, n=1, fan=1, lo=1001, hi=1001, fmt="fp8", bs=64),
        # the decode batch of 8 x 64K with six tokens to verify for each request (1 + 5 drafted)
        dict(name="tree_mla_b8_n6_64k", op="tree_mla", reqs=8, n=6, fan=2, lo=65530, hi=65530, fmt="fp8", bs=64),
        # a wide tree over one long context in NVFP4 latents
        dict(name="tree_mla_nvfp4_b1_n16_256k", op="tree_mla", reqs=1, n=16, fan=3, lo=262143, hi=262143, fmt="nvfp4",
             bs=64),
        # a serving batch: ragged contexts and ragged trees
        dict(name="tree_mla_b32_n12_ragged", op="tree_mla", reqs=32, n=12, fan=3, lo=4099, hi=131071, fmt="fp8", bs=64),
        # selection for the drafted tokens of the same decode batch (rows within one launch's reach)
        dict(name="tree_topk_b8_n6_64k", op="tree_topk", reqs=8, n=6, fan=2, lo=65530, hi=65530, bs=64),
        # and for a wide tree at a context of a million tokens
        dict(name="tree_topk_b1_n16_1m", op="tree_topk", reqs=1, n=16, fan=3, lo=1048560, hi=1048560, bs=64),
        # one conversation keeps three of eight drafted tokens: latency alone
        dict(name="commit_b1_n8", op="commit", reqs=1, n=24, acc=3, lo=1001, hi=1001, bs=64),
        # a large batch keeps what its trees' verification accepted, none to eight tokens each
        dict(name="commit_b256_n32", op="commit", reqs=256, n=32, acc=8, lo=500, hi=1501, bs=64),
        # eight beams restart from two parents
        dict(name="fork_p2_c8", op="fork", parents=2, kids=4, lo=1001, hi=4001, bs=64),
        # parallel sampling: every prompt of a batch forked into eight continuations
        dict(name="fork_p32_c256", op="fork", parents=32, kids=8, lo=2047, hi=40001, bs=64),
        # a small pool tidied between batches
        dict(name="compact_600", op="compact", rows=600, dead=0.25, reqs=16, bs=64),
        # a 1.1 GB pool with a third of its rows freed
        dict(name="compact_24k", op="compact", rows=24000, dead=0.33, reqs=64, bs=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree_mla", "tree_mla", "tree_topk", "commit", "fork", "compact"])
    bs = rng.choice([16, 32, 64, 64, 128, 256])
    if op in ("tree_mla", "tree_topk"):
        while True:
            c = dict(op=op, reqs=_log_int(rng, 1, 48), n=_log_int(rng, 1, 64), fan=rng.choice([1, 2, 3, 5]),
                     lo=_log_int(rng, 1, 200000), bs=bs)
            c["hi"] = max(c["lo"], _log_int(rng, c["lo"], 1000000 if op == "tree_topk" else 262144))
            if op == "tree_mla":
                c["fmt"] = rng.choice(["fp8", "fp8", "nvfp4"])
            ln, nd = _lens(c), _drafts(c)
            pairs = sum(a * b for a, b in zip(ln, nd))
            cells = sum(nd) * max(ln)
            if op == "tree_mla" and pairs <= MAX_PAIRS and sum(ln) <= 1.1e6 and sum(nd) <= 512:
                return c
            if op == "tree_topk" and cells <= 16.5e6:
                return c
    if op == "commit":
        lo = _log_int(rng, 1, 1200)
        acc = rng.randint(1, 8)
        return dict(op=op, reqs=_log_int(rng, 1, 256), n=acc * rng.randint(2, 4) + 1, acc=acc, lo=lo,
                    hi=rng.randint(lo, 1500), bs=bs)
    if op == "fork":
        lo, bs = _log_int(rng, 1, 20000), rng.choice([32, 64, 128])
        return dict(op=op, parents=_log_int(rng, 1, 32), kids=_log_int(rng, 1, 512 // max(bs, 64)), lo=lo,
                    hi=_log_int(rng, lo, 36000), bs=bs)
    rows = _log_int(rng, 64, 24000)
    return dict(op=op, rows=rows * 64 // max(bs, 64), dead=round(rng.uniform(0.02, 0.33), 3),
                reqs=_log_int(rng, 1, 64), bs=bs)


# ------------------------------------------------- sizes, from the case alone

def _lens(case):
    """Committed context of each request: spread over the logarithm, odd steps."""
    b, lo, hi = case.get("reqs", case.get("parents")), case["lo"], case["hi"]
    if b == 1:
        return [hi]
    out = []
    for i in range(b):
        j = (i * 7) % b                      # not in order of length
        out.append(max(1, int(round(lo * (hi / lo) ** (j / (b - 1))))))
    return out


def _drafts(case):
    """Drafted tokens of each request: all `n` where the contexts are equal, ragged otherwise."""
    b, n = case["reqs"], case["n"]
    if case["lo"] == case["hi"]:
        return [n] * b
    return [1 + (i * 5 + n - 1) % n for i in range(b)]


def _ancestors(n, fan):
    """For each drafted slot the list of slots it sees: its path to the root, itself included."""
    seen = []
    for i in range(n):
        seen.append([i] if i == 0 else seen[(i - 1) // fan] + [i])
    return seen


def _accepted(case, i):
    """Accepted drafted slots of request i, ascending.  They lie behind the first `acc` slots,
    so that a pass on moved data reads what the pass before read."""
    acc, n = case["acc"], case["n"]
    take = acc if case["reqs"] == 1 else (i * 5) % (acc + 1)
    step = max(1, (n - acc) // acc)
    return [acc + j * step for j in range(take)]


def _row_bytes(bs, fmt="fp8"):
    return bs * 132 + bs * (576 if fmt == "fp8" else 352)


def _moves(case):
    dead = int(case["rows"] * case["dead"])
    return dead, int(dead * (1.0 - case["dead"]))     # expected holes below the live count


def work(case):
    op, bs = case["op"], case["bs"]
    if op in ("tree_mla", "tree_topk"):
        ln, nd = _lens(case), _drafts(case)
        anc = [len(a) for a in _ancestors(max(nd), case["fan"])]
        vis = sum(n * L + sum(anc[:n]) for L, n in zip(ln, nd))
        t = sum(nd)
        words = (max(nd) + 31) // 32
        small = t * (8 + 4 * words) + len(ln) * 8
        if op == "tree_mla":
            tok = 576 if case["fmt"] == "fp8" else 324
            kv = sum((L + n) * tok + -(-(L + n) // bs) * 4 for L, n in zip(ln, nd))
            return dict(bytes=kv + t * HEADS * (LAT * 2 + VDIM * 2 + 4) + small, flops=2 * HEADS * (LAT + VDIM) * vis)
        return dict(bytes=vis * 4 + t * TOPK * 4 + small, flops=vis)
    if op == "commit":
        k = sum(len(_accepted(case, i)) for i in range(case["reqs"]))
        return dict(bytes=k * (2 * 708 + 12) + case["reqs"] * 12, flops=0)
    if op == "fork":
        ln = _lens(case)
        kids = case["kids"]
        blocks = sum(-(-L // bs) for L in ln)
        part = sum(1 for L in ln if L % bs) * kids
        # tables: the parents' rows once, the children's rows written, counts of the shared blocks; rows copied
        return dict(bytes=blocks * 4 + blocks * kids * 4 + blocks * 8 + part * 2 * _row_bytes(bs), flops=0)
    dead, moves = _moves(case)
    return dict(bytes=case["rows"] * 8 + 2 * 4 * (case["rows"] - dead) + moves * 2 * _row_bytes(bs), flops=0)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _e4m3(shape, g, lim=448.0):
    return torch.randn(shape, generator=g, device="cuda").clamp_(-lim, lim).to(torch.float8_e4m3fn).view(torch.uint8)


_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nvfp4(n, g):
    """n NVFP4 latent records of 352 bytes from N(0, 1)."""
    x = torch.randn((n, 36, 16), generator=g, device="cuda")
    sc = (x.abs().amax(2) / 6.0).to(torch.float8_e4m3fn)
    y = x / sc.float().clamp_min(1e-3)[:, :, None]
    mid = torch.tensor([(a + b) / 2 for a, b in zip(_GRID, _GRID[1:])], device="cuda")
    code = torch.bucketize(y.abs(), mid).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    code = code.view(n, 288, 2)
    rec = torch.zeros((n, 352), dtype=torch.uint8, device="cuda")
    rec[:, :288] = code[:, :, 0] | (code[:, :, 1] << 4)
    rec[:, 288:324] = sc.view(torch.uint8)
    return rec


def _latent_pool(rows, bs, fmt, g):
    """A pool with latents in every row (index pages of zero bytes: this operator reads none)."""
    rb = _row_bytes(bs, fmt)
    pool = torch.zeros((rows, rb), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 17) // bs)
    for r in range(0, rows, step):
        k = min(step, rows - r)
        lat = _e4m3((k * bs, 576), g) if fmt == "fp8" else _nvfp4(k * bs, g)
        pool[r:r + k, bs * 132:] = lat.view(k, -1)
    return pool


def _tables(lens, bs, rows, g):
    """Block table of requests with `lens` tokens over a permutation of the pool's rows."""
    blocks = [-(-L // bs) for L in lens]
    perm = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(lens), max(blocks) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, nb in enumerate(blocks):
        bt[i, :nb] = perm[at:at + nb]
        at += nb
    return bt


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tree_inputs(case):
    ln, nd = _lens(case), _drafts(case)
    words = (max(nd) + 31) // 32
    anc = _ancestors(max(nd), case["fan"])
    rows = []
    for i in range(max(nd)):
        w = [0] * words
        for a in anc[i]:
            w[a >> 5] |= 1 << (a & 31)
        rows.append([v - (1 << 32) if v >= 1 << 31 else v for v in w])
    mask = [rows[j] for n in nd for j in range(n)]
    return dict(lens=ln, drafts=nd, base=_i32(ln), ctx=_i32([a + b for a, b in zip(ln, nd)]), mask=_i32(mask),
                q_req=_i32([i for i, n in enumerate(nd) for _ in range(n)]),
                q_pos=_i32([L + j for L, n in zip(ln, nd) for j in range(n)]))


def prepare(case, seed):
    g = _gen(seed)
    op, bs = case["op"], case["bs"]
    st = dict(case=case, op=op, bs=bs)
    if op in ("tree_mla", "tree_topk"):
        st.update(_tree_inputs(case))
        total = [a + b for a, b in zip(st["lens"], st["drafts"])]
        rows = sum(-(-L // bs) for L in total) + 3
        st["bt"] = _tables(total, bs, rows, g)
        t = sum(st["drafts"])
        if op == "tree_mla":
            st["fmt"] = case["fmt"]
            st["pool"] = _latent_pool(rows, bs, case["fmt"], g)
            st["q"] = torch.randn((t, HEADS, LAT), generator=g, device="cuda").to(torch.bfloat16)
        else:
            st["fmt"], st["rows"] = "fp8", rows
            ld = (max(total) + 3) // 4 * 4
            st["scores"] = torch.randn((t, ld), generator=g, device="cuda")
    elif op == "commit":
        lens = _lens(case)
        total = [L + case["n"] for L in lens]
        rows = sum(-(-L // bs) for L in total) + 3
        st["bt"] = _tables(total, bs, rows, g)
        st["pool"] = torch.randint(0, 256, (rows, _row_bytes(bs)), generator=g, device="cuda", dtype=torch.uint8)
        st["base"], st["ctx"] = _i32(lens), _i32(total)
        acc = [_accepted(case, i) for i in range(case["reqs"])]
        st["accept"] = _i32([a + [-1] * (case["acc"] - len(a)) for a in acc])
    elif op == "fork":
        lens, kids = _lens(case), case["kids"]
        p = len(lens)
        rows = sum(-(-L // bs) for L in lens) + p * kids + 5
        st["bt"] = torch.full((p * (kids + 1), max(-(-L // bs) for L in lens) + 1), -1, dtype=torch.int32, device="cuda")
        st["bt"][:p] = _tables(lens, bs, rows, g)
        st["ctx"] = _i32(lens + [0] * (p * kids))
        st["ref"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        ids = st["bt"][:p].flatten()
        st["ref"][ids[ids >= 0].long()] = 1
        st["pool"] = torch.randint(0, 256, (rows, _row_bytes(bs)), generator=g, device="cuda", dtype=torch.uint8)
        st["parent"] = _i32([i % p for i in range(p * kids)])
        st["child"] = _i32([p + i for i in range(p * kids)])
        _plain_fork(st)                      # the branches that the pass finds and drops
    else:
        rows, reqs = case["rows"], case["reqs"]
        dead, _ = _moves(case)
        perm = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)[:rows - dead]
        per = -(-perm.numel() // reqs)
        bt = torch.full((reqs + 1, per + 1), -1, dtype=torch.int32, device="cuda")
        for i in range(reqs):
            part = perm[i * per:(i + 1) * per]
            bt[i, :part.numel()] = part
        bt[reqs] = bt[0]                     # a fork of the first request shares its blocks
        ids = bt.flatten()
        st["bt"], st["ref"] = bt, torch.bincount(ids[ids >= 0].long(), minlength=rows).to(torch.int32)
        st["pool"] = torch.randint(0, 256, (rows, _row_bytes(bs)), generator=g, device="cuda", dtype=torch.uint8)
        st["ctx"] = (bt >= 0).sum(1).to(torch.int32) * bs
    if own:
        _prepare_own(st)
    return st


# --------------------------------------------------------------- plain forms

def _visible(st, t0, n, base, total):
    """[n, total] truth values: what the drafted tokens t0 .. t0 + n - 1 of one request see."""
    s = torch.arange(total, device="cuda")
    d = (s - base).clamp_min(0)
    words = st["mask"][t0:t0 + n].long() & 0xFFFFFFFF
    w = torch.clamp(d >> 5, max=words.shape[1] - 1)
    bit = (words[:, w] >> (d & 31)) & 1
    return ((s < base) | (bit != 0)) & (s <= st["q_pos"][t0:t0 + n].long()[:, None])


def _latents(st, i, total):
    """fp32 [total, 576]: the dequantised latents of request i."""
    bs = st["bs"]
    nb = -(-total // bs)
    rows = st["pool"][st["bt"][i, :nb].long(), bs * 132:].reshape(nb * bs, -1)[:total]
    if st["fmt"] == "fp8":
        return rows.contiguous().view(torch.float8_e4m3fn).float()
    code = torch.stack((rows[:, :288] & 15, rows[:, :288] >> 4), 2).reshape(total, 576).long()
    grid = torch.tensor(_GRID + [-v for v in _GRID], device="cuda")
    scale = rows[:, 288:324].contiguous().view(torch.float8_e4m3fn).float()
    return (grid[code].view(total, 36, 16) * scale[:, :, None]).view(total, 576)


def _plain_tree_mla(st):
    outs, lses, t0 = [], [], 0
    for i, (L, n) in enumerate(zip(st["lens"], st["drafts"])):
        c = _latents(st, i, L + n)
        q = st["q"][t0:t0 + n].float().view(n * HEADS, LAT)
        s = (q @ c.t()).view(n, HEADS, -1) * SCALE
        s = s.masked_fill(~_visible(st, t0, n, L, L + n)[:, None, :], float("-inf"))
        m = s.amax(2, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(2)
        o = (p.view(n * HEADS, -1) @ c[:, :VDIM]).view(n, HEADS, VDIM) / z[:, :, None]
        outs.append(o.to(torch.bfloat16))
        lses.append(m[:, :, 0] + torch.log(z))
        t0 += n
    return torch.cat(outs), torch.cat(lses)


def _plain_tree_topk(st):
    outs, t0 = [], 0
    for L, n in zip(st["lens"], st["drafts"]):
        vis = _visible(st, t0, n, L, L + n)
        s = st["scores"][t0:t0 + n, :L + n].masked_fill(~vis, float("-inf"))
        k = min(TOPK, L + n)
        order = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :k]
        # visible positions come first (finite scores); what is left over sorts behind every position
        order = torch.where(torch.gather(vis, 1, order), order, 1 << 40).sort(1).values
        idx = torch.full((n, TOPK), -1, dtype=torch.int32, device="cuda")
        idx[:, :k] = torch.where(order < (1 << 40), order, -1).to(torch.int32)
        outs.append(idx)
        t0 += n
    return torch.cat(outs)


def _plain_commit(st):
    bs, pool, acc = st["bs"], st["pool"], st["accept"].long()
    ok = acc >= 0
    req = torch.arange(acc.shape[0], device="cuda")[:, None].expand_as(acc)[ok]
    base = st["base"].long()[req]
    src = base + acc[ok]
    dst = base + torch.arange(acc.shape[1], device="cuda").expand_as(acc)[ok]

    def cells(pos):
        slot = (pos % bs)[:, None]
        off = torch.cat((slot * 128 + torch.arange(128, device="cuda"), bs * 128 + slot * 4 + torch.arange(4, device="cuda"),
                         bs * 132 + slot * 576 + torch.arange(576, device="cuda")), 1)
        return st["bt"][req, pos // bs].long()[:, None], off

    r, o = cells(src)
    rec = pool[r, o]
    r, o = cells(dst)
    pool[r, o] = rec
    return pool, (st["base"] + ok.sum(1)).to(torch.int32)


def _plain_fork(st):
    bs, bt, ref, ctx, pool = st["bs"], st["bt"], st["ref"], st["ctx"], st["pool"]
    parent, child = st["parent"].long(), st["child"].long()
    old = bt[child]                                           # free the branches
    ref.index_add_(0, old.clamp_min(0).flatten().long(), -(old >= 0).flatten().to(torch.int32))
    lens = ctx[parent].long()                                 # fork
    full, part = lens // bs, lens % bs != 0
    rank = torch.cumsum(part, 0)
    new = torch.searchsorted(torch.cumsum(ref == 0, 0), rank).clamp_max(ref.numel() - 1)
    rows = bt[parent]
    col = torch.arange(bt.shape[1], device="cuda")[None]
    share = col < full[:, None]
    ref.index_add_(0, rows.clamp_min(0).flatten().long(), share.flatten().to(torch.int32))
    ref.index_add_(0, new, part.to(torch.int32))
    last = part[:, None] & (col == full[:, None])
    bt[child] = torch.where(share, rows, torch.where(last, new.to(torch.int32)[:, None], -1))
    ctx[child] = lens.to(torch.int32)
    tail = torch.gather(rows, 1, full[:, None])[:, 0]         # the partial block of each parent
    src = torch.where(part, tail, -1)
    dst = torch.where(part, new.to(torch.int32), -1)
    keep = part.nonzero()[:, 0]
    pool[dst[keep].long()] = pool[src[keep].long()]
    return bt, ref, ctx, pool, src, dst


def _plain_compact(st):
    ref, bt, pool = st["ref"], st["bt"], st["pool"]
    rows = ref.numel()
    live = ref > 0
    n_live = live.sum()
    r = torch.arange(rows, device="cuda")
    holes = (~live & (r < n_live)).nonzero()[:, 0]
    movers = (live & (r >= n_live)).nonzero()[:, 0]
    m = holes.numel()
    to = torch.where(live, r, -1)
    to[movers] = holes
    out_ref = torch.where(live & (r < n_live), ref, 0)
    out_ref[holes] = ref[movers]
    out_bt = torch.where(bt >= 0, to[bt.clamp_min(0).long()], -1).to(torch.int32)
    src = torch.full((rows // 2,), -1, dtype=torch.int32, device="cuda")
    dst = torch.full((rows // 2,), -1, dtype=torch.int32, device="cuda")
    src[:m], dst[:m] = movers.to(torch.int32), holes.to(torch.int32)
    pool[holes] = pool[movers]
    return out_bt, out_ref, torch.stack((n_live, torch.tensor(m, device="cuda"))).to(torch.int32), src, dst, pool


# ------------------------------------------------------- the library's calls

def _prepare_own(st):
    import dsa_sparse_attention_gb300 as dsa
    st["dsa"] = dsa
    op, bs = st["op"], st["bs"]
    fmt = dsa.DSA_LAT_NVFP4 if st.get("fmt") == "nvfp4" else dsa.DSA_LAT_FP8
    rb = _row_bytes(bs, st.get("fmt", "fp8"))
    pool = st.get("pool")
    rows = pool.shape[0] if pool is not None else st["rows"]
    st["layout"] = dsa.make_layout(pool, rows, rb, 0, bs * 132, bs, dsa.DSA_IDX_FP8, fmt)
    new = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda")
    if op in ("tree_mla", "tree_topk"):
        t = st["q_req"].numel()
        longest = max(a + b for a, b in zip(st["lens"], st["drafts"]))
        st["batch"] = dsa.make_batch(st["q_req"], st["q_pos"], st["ctx"], st["bt"], longest)
        st["tree"] = dsa.make_tree(st["base"], st["mask"])
        if op == "tree_mla":
            st["ws"] = dsa.alloc_tree_workspace(st["layout"], st["batch"])
            st["out"] = new(t, HEADS, VDIM, dtype=torch.bfloat16)
            st["lse"] = new(t, HEADS, dtype=torch.float32)
        else:
            st["ws"] = dsa.alloc_workspace(st["layout"], st["batch"], TOPK)
            st["idx"] = new(t, TOPK)
    elif op == "commit":
        none = torch.empty(0, dtype=torch.int32, device="cuda")
        st["batch"] = dsa.make_batch(none, none, st["ctx"], st["bt"], int(st["ctx"].max()))
        st["new_lens"] = new(st["base"].numel())
    else:
        st["pages"] = dsa.make_pages(st["ref"], st["bt"], st["ctx"])
        n = st["child"].numel() if op == "fork" else rows // 2
        st["src"], st["dst"] = new(n), new(n)
        if op == "compact":
            st["bt2"], st["ref2"], st["counts"] = torch.empty_like(st["bt"]), torch.empty_like(st["ref"]), new(2)
            st["pages2"] = dsa.make_pages(st["ref2"], st["bt2"], st["ctx"])
    if "ws" not in st:
        st["ws"] = dsa.alloc_cache_workspace(st["layout"], st["bt"].shape[0])


def _run_own(st):
    dsa, op, lay, ws = st["dsa"], st["op"], st["layout"], st["ws"]
    if op == "tree_mla":
        dsa.dsa_tree_mla(lay, st["batch"], st["tree"], st["q"], SCALE, st["out"], st["lse"], ws=ws)
        return st["out"], st["lse"]
    if op == "tree_topk":
        dsa.dsa_tree_topk(lay, st["batch"], st["tree"], st["scores"], st["scores"].shape[1], TOPK, st["idx"], ws=ws)
        return st["idx"]
    if op == "commit":
        dsa.dsa_tree_commit(lay, st["batch"], st["base"], st["accept"], st["new_lens"], ws=ws)
        return st["pool"], st["new_lens"]
    if op == "fork":
        dsa.dsa_cache_free(lay, st["pages"], st["child"], ws=ws)
        dsa.dsa_cache_fork(lay, st["pages"], st["parent"], st["child"], st["src"], st["dst"], ws=ws)
        dsa.dsa_cache_copy(lay, st["src"], st["dst"], ws=ws)
        return st["bt"], st["ref"], st["ctx"], st["pool"], st["src"], st["dst"]
    dsa.dsa_cache_compact(lay, st["pages"], st["pages2"], st["src"], st["dst"], st["counts"], ws=ws)
    dsa.dsa_cache_copy(lay, st["src"], st["dst"], st["counts"][1:], ws=ws)
    return st["bt2"], st["ref2"], st["counts"], st["src"], st["dst"], st["pool"]


def run(state):
    if own:
        return _run_own(state)
    return {"tree_mla": _plain_tree_mla, "tree_topk": _plain_tree_topk, "commit": _plain_commit, "fork": _plain_fork,
            "compact": _plain_compact}[state["op"]](state)


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    """What run returns, from the definitions.  The attention sums over each token's own list of
    visible positions in float64; the integer operators walk their lists on the host."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, bs = case["op"], case["bs"]
    if op == "tree_mla":
        grid = torch.tensor(_GRID + [-v for v in _GRID], dtype=torch.float64, device="cuda")
        codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        anc = _ancestors(max(st["drafts"]), case["fan"])
        outs, lses, t = [], [], 0
        for i, (L, n) in enumerate(zip(st["lens"], st["drafts"])):
            pos = torch.arange(L + n, device="cuda")
            rec = st["pool"][:, bs * 132:].reshape(st["pool"].shape[0], bs, -1)[st["bt"][i].long()[pos // bs], pos % bs]
            if case["fmt"] == "fp8":
                c = codes[rec.int()]
            else:
                v = torch.empty((L + n, 576), dtype=torch.float64, device="cuda")
                v[:, 0::2], v[:, 1::2] = grid[(rec[:, :288] % 16).int()], grid[(rec[:, :288] // 16).int()]
                c = v * codes[rec[:, 288:324].int()].repeat_interleave(16, 1)
            for j in range(n):
                drafted = torch.tensor([L + a for a in anc[j]], device="cuda")
                dots = torch.cat((c[:L], c[drafted]), 0) @ st["q"][t].double().t() * SCALE      # [visible, 96]
                lse = torch.logsumexp(dots, 0)
                w = torch.exp(dots - lse)
                outs.append(w[:L].t() @ c[:L, :VDIM] + w[L:].t() @ c[drafted, :VDIM])
                lses.append(lse)
                t += 1
        return torch.stack(outs), torch.stack(lses)
    if op == "tree_topk":
        import numpy as np
        anc = _ancestors(max(st["drafts"]), case["fan"])
        scores = st["scores"].cpu().numpy()
        out = np.full((scores.shape[0], TOPK), -1, np.int32)
        t = 0
        for L, n in zip(st["lens"], st["drafts"]):
            for j in range(n):
                vis = np.concatenate((np.arange(L), np.asarray(anc[j]) + L))
                best = vis[np.lexsort((vis, -scores[t, vis].astype(np.float64)))[:TOPK]]
                out[t, :best.size] = np.sort(best)
                t += 1
        return torch.from_numpy(out)
    if op == "commit":
        pool, bt = st["pool"].cpu(), st["bt"].cpu()
        start = pool.clone()
        lens = []
        for i, L in enumerate(_lens(case)):
            path = _accepted(case, i)
            for j, a in enumerate(path):
                (rs, ss), (rd, sd) = [(int(bt[i, p // bs]), p % bs) for p in (L + a, L + j)]
                for at, w in ((0, 128), (bs * 128, 4), (bs * 132, 576)):
                    pool[rd, at + sd * w:at + (sd + 1) * w] = start[rs, at + ss * w:at + (ss + 1) * w]
            lens.append(L + len(path))
        return pool, torch.tensor(lens, dtype=torch.int32)
    if op == "fork":
        bt, ref, ctx, pool = (st[k].cpu() for k in ("bt", "ref", "ctx", "pool"))
        kids = list(zip(st["parent"].tolist(), st["child"].tolist()))
        count = ref.tolist()
        for _, c in kids:
            for b in bt[c].tolist():
                if b >= 0:
                    count[b] -= 1
        free = iter([r for r, v in enumerate(count) if v == 0])
        src, dst = [], []
        for p, c in kids:
            L = int(ctx[p])
            row = bt[p, :L // bs].tolist()
            for b in row:
                count[b] += 1
            pair = (-1, -1)
            if L % bs:
                pair = (int(bt[p, L // bs]), next(free))
                count[pair[1]] = 1
                pool[pair[1]] = pool[pair[0]]
                row.append(pair[1])
            bt[c] = torch.tensor(row + [-1] * (bt.shape[1] - len(row)), dtype=torch.int32)
            ctx[c] = L
            src.append(pair[0])
            dst.append(pair[1])
        return (bt, torch.tensor(count, dtype=torch.int32), ctx, pool, torch.tensor(src, dtype=torch.int32),
                torch.tensor(dst, dtype=torch.int32))
    ref, bt, pool = st["ref"].tolist(), st["bt"].cpu(), st["pool"].cpu()
    n_live = sum(1 for v in ref if v > 0)
    holes = [r for r in range(n_live) if ref[r] == 0]
    movers = [r for r in range(n_live, len(ref)) if ref[r] > 0]
    to = list(range(len(ref))) + [-1]                         # entry -1 stays -1
    for h, s in zip(holes, movers):
        to[s] = h
        ref[h], ref[s] = ref[s], 0
        pool[h] = pool[s]
    pad = [-1] * (len(ref) // 2 - len(holes))
    out_bt = torch.tensor([[to[b] for b in row] for row in bt.tolist()], dtype=torch.int32)
    as32 = lambda v: torch.tensor(v, dtype=torch.int32)
    return out_bt, as32(ref), as32([n_live, len(holes)]), as32(movers + pad), as32(holes + pad), pool
