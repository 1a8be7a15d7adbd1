"""The operators of prompts over the packed cache, as they are measured.

Three operators, each in its plain form (elementary torch operations) and as the
calls that a program makes of the library:

  attn    attention of packed sequences with the heads' own keys and values: causal or
          over all keys, query heads in groups that share a key head, 64 of the key's
          dims optionally shared by all heads, optionally joined with an earlier result
          (out, lse) over other keys of the same sequences
  append  new tokens' index keys and latents quantised into the pages of the cache, and
          their values read back
  read    the values of whole contexts read back from the pages into packed rows

Sizes depend on the case alone, values on the seed.  Rows of the pool are
[index page | latent page] with blocks of `bs` tokens.  FP8: 128 e4m3 codes and an fp32
scale a key, 576 e4m3 codes a latent.  FP4: MXFP4 keys (64 bytes of e2m1, an E8M0
exponent per 32 dims), NVFP4 latents (288 bytes of e2m1, an e4m3 scale per 16 dims, 28
bytes of padding).
"""
import math

import torch

own = False

KEY, LAT = 128, 576
MAX_FLOPS = 2.0e12          # of a drawn attention case
MAX_BYTES = 1.5e9           # of any drawn case


# ------------------------------------------------------------------ the cases

def listed():
    mla = dict(heads=96, kv=96, dim=128, shared=64, dt="bf16")     # per-head form of the 576-dim latents
    return [
        # a short question: latency alone
        dict(name="attn_b1_33", op="attn", reqs=1, new_lo=33, new=33, ctx_lo=0, ctx=0, causal=True, join=False, **mla),
        # a prompt at the limit below which every token is selected (top-k 2,048)
        dict(name="attn_b1_2048", op="attn", reqs=1, new_lo=2048, new=2048, ctx_lo=0, ctx=0, causal=True, join=False, **mla),
        # a prefill chunk of 8,192 tokens
        dict(name="attn_b1_8192", op="attn", reqs=1, new_lo=8192, new=8192, ctx_lo=0, ctx=0, causal=True, join=False, **mla),
        # 500 new tokens behind a context of 64K
        dict(name="attn_b1_500_on_64k", op="attn", reqs=1, new_lo=500, new=500, ctx_lo=65536, ctx=65536, causal=True,
             join=False, **mla),
        # a serving batch of short and long prompts, grouped heads
        dict(name="attn_b32_ragged", op="attn", reqs=32, new_lo=17, new=4099, ctx_lo=0, ctx=0, causal=True, join=False,
             heads=64, kv=8, dim=128, shared=0, dt="fp16"),
        # one new token for each of 16 conversations
        dict(name="attn_b16_step", op="attn", reqs=16, new_lo=1, new=1, ctx_lo=1000, ctx=32766, causal=True, join=False,
             heads=64, kv=8, dim=128, shared=0, dt="bf16"),
        # a chunk of earlier context, joined with the result over what came before it
        dict(name="attn_b4_join", op="attn", reqs=4, new_lo=301, new=301, ctx_lo=7891, ctx=7891, causal=False, join=True,
             heads=32, kv=32, dim=64, shared=0, dt="bf16"),
        # the token of one decode step
        dict(name="append_b1_1", op="append", reqs=1, new_lo=1, new=1, ctx_lo=1000, ctx=1000, fmt="fp8", bs=64),
        # the chunks of four prompts
        dict(name="append_b4_8192_fp4", op="append", reqs=4, new_lo=2048, new=2048, ctx_lo=0, ctx=4096, fmt="fp4", bs=64),
        # one short conversation
        dict(name="read_b1_777", op="read", reqs=1, new_lo=777, new=777, ctx_lo=0, ctx=0, fmt="fp8", bs=64),
        # the contexts of the decode batch of 8 x 64K
        dict(name="read_b8_64k", op="read", reqs=8, new_lo=65536, new=65536, ctx_lo=0, ctx=0, fmt="fp8", bs=64),
        # contexts of all lengths, 4-bit pages, from the middle of a block on
        dict(name="read_b16_ragged_fp4", op="read", reqs=16, new_lo=4099, new=131071, ctx_lo=7, ctx=7, fmt="fp4", bs=64),
    ]


# (query heads, key heads, dims of a head, shared dims)
_HEADS = [(96, 96, 128, 64), (96, 96, 128, 64), (64, 8, 128, 0), (32, 32, 64, 0), (28, 4, 128, 0), (40, 8, 64, 0),
          (48, 1, 128, 64), (16, 2, 64, 64)]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "read"])
    while True:
        c = dict(op=op, reqs=_log_int(rng, 1, 48))
        if op == "attn":
            c["heads"], c["kv"], c["dim"], c["shared"] = rng.choice(_HEADS)
            c["dt"] = rng.choice(["bf16", "bf16", "fp16"])
            kind = rng.choice(["prompt", "chunk", "step", "join"])
            c["new_lo"] = 1 if kind == "step" else _log_int(rng, 1, 4000)
            c["new"] = 1 if kind == "step" else _log_int(rng, c["new_lo"], 12000)
            c["ctx_lo"] = 0 if kind == "prompt" else _log_int(rng, 1, 20000)
            c["ctx"] = 0 if kind == "prompt" else _log_int(rng, c["ctx_lo"], 66000)
            c["causal"], c["join"] = kind != "join", kind == "join"
        else:
            c["fmt"], c["bs"] = rng.choice(["fp8", "fp4"]), rng.choice([16, 32, 64, 64, 128, 256])
            most = 12000 if op == "append" else 131071
            c["new_lo"] = _log_int(rng, 1, most)
            c["new"] = _log_int(rng, c["new_lo"], most)
            c["ctx_lo"] = rng.randint(0, 3000)
            c["ctx"] = rng.randint(c["ctx_lo"], 5000)
        w = work(c)
        if w["bytes"] <= MAX_BYTES and w["flops"] <= MAX_FLOPS and w["bytes"] >= 1000:
            return c


# ------------------------------------------------- sizes, from the case alone

def _spread(lo, hi, n, step):
    """n lengths from lo to hi, even in their logarithm, not in order of length."""
    if lo == hi or n == 1:
        return [hi] * n
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * ((i * step) % n) / (n - 1)))) - 1 for i in range(n)]


def _lens(case):
    """(new tokens, tokens before them) of each sequence."""
    n = case["reqs"]
    new = [max(1, v) for v in _spread(case["new_lo"], case["new"], n, 7 if n % 7 else 5)]
    return new, _spread(case["ctx_lo"], case["ctx"], n, 11 if n % 11 else 3)


def _keys(case):
    """Keys of each sequence: context and new tokens, or the context alone where it is joined."""
    new, ctx = _lens(case)
    return [c if case["join"] else c + n for n, c in zip(new, ctx)]


def _pairs(case):
    new, _ = _lens(case)
    if not case["causal"]:
        return sum(n * k for n, k in zip(new, _keys(case)))
    return sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(new, _keys(case)))


def _sizes(fmt):
    """Bytes of a key and of a latent record as they lie in the pages."""
    return (KEY + 4, LAT) if fmt == "fp8" else (KEY // 2 + 4, 352)


def work(case):
    new, ctx = _lens(case)
    t = sum(new)
    if case["op"] == "attn":
        h, g, d, e = case["heads"], case["kv"], case["dim"], case["shared"]
        n = sum(_keys(case))
        rows = t * h * ((2 * d + e) * 2 + 4) + (t * h * (d * 2 + 4) if case["join"] else 0)
        return dict(bytes=rows + n * (g * 2 * d + e) * 2 + 8 * (len(new) + 1), flops=2 * (2 * d + e) * h * _pairs(case))
    key, lat = _sizes(case["fmt"])
    lat = min(lat, 324) if case["fmt"] == "fp4" else lat          # a reader needs no padding
    table = sum(-(-(n + c) // case["bs"]) - c // case["bs"] for n, c in zip(new, ctx)) * 4
    values = t * (KEY + LAT) * 2
    if case["op"] == "read":
        return dict(bytes=values + t * (key + lat) + table + 12 * len(new), flops=t * (KEY + LAT))
    # the new records are written from the values, and read back into others
    return dict(bytes=2 * values + t * (2 * key + lat + _sizes(case["fmt"])[1]) + t * 8 + table + 12 * len(new),
                flops=2 * t * (KEY + LAT))


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _pool(case, rows, g):
    """A pool whose pages hold records of N(0, 1) values."""
    bs, fmt = case["bs"], case["fmt"]
    key, lat = _sizes(fmt)
    pool = torch.zeros((rows, bs * (key + lat)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 16) // bs)
    for r in range(0, rows, step):
        n = min(step, rows - r) * bs
        rand = lambda hi, *shape: torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.uint8)
        if fmt == "fp8":
            e4m3 = lambda d: torch.randn((n, d), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
            scale = (torch.rand((n, 1), generator=g, device="cuda") * 1.5 + 0.5).view(torch.uint8)
            codes, scales, rec = e4m3(KEY), scale, e4m3(LAT)
        else:
            codes, scales = rand(256, n, KEY // 2), 124 + rand(5, n, 4)
            rec = torch.zeros((n, lat), dtype=torch.uint8, device="cuda")
            rec[:, :288] = rand(256, n, 288)
            rec[:, 288:324] = 32 + rand(25, n, 36)                # scales of 1/16 to 1
        part = pool[r:r + n // bs]
        part[:, :bs * codes.shape[1]] = codes.view(n // bs, -1)
        part[:, bs * codes.shape[1]:bs * key] = scales.view(n // bs, -1)
        part[:, bs * key:] = rec.view(n // bs, -1)
    return pool


def prepare(case, seed):
    g = _gen(seed)
    new, ctx = _lens(case)
    st = dict(case=case, op=case["op"], new=new, ctx=ctx)
    t = sum(new)
    if case["op"] == "attn":
        dt = torch.bfloat16 if case["dt"] == "bf16" else torch.float16
        h, kv, d, e = case["heads"], case["kv"], case["dim"], case["shared"]
        st["keys"] = _keys(case)
        n = sum(st["keys"])
        randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=dt)
        st["scale"] = 1.0 / math.sqrt(d + e)
        # keys with a spread of the logits of about 1.5 for unit queries, as trained heads have
        st["q"] = randn(t, h, d + e).mul_(1.5)
        # keys and values of a head lie side by side, as one projection of the latents writes them
        kvs = randn(n, kv, 2 * d)
        st["k"], st["v"] = kvs[:, :, :d], kvs[:, :, d:]
        st["k_shared"] = randn(n, LAT)[:, LAT - e:] if e else None     # the last dims of the latents read back
        st["cu_q"], st["cu_k"] = _i32(_cu(new)), _i32(_cu(st["keys"]))
        if case["join"]:
            st["prev_out"] = randn(t, h, d)
            st["prev_lse"] = torch.randn((t, h), generator=g, device="cuda") + 8.0
    else:
        bs = case["bs"]
        blocks = [-(-(n + c) // bs) for n, c in zip(new, ctx)]
        rows = sum(blocks) + 3
        st["pool"] = _pool(case, rows, g)
        perm = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
        st["bt"] = torch.full((len(new), max(blocks) + 1), -1, dtype=torch.int32, device="cuda")
        for i, (nb, at) in enumerate(zip(blocks, _cu(blocks))):
            st["bt"][i, :nb] = perm[at:at + nb]
        st["lens"] = _i32([n + c for n, c in zip(new, ctx)])
        st["cu"], st["start"] = _i32(_cu(new)), _i32(ctx)
        lens = torch.tensor(new, device="cuda")
        req = torch.repeat_interleave(torch.arange(len(new), device="cuda"), lens)
        st["q_req"] = req.to(torch.int32)
        st["q_pos"] = (torch.arange(t, device="cuda") - st["cu"].long()[req] + st["start"].long()[req]).to(torch.int32)
        if case["op"] == "append":
            st["k_new"] = torch.randn((t, KEY), generator=g, device="cuda").to(torch.bfloat16)
            st["latent"] = torch.randn((t, LAT), generator=g, device="cuda").to(torch.bfloat16)
    if own:
        _prepare_own(st)
    return st


# --------------------------------------------------------------- plain forms

def _plain_attn(st):
    case = st["case"]
    h, kv, d, e = case["heads"], case["kv"], case["dim"], case["shared"]
    t = sum(st["new"])
    out = torch.empty((t, h, d), dtype=st["q"].dtype, device="cuda")
    lse = torch.empty((t, h), dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for n, m in zip(st["new"], st["keys"]):
        vis = None
        if case["causal"]:
            vis = torch.arange(m, device="cuda")[None] <= torch.arange(n, device="cuda")[:, None] + (m - n)
            vis = vis.repeat_interleave(h // kv, 0)
        step = max(1, int(2 ** 29 // (n * (h // kv) * m)))           # key heads whose scores take 2 GB at most
        for a in range(0, kv, step):
            b = min(kv, a + step)
            q = st["q"][q0:q0 + n].view(n, kv, h // kv, d + e)[:, a:b].permute(1, 0, 2, 3).reshape(b - a, -1, d + e).float()
            k = st["k"][k0:k0 + m, a:b].permute(1, 2, 0).float()
            s = q[..., :d] @ k
            if e:
                s += q[..., d:] @ st["k_shared"][k0:k0 + m].t().float()
            s *= st["scale"]
            if vis is not None:
                s.masked_fill_(~vis, float("-inf"))
            top = s.amax(2, keepdim=True)
            s = s.sub_(top).exp_()
            z = s.sum(2, keepdim=True)
            o = (s @ st["v"][k0:k0 + m, a:b].permute(1, 0, 2).float()) / z
            rows = lambda x: x.view(b - a, n, h // kv, -1).permute(1, 0, 2, 3).reshape(n, (b - a) * (h // kv), -1)
            at = slice(a * (h // kv), b * (h // kv))
            o, l = rows(o), rows(top + torch.log(z))[:, :, 0]
            if case["join"]:
                both = torch.logaddexp(st["prev_lse"][q0:q0 + n, at], l)
                o = (st["prev_out"][q0:q0 + n, at].float() * torch.exp(st["prev_lse"][q0:q0 + n, at] - both)[..., None]
                     + o * torch.exp(l - both)[..., None])
                l = both
            out[q0:q0 + n, at] = o.to(out.dtype)
            lse[q0:q0 + n, at] = l
        q0, k0 = q0 + n, k0 + m
    return out, lse


def _codes4(x):
    """e2m1 codes of fp32 values: nearest, ties to the even code, at most 6."""
    grid = torch.tensor(_GRID, device="cuda")
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    up = torch.bucketize(a, mid, right=True)                         # a midpoint goes up,
    code = torch.where((up > 0) & (a == mid[(up - 1).clamp_min(0)]) & (up % 2 == 1), up - 1, up)   # or to the even code
    return code.to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)


def _pack4(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _records(k, lat, fmt):
    """(key codes, key scales, latent records) as bytes."""
    k, lat = k.float(), lat.float()
    if fmt == "fp8":
        top = k.abs().amax(1, keepdim=True)
        s = torch.where(top > 0, top / 448.0, 1.0)
        byte = lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)
        return byte(k / s), s.view(torch.uint8), byte(lat.clamp(-448, 448))
    x = k.view(-1, 4, 32)
    _, up = torch.frexp(x.abs().amax(2))                              # |x| < 2^up
    exps = torch.where(x.abs().amax(2) > 0, (up + 124).clamp(0, 254), 0)
    codes = _pack4(_codes4(torch.ldexp(x, 127 - exps[:, :, None])).view(-1, KEY))
    y = lat.view(-1, 36, 16)
    sc = (y.abs().amax(2) / 6.0).clamp_max(448).to(torch.float8_e4m3fn)
    v = sc.float()[:, :, None]
    rec = torch.zeros((y.shape[0], 352), dtype=torch.uint8, device="cuda")
    rec[:, :288] = _pack4(_codes4(torch.where(v > 0, y / torch.where(v > 0, v, 1.0), 0.0)).view(-1, LAT))
    rec[:, 288:324] = sc.view(torch.uint8)
    return codes, exps.to(torch.uint8), rec


def _places(st):
    """(row, slot) of every packed token."""
    bs = st["case"]["bs"]
    pos = st["q_pos"].long()
    return st["bt"][st["q_req"].long(), pos // bs].long(), pos % bs


def _pages(st):
    """Views of the pool: key codes, key scales, latent records, each [rows, bs, bytes]."""
    bs, pool = st["case"]["bs"], st["pool"]
    key, lat = _sizes(st["case"]["fmt"])
    kc, rows = key - 4, pool.shape[0]
    return (pool[:, :bs * kc].view(rows, bs, kc), pool[:, bs * kc:bs * key].view(rows, bs, 4),
            pool[:, bs * key:].view(rows, bs, lat))


def _values4(byte):
    grid = torch.tensor(_GRID + [-v for v in _GRID], device="cuda")
    pair = grid[torch.stack((byte & 15, byte >> 4), -1).int()]
    return pair.view(*byte.shape[:-1], -1)


def _plain_read(st):
    row, slot = _places(st)
    codes, scales, rec = (v[row, slot] for v in _pages(st))
    if st["case"]["fmt"] == "fp8":
        k = codes.view(torch.float8_e4m3fn).float() * scales.view(torch.float32)
        return k.to(torch.bfloat16), rec.view(torch.float8_e4m3fn).to(torch.bfloat16)
    k = torch.ldexp(_values4(codes).view(-1, 4, 32), scales.int()[:, :, None] - 127).view(-1, KEY)
    sc = rec[:, 288:324].contiguous().view(torch.float8_e4m3fn).float()
    lat = (_values4(rec[:, :288]).view(-1, 36, 16) * sc[:, :, None]).view(-1, LAT)
    return k.to(torch.bfloat16), lat.to(torch.bfloat16)


def _plain_append(st):
    row, slot = _places(st)
    for page, new in zip(_pages(st), _records(st["k_new"], st["latent"], st["case"]["fmt"])):
        page[row, slot] = new
    return _plain_read(st)


# ------------------------------------------------------- the library's calls

def _prepare_own(st):
    import dsa_sparse_attention_gb300 as dsa
    st["dsa"] = dsa
    case, t = st["case"], sum(st["new"])
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")
    if st["op"] == "attn":
        st["out"], st["lse"] = new(t, case["heads"], case["dim"], dtype=st["q"].dtype), new(t, case["heads"], dtype=torch.float32)
        st["prompt"] = dsa.make_prompt(st["cu_q"], st["cu_k"], st["q"], st["k"], st["v"], k_shared=st["k_shared"],
                                       max_q=max(st["new"]), max_k=max(st["keys"]),
                                       flags=dsa.DSA_PROMPT_CAUSAL if case["causal"] else 0)
        st["ws"] = dsa.alloc_prompt_workspace(st["prompt"])
        return
    bs, fp8 = case["bs"], case["fmt"] == "fp8"
    key, lat = _sizes(case["fmt"])
    st["layout"] = dsa.make_layout(st["pool"], st["pool"].shape[0], bs * (key + lat), 0, bs * key, bs,
                                   dsa.DSA_IDX_FP8 if fp8 else dsa.DSA_IDX_MXFP4,
                                   dsa.DSA_LAT_FP8 if fp8 else dsa.DSA_LAT_NVFP4)
    longest = max(n + c for n, c in zip(st["new"], st["ctx"]))
    st["batch"] = dsa.make_batch(st["q_req"], st["q_pos"], st["lens"], st["bt"], longest)
    st["spans"] = dsa.make_spans(st["cu"], st["start"], t)
    st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    st["k_out"], st["lat_out"] = new(t, KEY), new(t, LAT)


def _run_own(st):
    dsa = st["dsa"]
    if st["op"] == "attn":
        dsa.dsa_prompt_attn(st["prompt"], st["q"], st["k"], st["v"], st["scale"], st["out"], st["lse"],
                            k_shared=st["k_shared"], prev_out=st.get("prev_out"), prev_lse=st.get("prev_lse"), ws=st["ws"])
        return st["out"], st["lse"]
    if st["op"] == "append":
        dsa.dsa_write_tokens(st["layout"], st["batch"], st["k_new"], st["latent"], ws=st["ws"])
    dsa.dsa_read_tokens(st["layout"], st["batch"], st["spans"], st["k_out"], st["lat_out"], ws=st["ws"])
    return st["k_out"], st["lat_out"]


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "append": _plain_append, "read": _plain_read}[state["op"]](state)


# ------------------------------------------- the definitions, in 64 bits

def _table4():
    return torch.tensor([(-1.0 if c & 8 else 1.0) * _GRID[c & 7] for c in range(16)], dtype=torch.float64, device="cuda")


def _table8():
    """e4m3 codes by the format's own rule: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(float("nan") if c & 127 == 127 else -v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _nearest(x, table, most):
    """x rounded to the nearest of the table's non-negative values (in order), with x's sign; ties to the even place."""
    mids = (table[1:] + table[:-1]) / 2
    a = x.abs().clamp(max=most)
    lo, hi = torch.bucketize(a, mids), torch.bucketize(a, mids, right=True)      # differ at a midpoint alone
    return torch.where(lo % 2 == 0, table[lo], table[hi]) * torch.where(x < 0, -1.0, 1.0).double()


def exact(case, seed):
    """What run returns, from the definitions: each head's softmax in float64; values quantised and read back
    by the formats' rules on float64 tables (a scale and a quotient are fp32 by definition)."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "attn":
        h, kv, d, e = case["heads"], case["kv"], case["dim"], case["shared"]
        outs = torch.empty((sum(st["new"]), h, d), dtype=torch.float64, device="cuda")
        lses = torch.empty((sum(st["new"]), h), dtype=torch.float64, device="cuda")
        q0, k0 = 0, 0
        for n, m in zip(st["new"], st["keys"]):
            hidden = None
            if case["causal"]:
                hidden = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1)
            for j in range(h):
                g = j * kv // h
                key = st["k"][k0:k0 + m, g].double()
                if e:
                    key = torch.cat((key, st["k_shared"][k0:k0 + m].double()), 1)
                dots = st["q"][q0:q0 + n, j].double().mm(key.t()) * st["scale"]
                if hidden is not None:
                    dots[hidden] = float("-inf")
                l = torch.logsumexp(dots, 1)
                o = torch.exp(dots - l[:, None]).mm(st["v"][k0:k0 + m, g].double())
                if case["join"]:
                    w = torch.sigmoid(l - st["prev_lse"][q0:q0 + n, j].double())
                    o = w[:, None] * o + (1 - w)[:, None] * st["prev_out"][q0:q0 + n, j].double()
                    l = st["prev_lse"][q0:q0 + n, j].double() - torch.log1p(-w)
                outs[q0:q0 + n, j], lses[q0:q0 + n, j] = o, l
            q0, k0 = q0 + n, k0 + m
        return outs, lses
    bs, t4, t8 = case["bs"], _table4(), _table8()
    if case["op"] == "append":
        k, lat = st["k_new"].double(), st["latent"].double()
        pos8 = t8[:127]
        if case["fmt"] == "fp8":
            s = (k.abs().amax(1, keepdim=True) / 448).float()
            s[s == 0] = 1
            k = _nearest((k / s.double()).float().double(), pos8, 448.0) * s.double()
            return k, _nearest(lat, pos8, 448.0)
        x = k.view(-1, 4, 32)
        size = 2.0 ** (torch.floor(torch.log2(x.abs().amax(2, keepdim=True))) - 2)
        k = (_nearest(x / size, t4[:8], 6.0) * size).view(-1, KEY)
        y = lat.view(-1, 36, 16)
        s = _nearest((y.abs().amax(2, keepdim=True) / 6).float().double(), pos8, 448.0)
        lat = (_nearest((y / s).float().double(), t4[:8], 6.0) * s).view(-1, LAT)
        return k, lat
    keys = torch.empty((sum(st["new"]), KEY), dtype=torch.float64, device="cuda")
    lats = torch.empty((sum(st["new"]), LAT), dtype=torch.float64, device="cuda")
    key, rec = _sizes(case["fmt"])
    at = 0
    for i, (n, c) in enumerate(zip(st["new"], st["ctx"])):
        page = st["pool"][st["bt"][i, :-(-(n + c) // bs)].long()]                # the request's pages, in order
        part = lambda a, width: page[:, bs * a:bs * (a + width)].reshape(-1, width)[c:c + n]
        if case["fmt"] == "fp8":
            keys[at:at + n] = t8[part(0, KEY).int()] * part(KEY, 4).contiguous().view(torch.float32).double()
            lats[at:at + n] = t8[part(key, rec).int()]
        else:
            b = part(0, KEY // 2).int()
            keys[at:at + n, 0::2], keys[at:at + n, 1::2] = t4[b % 16], t4[b // 16]
            keys[at:at + n] *= (2.0 ** (part(KEY // 2, 4).double() - 127)).repeat_interleave(32, 1)
            r = part(key, rec).int()
            lats[at:at + n, 0::2], lats[at:at + n, 1::2] = t4[r[:, :288] % 16], t4[r[:, :288] // 16]
            lats[at:at + n] *= t8[r[:, 288:324]].repeat_interleave(16, 1)
        at += n
    return keys, lats
