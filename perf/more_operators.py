"""Cases, plain forms and exact values of the operators that give a decoder
block positions and sparse attention over its NVFP4 key/value cache: rotary
positions with several axes, the rotation on the way into the cache, an index
of block means, the selection of blocks for each query by their means, and
attention over the selected blocks. ``own`` selects what ``run`` calls:
elementary torch operations (False) or this package (True).

The cache's pool is ``uint8 [pages, kv_heads, page_tokens / 16, 18 D]``: a
block of 16 tokens holds its key codes ``[16, D/2]`` (element 2j in the low
nibble of byte j), key scales ``[16, D/16]`` (E4M3), value codes and value
scales. A value decodes as e2m1 * e4m3 / gs with one global scale for the keys
and one for the values. The index holds one f16 row ``[D]`` of each head for
the blocks of ``block`` tokens that start in a page.
"""
import math
import random

import numpy as np
import torch

own = False

K_GS, V_GS = 112.0, 224.0       # calibrated as 2688 / amax: keys with outlier channels reach 24, values 12
DEV = "cuda"


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's queries and keys of a small batch: latency
        dict(name="rope decode", op="rope", tokens=8, qheads=32, heads=8, dim=128, rot=128, axes=1, pairs="half", far=9000,
             fused=True),
        # frames of a video among text: time, height and width
        dict(name="rope video", op="rope", tokens=16384, qheads=32, heads=8, dim=128, rot=128, axes=3, pairs="half",
             far=131072, fused=False),
        # one decode step of 32 requests: queries rotated, keys rotated into the cache, values with them
        dict(name="append decode", op="append", tokens=32, reqs=32, qheads=32, heads=8, dim=128, rot=128, axes=1,
             pairs="half", page=64, far=9000, fused=True),
        # four prompts at far positions, sliced out of a fused qkv product, three quarters of a head rotated
        dict(name="append prompts", op="append", tokens=8191, reqs=4, qheads=32, heads=8, dim=128, rot=96, axes=3,
             pairs="adjacent", page=64, far=131072, fused=True),
        # a decode step: hardly any block becomes complete
        dict(name="index decode", op="index", batch=64, kv=4096, nq=1, heads=8, dim=128, page=64, block=64, ragged=True),
        # four prompts enter, in pages smaller than a block
        dict(name="index prompts", op="index", batch=4, kv=9001, nq=8191, heads=8, dim=128, page=16, block=64, ragged=True),
        # one token of each of four long contexts picks its blocks
        dict(name="select decode", op="select", batch=4, kv=131072, nq=1, qheads=32, heads=8, dim=128, page=128, block=64,
             top=16, sink=1, local=2, ragged=False),
        # a chunk of a prompt on top of what is cached
        dict(name="select chunk", op="select", batch=1, kv=65536, nq=4096, qheads=32, heads=8, dim=128, page=64, block=64,
             top=16, sink=1, local=2, ragged=False),
        # one user, one token: latency
        dict(name="sparse decode one", op="sparse", batch=1, kv=32768, nq=1, qheads=32, heads=8, dim=128, page=64, block=64,
             top=16, sink=1, local=2, ragged=False, lse=False),
        # a serving batch of unequal lengths
        dict(name="sparse decode batch", op="sparse", batch=64, kv=32768, nq=1, qheads=64, heads=8, dim=128, page=16,
             block=64, top=32, sink=1, local=2, ragged=True, lse=False),
        # drafted tokens, four for each request, small blocks
        dict(name="sparse drafts", op="sparse", batch=16, kv=9001, nq=4, qheads=32, heads=8, dim=64, page=32, block=32,
             top=24, sink=1, local=4, ragged=True, lse=True),
        # a chunk of a prompt on top of what is cached
        dict(name="sparse chunk", op="sparse", batch=1, kv=32768, nq=2048, qheads=32, heads=8, dim=128, page=64, block=64,
             top=16, sink=1, local=2, ragged=False, lse=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "index", "select", "sparse", "sparse"])
    if op == "rope":
        dim = rng.choice([64, 72, 80, 96, 128, 128, 256])
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(4, dim // 2)
        heads = rng.choice([0, 1, 2, 8])
        qheads = max(1, heads) * rng.choice([1, 4, 5, 8])
        most = 16384 * 40 * 128 // ((qheads + heads) * dim)
        return dict(op=op, tokens=_logint(rng, 1, min(16384, most)), qheads=qheads, heads=heads, dim=dim, rot=rot,
                    axes=rng.choice([1, 2, 3]), pairs=rng.choice(["half", "adjacent"]), far=_logint(rng, 10, 1000000),
                    fused=heads > 0 and rng.random() < 0.5)
    heads, page = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
    qheads, dim = heads * rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128])
    if op == "append":
        tokens = _logint(rng, 1, 8191 * 32 // max(32, qheads))
        return dict(op=op, tokens=tokens, reqs=min(tokens, _logint(rng, 1, 64)), qheads=qheads, heads=heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 1, 3]),
                    pairs=rng.choice(["half", "adjacent"]), page=page, far=_logint(rng, 10, 1000000),
                    fused=rng.random() < 0.7)
    block, ragged = rng.choice([32, 64, 64, 128]), rng.random() < 0.7
    if op == "index":
        nq = rng.choice([1, _logint(rng, 1, 8191)])
        batch = _logint(rng, 1, min(64, 4 * 8191 // nq))
        return dict(op=op, batch=batch, kv=nq + _logint(rng, 1, 9000), nq=nq, heads=heads, dim=dim, page=page, block=block,
                    ragged=ragged)
    sink = rng.choice([0, 1, 2])
    local = rng.randint(1, 4)
    top = max(rng.choice([4, 8, 16, 16, 24, 32]), sink + local + 1)
    kind = rng.choice(["decode", "decode", "drafts", "chunk"])
    c = dict(op=op, qheads=qheads, heads=heads, dim=dim, page=page, block=block, top=top, sink=sink, local=local,
             ragged=ragged)
    if kind == "chunk":
        c["batch"] = rng.randint(1, 4)
        c["nq"] = _logint(rng, 16, 2048 * 32 // max(32, qheads) * 16 // max(16, top * block // 64) // c["batch"])
        c["kv"] = c["nq"] + _logint(rng, 16, 32768)
    else:
        c["nq"] = 1 if kind == "decode" else rng.randint(2, 6)
        c["batch"] = _logint(rng, 1, 64)
        c["kv"] = c["nq"] + min(_logint(rng, 16, 131072), 64 * 32768 // c["batch"] // c["nq"])
    if op == "sparse":
        c["lse"] = rng.random() < 0.3
    else:
        c["kv"] = max(c["kv"], c["nq"] + 9 * top * block)       # contexts with something to select
    return c


def _lengths(c):
    """(context before the step, new tokens) of each request, from the case alone."""
    r = random.Random(9173)
    if c["op"] == "append":
        cuts = sorted(r.sample(range(1, c["tokens"]), c["reqs"] - 1)) if c["reqs"] > 1 else []
        new = [b - a for a, b in zip([0] + cuts, cuts + [c["tokens"]])]
        return [r.randint(0, 300) for _ in new], new
    ctx, new = [], []
    for _ in range(c["batch"]):
        n = c["nq"] if not c["ragged"] or c["nq"] < 16 else r.randint(c["nq"] // 8, c["nq"])
        total = r.randint(max(n, c["kv"] // 8), c["kv"]) if c["ragged"] else c["kv"]
        ctx.append(total - n)
        new.append(n)
    return ctx, new


def _seen_blocks(c):
    """For every new token: (blocks it may pick from, blocks it picks, tokens in those)."""
    B = c["block"]
    for a, n in zip(*_lengths(c)):
        for p in range(a, a + n):
            own_block = p // B
            k = min(own_block + 1, c["top"])
            yield own_block + 1, k, (k - 1) * B + p % B + 1


def work(c):
    D = c["dim"]
    if c["op"] == "rope":
        rows = c["tokens"] * (c["qheads"] + c["heads"])
        return {"bytes": 4.0 * rows * D + 4.0 * c["axes"] * c["tokens"], "flops": 3.0 * rows * c["rot"]}
    if c["op"] == "append":
        n = c["tokens"] * D
        # queries in and out, keys and values in, into the cache, and what is read back
        return {"bytes": 4.0 * n * c["qheads"] + 2 * c["heads"] * n * (2 + 0.5625 + 0.5625 + 2) + 12.0 * c["tokens"],
                "flops": 3.0 * c["tokens"] * c["rot"] * (c["qheads"] + c["heads"]) + 24.0 * n * c["heads"]}
    if c["op"] == "index":
        done = sum((a + n) // c["block"] - a // c["block"] for a, n in zip(*_lengths(c)))
        per = c["heads"] * D
        return {"bytes": done * per * (c["block"] * 0.5625 + 2) + 12.0 * c["batch"],
                "flops": 2.0 * done * per * c["block"]}
    if c["op"] == "select":
        ctx, new = _lengths(c)
        means = sum((a + n) // c["block"] for a, n in zip(ctx, new)) * c["heads"] * D
        pairs = sum(s for s, _, _ in _seen_blocks(c)) * c["heads"]
        T = sum(new)
        return {"bytes": 2.0 * T * c["qheads"] * D + 2.0 * means + 4.0 * T * c["heads"] * c["top"],
                "flops": 2.0 * pairs * D}
    ctx, new = _lengths(c)
    picked = [t for _, _, t in _seen_blocks(c)]
    at, read = 0, 0
    for a, n in zip(ctx, new):
        read += min(a + n, sum(picked[at:at + n]))   # no cached token more than once for a request
        at += n
    return {"bytes": 4.0 * sum(new) * c["qheads"] * D + read * c["heads"] * 2 * D * 0.5625
            + 4.0 * sum(new) * c["heads"] * c["top"], "flops": 4.0 * sum(picked) * c["qheads"] * D}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 29)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(new):
    return _i32([0] + list(np.cumsum(np.array(new, dtype=np.int64))))


def _pages(total_tokens, page, g):
    """Pages dealt out at random: (block table, pages of the pool)."""
    need = torch.tensor([-(-t // page) for t in total_tokens])
    total = int(need.sum()) + 5
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
    at = torch.cumsum(need, 0) - need
    col = torch.arange(max(1, int(need.max())))[None, :]
    table = torch.where(col < need[:, None], perm[(at[:, None] + col).clamp(max=total - 1)], -1).to(torch.int32)
    return table.to(DEV), total


def _inv_freq(c):
    """Frequencies of the pairs as a model's configuration gives them, and the axis of each."""
    half = c["rot"] // 2
    freq = [10000.0 ** (-i / half) for i in range(half)]
    if c["axes"] == 1:
        return freq, [0] * half
    first = half // 4 if c["axes"] == 3 else half // 2           # time gets a quarter, height and width the rest
    rest = (half - first) // (c["axes"] - 1)
    return freq, [0 if i < first else min(1 + (i - first) // max(rest, 1), c["axes"] - 1) for i in range(half)]


def _positions(c, T, g):
    """Text positions that ascend from a far start, or (time, height, width) of frames after some text."""
    start = int(torch.randint(0, c["far"], (1,), generator=g, device=DEV))
    t = torch.arange(T, device=DEV)
    if c["axes"] == 1:
        return (start + t).to(torch.int32)
    side = 24
    axes = [start + t // (side * side), start + t // side % side, start + t % side]
    return torch.stack(axes[3 - c["axes"]:]).to(torch.int32).contiguous()


def _bf16(shape, g, gain=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * gain).to(torch.bfloat16)


def _keys_like(shape, g):
    """A few outlier channels, as keys have them."""
    x = torch.randn(shape, generator=g, device=DEV)
    x[..., 3::29] *= 4.0
    return x


def _random_pool(total, Hk, P, D, g):
    pool = torch.empty(total, Hk, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
    half = 9 * D
    for at, keys in ((0, True), (half, False)):
        shape = (total, Hk, P // 16, 16, D)
        codes, sf = _quantise(_keys_like(shape, g) if keys else torch.randn(shape, generator=g, device=DEV),
                              K_GS if keys else V_GS)
        pool[..., at:at + 8 * D] = codes.flatten(3)
        pool[..., at + 8 * D:at + half] = sf.flatten(3)
    return pool


def _entries(c, total):
    return total * max(1, c["page"] // c["block"])


def _row_of(cu, T):
    """Request and place within it of every row."""
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, t - cu[b]


def _rank_blocks(c, score, own_block):
    """The picked blocks, ascending and padded with -1, of scores [T, Hk, n]: the first ``sink`` and last ``local``
    that a query sees, then the largest scores, the lower block of equal ones first."""
    n = score.shape[-1]
    j = torch.arange(n, device=DEV)
    own_block = own_block[:, None, None]
    score = torch.where((j < c["sink"]) | (j > own_block - c["local"]), math.inf, score)
    score = torch.where(j > own_block, -math.inf, score)
    top = min(c["top"], n)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    best = torch.where(best > own_block, n, best).sort(-1).values
    best = torch.where(best == n, -1, best).to(torch.int32)
    pad = torch.full((*best.shape[:2], c["top"] - top), -1, dtype=torch.int32, device=DEV)
    return torch.cat((best, pad), -1)


def _agreeing_scores(c, cu, T, n, g):
    """Scores of which neighbouring queries share most, as they do in text."""
    b, i = _row_of(cu.long(), T)
    seg = b * 4096 + i // 32
    _, seg = torch.unique(seg, return_inverse=True)
    base = torch.randn(int(seg.max()) + 1, c["heads"], n, generator=g, device=DEV)
    return base[seg] + 0.4 * torch.randn(T, c["heads"], n, generator=g, device=DEV)


def prepare(c, seed):
    g = _gen(seed)
    st = {"case": c}
    D = c["dim"]
    if c["op"] in ("rope", "append"):
        T, Hq, Hk = c["tokens"], c["qheads"], c["heads"]
        # queries, keys and values as the projections leave them: columns of a fused product, or their own
        qkv = torch.empty(T, Hq + 2 * Hk, D, dtype=torch.bfloat16, device=DEV)
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV))
        qkv[:, Hq:Hq + Hk, 3::29] *= 4.0
        parts = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        st["q"], st["k"], st["v"] = parts if c["fused"] else (p.contiguous() for p in parts)
        st["pos"] = _positions(c, T, g)
        freq, axis = _inv_freq(c)
        st["freq"], st["axis"] = torch.tensor(freq, dtype=torch.float64, device=DEV), torch.tensor(axis, device=DEV)
        if own:
            from nvfp4_mixture_experts_moe_gb300 import Rope
            st["rope"] = Rope(c["rot"], inv_freq=freq, axes=axis, pairs=c["pairs"])
        if c["op"] == "rope":
            return st
    ctx, new = _lengths(c)
    P, Hk = c["page"], c["heads"]
    table, total = _pages([a + n for a, n in zip(ctx, new)], P, g)
    cu, kv_len, T = _cu(new), _i32([a + n for a, n in zip(ctx, new)]), sum(new)
    if own:
        from nvfp4_mixture_experts_moe_gb300 import Kv4BlockIndex, Kv4Cache

        def cache_of(pool):
            return Kv4Cache(total, P, Hk, D, K_GS, V_GS, pool=pool)
    if c["op"] == "append":
        b, i = _row_of(cu.long(), T)
        at = _i32(ctx).long()[b] + i
        st["slots"] = (table[b, at // P].long() * P + at % P).to(torch.int32)
        st["pool"] = torch.zeros(total, Hk, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
        if own:
            st["cache"] = cache_of(st["pool"])
        return st
    st.update(cu=cu, kv_len=kv_len, table=table, max_q=max(new))
    if c["op"] == "index":
        st["pool"] = _random_pool(total, Hk, P, D, g)
        st["means"] = torch.randn(_entries(c, total), Hk, D, generator=g, device=DEV).to(torch.float16)   # earlier ones
        if own:
            st["index"] = Kv4BlockIndex(cache_of(st["pool"]), c["block"], means=st["means"])
        return st
    st["q"] = _bf16((T, c["qheads"], D), g)
    if c["op"] == "select":
        # means of blocks that each have a subject of their own, on the index's grid
        means = 0.7 * torch.randn(_entries(c, total), Hk, D, generator=g, device=DEV, dtype=torch.float32) * K_GS
        means[..., 3::29] *= 2.0
        st["means"] = _grid(means.double(), 6, -1).to(torch.float16)
        if own:
            st["index"] = Kv4BlockIndex(cache_of(torch.empty(total, Hk, P // 16, 18 * D, dtype=torch.uint8, device=DEV)),
                                        c["block"], means=st["means"])
        return st
    st["pool"] = _random_pool(total, Hk, P, D, g)
    b, i = _row_of(cu.long(), T)
    n = -(-max(a + m for a, m in zip(ctx, new)) // c["block"])
    st["blocks"] = _rank_blocks(c, _agreeing_scores(c, cu, T, n, g), (_i32(ctx).long()[b] + i) // c["block"])
    if own:
        st["cache"] = cache_of(st["pool"])
    return st


# --------------------------------------------------------------- plain forms

def _quantise(x, gs):
    """NVFP4 with a given global scale: packed codes and E4M3 scale bytes of blocks of 16 along the last axis."""
    b = x.unflatten(-1, (-1, 16))
    six, gs = torch.full((), 6.0, device=x.device), torch.full((), gs, device=x.device)
    s = b.abs().amax(-1, keepdim=True) / six * gs
    sf = s.clamp(max=448.0).to(torch.float8_e4m3fn)
    f = sf.float()
    y = torch.where(f > 0, b * (gs / f), torch.zeros_like(b))
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(y)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, sf.squeeze(-1).view(torch.uint8)


def _dequantise(codes, sf, gs):
    """Values of packed codes [..., D/2] with scale bytes [..., D/16], fp32."""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = mag[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    s = sf.view(torch.float8_e4m3fn).float()[..., None]
    return (v.unflatten(-1, (-1, 16)) * s / torch.full((), gs, device=v.device)).flatten(-2)


def _halves(pool, D):
    """The pool's four parts: key codes, key scales, value codes, value scales, tokens on the axis before the last."""
    return (pool[..., :8 * D].unflatten(-1, (16, -1)), pool[..., 8 * D:9 * D].unflatten(-1, (16, -1)),
            pool[..., 9 * D:17 * D].unflatten(-1, (16, -1)), pool[..., 17 * D:].unflatten(-1, (16, -1)))


def _exponent(x):
    """floor(log2(x)), at least -100."""
    return torch.frexp(x.clamp(min=2.0 ** -100)).exponent.long() - 1


def _two(e):
    """2^e in 64 bits."""
    return (e + 1023 << 52).view(torch.float64)


def _grid(x, bits, *axes):
    """x rounded to multiples of 2^(E - bits), E the exponent of the largest magnitude over the axes (64 bits)."""
    e = _exponent(x.abs().amax(axes, keepdim=True)) - bits
    return (x * _two(-e)).round() * _two(e)


def _turned(x, st):
    """Rows [T, heads, D] rotated, in 32 bits; the angles in 64."""
    c = st["case"]
    pos = st["pos"].double().reshape(c["axes"], -1)[st["axis"]].T           # the position that each pair goes by
    angle = pos * st["freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    if c["pairs"] == "half":
        a, b = x[..., :c["rot"] // 2], x[..., c["rot"] // 2:c["rot"]]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((y, x[..., c["rot"]:]), -1)


def _plain_append(st):
    c = st["case"]
    P, Hk, D = c["page"], c["heads"], c["dim"]
    s = st["slots"].long()
    kc, ks, vc, vs = _halves(st["pool"], D)
    at = ((s // P)[:, None], torch.arange(Hk, device=DEV)[None, :], (s % P // 16)[:, None], (s % 16)[:, None])
    kc[at], ks[at] = _quantise(_turned(st["k"], st), K_GS)
    vc[at], vs[at] = _quantise(st["v"].float(), V_GS)
    return {"q": _turned(st["q"], st).to(torch.bfloat16), "k": _dequantise(kc[at], ks[at], K_GS).to(torch.bfloat16),
            "v": _dequantise(vc[at], vs[at], V_GS).to(torch.bfloat16)}


def _block_tokens(c, table, blocks):
    """(page, 16-token block, token) of every token of the blocks [..., n] of the requests' tables [..., pages]."""
    tok = (blocks[..., None] * c["block"] + torch.arange(c["block"], device=DEV)).flatten(-2)
    page = torch.gather(table, -1, (tok // c["page"]).clamp(0, table.shape[-1] - 1)).clamp(min=0)
    return tok, page, tok % c["page"] // 16, tok % 16


def _plain_index(st):
    c = st["case"]
    B, P, D = c["block"], c["page"], c["dim"]
    kv, new = st["kv_len"].long(), (st["cu"][1:] - st["cu"][:-1]).long()
    n = (st["max_q"] + B - 1) // B + 1
    blk = (kv - new)[:, None] // B + torch.arange(n, device=DEV)                      # the blocks with new tokens
    done = (blk < kv[:, None] // B).flatten()
    table = st["table"].long()
    tok, page, sub, row = _block_tokens(c, table, blk.clamp(max=(table.shape[1] * P - 1) // B))
    kc, ks, _, _ = _halves(st["pool"], D)
    at = tuple(i.unflatten(1, (n, B)).flatten(0, 1)[done][:, None] for i in (page, sub, row))
    h = torch.arange(c["heads"], device=DEV)[None, :, None]
    keys = _dequantise(kc[at[0], h, at[1], at[2]], ks[at[0], h, at[1], at[2]], 1.0)   # [blocks, heads, tokens, D]
    first = page.unflatten(1, (n, B)).flatten(0, 1)[done][:, 0]
    entry = first * max(1, P // B) + blk.flatten()[done] * B % P // B
    st["means"][entry] = _grid(keys.double().mean(2), 6, -1).to(torch.float16)
    return {"means": st["means"]}


def _plain_select(st):
    c = st["case"]
    B, P, Hk, Q = c["block"], c["page"], c["heads"], st["max_q"]
    cu, kv, table, T = st["cu"].long(), st["kv_len"].long(), st["table"].long(), st["q"].shape[0]
    b, i = _row_of(cu, T)
    q = st["q"].double().unflatten(1, (Hk, -1))
    step = _two(5 - _exponent(q.abs().amax((2, 3), keepdim=True)))
    u = (q * step).round().sum(2).float()                                  # [T, Hk, D], whole numbers
    n = (table.shape[1] * P + B - 1) // B
    start = torch.arange(n, device=DEV) * B
    entry = table[:, start // P].clamp(min=0) * max(1, P // B) + start % P // B
    means = st["means"][entry].float().permute(0, 2, 3, 1)                 # [requests, Hk, D, n]
    rows = (cu[:-1, None] + torch.arange(Q, device=DEV)).clamp(max=T - 1)
    score = torch.matmul(u[rows].transpose(1, 2), means).transpose(1, 2)   # exact: whole numbers times a power of two
    own_block = ((kv - cu[1:] + cu[:-1])[b] + i) // B
    return {"blocks": _rank_blocks(c, score[b, i], own_block)}


def _plain_sparse(st):
    c = st["case"]
    D, P, Hk, T = c["dim"], c["page"], c["heads"], st["q"].shape[0]
    cu, kv = st["cu"].long(), st["kv_len"].long()
    b, i = _row_of(cu, T)
    last = (kv - cu[1:] + cu[:-1])[b] + i
    blocks = st["blocks"].long()
    tok, page, sub, row = _block_tokens(c, st["table"].long()[b][:, None].expand(-1, Hk, -1), blocks.clamp(min=0))
    see = (blocks >= 0)[..., None].expand(-1, -1, -1, c["block"]).flatten(2) & (tok <= last[:, None, None])
    h = torch.arange(Hk, device=DEV)[None, :, None]
    kc, ks, vc, vs = _halves(st["pool"], D)
    at = (page, h, sub, row)
    q = st["q"].float().unflatten(1, (Hk, -1))
    s = torch.matmul(q, _dequantise(kc[at], ks[at], K_GS).transpose(2, 3)) * D ** -0.5
    s = s.masked_fill(~see[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _dequantise(vc[at], vs[at], V_GS))
    out = {"out": torch.where(total > 0, o / total, 0.0).flatten(1, 2).to(torch.bfloat16)}
    if c["lse"]:
        out["lse"] = (m + total.log()).squeeze(-1).flatten(1, 2)
    return out


def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "rope":
            q = _turned(st["q"], st).to(torch.bfloat16)
            return {"q": q, "k": _turned(st["k"], st).to(torch.bfloat16)} if c["heads"] else {"q": q}
        return {"append": _plain_append, "index": _plain_index, "select": _plain_select, "sparse": _plain_sparse}[c["op"]](st)
    if c["op"] == "rope":
        if not c["heads"]:
            return {"q": st["rope"](st["q"], st["pos"])}
        q, k = st["rope"](st["q"], st["pos"], k=st["k"])
        return {"q": q, "k": k}
    if c["op"] == "append":
        q = st["cache"].append_rotated(st["q"], st["k"], st["v"], st["slots"], st["pos"], st["rope"])
        k, v = st["cache"].read(st["slots"])
        return {"q": q, "k": k, "v": v}
    if c["op"] == "index":
        st["index"].update(st["cu"], st["kv_len"], st["table"], max_q=st["max_q"])
        return {"means": st["means"]}
    if c["op"] == "select":
        return {"blocks": st["index"].select(st["q"], st["cu"], st["kv_len"], st["table"], max_q=st["max_q"],
                                             top=c["top"], sink=c["sink"], local=c["local"])}
    o, lse = st["cache"].sparse_attention(st["q"], st["cu"], st["kv_len"], st["table"], st["blocks"],
                                          block_tokens=c["block"], max_q=st["max_q"], want_lse=c["lse"])
    return {"out": o, "lse": lse} if c["lse"] else {"out": o}


# --------------------------------------------------------------- exact values

_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def _e4m3_table():
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


def _nearest_even(x, grid):
    """Index of the nearest of an ascending grid, ties to the even index, clamped to its ends."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    mid = (grid[lo] + grid[hi]) / 2
    return np.where((x > mid) | ((x == mid) & (hi % 2 == 0)), hi, lo)


def _stored(x, gs):
    """The values that the cache holds for x: the quantiser's decisions are defined on correctly rounded fp32 steps."""
    f = np.float32
    b = x.astype(f).reshape(x.shape[:-1] + (-1, 16))
    s = np.abs(b).max(-1) / f(6.0) * f(gs)
    grid = _e4m3_table()[:127]
    sf = grid[_nearest_even(s.astype(np.float64), grid)].astype(f)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(sf[..., None] > 0, b * (f(gs) / sf)[..., None], f(0))
    v = _E2M1[_nearest_even(np.abs(y).astype(np.float64), _E2M1)]
    return (np.copysign(v, y) * sf[..., None].astype(np.float64) / gs).reshape(x.shape)


def _rotated(x, c, pos):
    """Each pair as a complex number times exp(i angle)."""
    freq, axis = _inv_freq(c)
    pos = pos.cpu().numpy().reshape(c["axes"], -1).astype(np.float64)
    turn = np.exp(1j * pos[axis].T * np.array(freq))[:, None]
    x = x.double().cpu().numpy()
    y, half = x.copy(), c["rot"] // 2
    lo, hi = (slice(0, half), slice(half, c["rot"])) if c["pairs"] == "half" else (slice(0, c["rot"], 2),
                                                                                slice(1, c["rot"], 2))
    z = (x[..., lo] + 1j * x[..., hi]) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_rows(pool, pages, h, D, at, gs):
    """Cached rows of one request's pages and head in float64, on the pool's device."""
    blk = pool[pages.long(), h].flatten(0, 1)                              # [pages * P/16, 18 D]
    codes = blk[:, at:at + 8 * D].reshape(-1, D // 2)
    sf = blk[:, at + 8 * D:at + 9 * D].reshape(-1, D // 16)
    mag = torch.tensor(np.concatenate((_E2M1, -_E2M1)), device=pool.device)
    v = torch.empty(len(codes), D, dtype=torch.float64, device=pool.device)
    v[:, 0::2], v[:, 1::2] = mag[(codes & 15).long()], mag[(codes >> 4).long()]
    scale = torch.tensor(_e4m3_table(), device=pool.device)[sf.long()]
    return v * scale.repeat_interleave(16, 1) / gs


def exact(c, seed):
    if c["op"] == "select":
        return None  # whole numbers
    st = prepare(c, seed)
    if c["op"] in ("rope", "append"):
        q = _rotated(st["q"], c, st["pos"])
        if c["op"] == "rope" and not c["heads"]:
            return {"q": q}
        k = _rotated(st["k"], c, st["pos"])
        if c["op"] == "rope":
            return {"q": q, "k": k}
        return {"q": q, "k": _stored(k, K_GS), "v": _stored(st["v"].float().cpu().numpy(), V_GS)}
    Hk, D, P, B = c["heads"], c["dim"], c["page"], c["block"]
    ctx, new = _lengths(c)
    if c["op"] == "index":
        means = st["means"].double().cpu().numpy()
        for b, (a, n) in enumerate(zip(ctx, new)):
            first, end = a // B, (a + n) // B
            if first == end:
                continue
            pages = st["table"][b, first * B // P:-(-end * B // P)]
            skip = first * B - first * B // P * P
            for h in range(Hk):
                rows = _exact_rows(st["pool"], pages, h, D, 0, 1.0)[skip:skip + (end - first) * B]
                mean = rows.cpu().numpy().reshape(end - first, B, D).sum(1) / B
                step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(mean).max(1), 2.0 ** -100))) - 6)
                for j in range(end - first):
                    at = (first + j) * B
                    entry = int(st["table"][b, at // P]) * max(1, P // B) + at % P // B
                    means[entry, h] = np.rint(mean[j] / step[j]) * step[j]
        return {"means": means}
    g, row = c["qheads"] // Hk, 0
    q = st["q"].double()
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b, (a, n) in enumerate(zip(ctx, new)):
        pages = st["table"][b, :-(-(a + n) // P)]
        blocks_of = -(-(a + n) // B)
        for h in range(Hk):
            key, val = (_exact_rows(st["pool"], pages, h, D, at, gs)[:a + n] for at, gs in ((0, K_GS), (9 * D, V_GS)))
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                picked = torch.zeros(i1 - i0, blocks_of + 1, dtype=torch.bool, device=DEV)
                ids = st["blocks"][row + i0:row + i1, h].long()
                picked.scatter_(1, torch.where(ids < 0, blocks_of, ids), True)
                see = picked[:, :blocks_of].repeat_interleave(B, 1)[:, :a + n]
                see &= torch.arange(a + n, device=DEV) <= torch.arange(a + i0, a + i1, device=DEV)[:, None]
                s = q[row + i0:row + i1, h * g:(h + 1) * g].transpose(0, 1) @ key.T / math.sqrt(D)
                s = s.masked_fill(~see, -math.inf)
                top = torch.logsumexp(s, -1)
                out[row + i0:row + i1, h * g:(h + 1) * g] = ((s - top[..., None]).exp() @ val).transpose(0, 1)
                lse[row + i0:row + i1, h * g:(h + 1) * g] = top.T
        row += n
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
