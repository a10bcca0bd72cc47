"""Cases, plain forms and exact values of the operators around the MoE layer:
the NVFP4 key/value cache (append, read back, attention over it), the tables
that place a step's tokens in that cache, and the norms before and after a
block. ``own`` selects what ``run`` calls: elementary torch operations in fp32
(False) or this package (True).

The cache's pool is ``uint8 [pages, kv_heads, page_tokens / 16, SB]``: a block
of 16 tokens holds its key codes ``[16, D/2]`` (element 2j in the low nibble
of byte j), key scales ``[16, D/16]`` (E4M3), value codes and value scales, SB
= 18 D bytes. A value decodes as e2m1 * e4m3 / gs with one global scale for
the keys and one for the values.
"""
import math
import random

import numpy as np
import torch

own = False

K_GS, V_GS = 112.0, 224.0       # calibrated as 2688 / amax: keys with outlier channels reach 24, values 12
EPS = 1e-6
DEV = "cuda"


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a serving step's bookkeeping: every request decodes one token
        dict(name="step decode", op="step", batch=64, page=64, ctx=4096, new=1, pad=0),
        # a step that admits prompts next to decodes, into small pages, padded as for graph replay
        dict(name="step prompts", op="step", batch=500, page=16, ctx=9000, new=260, pad=321),
        # one decode step of 32 requests writes its keys and values
        dict(name="append decode", op="append", tokens=32, reqs=32, heads=8, dim=128, page=64, fused=True),
        # four prompts' keys and values, sliced out of a fused qkv product
        dict(name="append prompts", op="append", tokens=8191, reqs=4, heads=8, dim=128, page=64, fused=True),
        # decode batch of the flagship decode layer's width
        dict(name="norm decode", op="norm", tokens=8, hidden=4096, gate="channel", res="bf16", post=True, pre=True),
        # prompt batch of the widest layer, a gate for each token
        dict(name="norm prompts", op="norm", tokens=16384, hidden=7168, gate="token", res="bf16", post=True, pre=True),
        # one user, one token: latency
        dict(name="attn decode one", op="attn", batch=1, kv=1000, nq=1, qheads=32, heads=8, dim=128, page=64,
             ragged=False, window=0, lse=False, idle=0),
        # a serving batch of unequal lengths, some slots idle
        dict(name="attn decode batch", op="attn", batch=64, kv=8192, nq=1, qheads=64, heads=8, dim=128, page=16,
             ragged=True, window=0, lse=False, idle=3),
        # long contexts
        dict(name="attn decode long", op="attn", batch=4, kv=131072, nq=1, qheads=32, heads=8, dim=128, page=128,
             ragged=False, window=0, lse=True, idle=0),
        # drafted tokens scored against the cache, four for each request
        dict(name="attn drafts", op="attn", batch=16, kv=9001, nq=4, qheads=32, heads=8, dim=64, page=32,
             ragged=True, window=0, lse=False, idle=0),
        # a whole prompt
        dict(name="attn prompt", op="attn", batch=1, kv=4096, nq=4096, qheads=32, heads=8, dim=128, page=64,
             ragged=False, window=0, lse=False, idle=0),
        # prompt chunks of several requests on top of what they hold, sliding window
        dict(name="attn chunks", op="attn", batch=6, kv=12001, nq=700, qheads=16, heads=2, dim=64, page=16,
             ragged=True, window=4096, lse=True, idle=0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "append", "norm", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "step":
        new = rng.choice([1, 1, _logint(rng, 2, 260)])
        return dict(op=op, batch=_logint(rng, 1, 500), page=page, ctx=_logint(rng, 1, 9000), new=new,
                    pad=rng.choice([0, rng.randint(1, 321)]))
    if op == "append":
        tokens = _logint(rng, 1, 8191)
        return dict(op=op, tokens=tokens, reqs=min(tokens, _logint(rng, 1, 64)), heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 128]), page=page, fused=rng.random() < 0.7)
    if op == "norm":
        hidden = rng.choice([256, 1000, 2048, 4096, 5120, 7168, 8192, rng.randint(100, 7168)])
        return dict(op=op, tokens=_logint(rng, 1, 16384), hidden=min(hidden, 7168),
                    gate=rng.choice(["none", "channel", "token"]), res=rng.choice(["bf16", "bf16", "f32"]),
                    post=rng.random() < 0.8, pre=rng.random() < 0.9)
    heads = rng.choice([1, 2, 4, 8])
    qheads = heads * rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 128])
    kind = rng.choice(["decode", "decode", "drafts", "prompt"])
    lse = rng.random() < 0.3
    if kind in ("decode", "drafts"):
        batch = _logint(rng, 1, 64)
        kv = min(_logint(rng, 16, 131072), 4 * 131072 // batch)
        nq = 1 if kind == "decode" else rng.randint(2, 9)
        idle = rng.choice([0, rng.randint(0, batch // 8)])
        window = rng.choice([0, 0, 0, _logint(rng, 64, 8192)])
        return dict(op=op, batch=batch, kv=max(kv, nq), nq=nq, qheads=qheads, heads=heads, dim=dim, page=page,
                    ragged=rng.random() < 0.7, window=window, lse=lse, idle=idle)
    batch = rng.randint(1, 6)
    nq = _logint(rng, 24, 4096 // batch)
    kv = max(nq, min(_logint(rng, 24, 16384), 32 * 4096 * 4096 // (batch * nq * qheads)))
    return dict(op=op, batch=batch, kv=kv, nq=nq, qheads=qheads, heads=heads, dim=dim, page=page,
                ragged=rng.random() < 0.7, window=rng.choice([0, 0, _logint(rng, 64, 4096)]), lse=lse, idle=0)


def _lengths(c):
    """(context before the step, new tokens) of each request, from the case alone."""
    r = random.Random(9173)
    if c["op"] == "step":
        new = [1 if c["new"] == 1 or r.random() < 0.5 else r.randint(1, c["new"]) for _ in range(c["batch"])]
        return [r.randint(0, c["ctx"]) for _ in new], new
    if c["op"] == "append":
        cuts = sorted(r.sample(range(1, c["tokens"]), c["reqs"] - 1)) if c["reqs"] > 1 else []
        new = [b - a for a, b in zip([0] + cuts, cuts + [c["tokens"]])]
        return [r.randint(0, 300) for _ in new], new
    kv, new = [], []
    for b in range(c["batch"]):
        n = c["nq"] if not c["ragged"] or c["nq"] < 24 else r.randint(1, c["nq"])
        total = r.randint(max(n, c["kv"] // 8), c["kv"]) if c["ragged"] else c["kv"]
        if b % 8 == 3 and b // 8 < c["idle"]:
            n, total = 0, 0  # an idle slot of a padded batch
        kv.append(total - n)
        new.append(n)
    return kv, new


def work(c):
    if c["op"] == "step":
        ctx, new = _lengths(c)
        pages = sum(-(-(a + b) // c["page"]) + -(-a // c["page"]) for a, b in zip(ctx, new))
        # lengths in, tables read, new pages in and out, two indices for each token
        return {"bytes": 4.0 * (5 * len(ctx) + pages + 2 * (sum(new) + c["pad"])), "flops": 0.0}
    if c["op"] == "append":
        n = c["tokens"] * c["heads"] * c["dim"] * 2
        return {"bytes": n * (2 + 0.5625 + 0.5625 + 2) + 8.0 * c["tokens"], "flops": 12.0 * n}
    if c["op"] == "norm":
        n = c["tokens"] * c["hidden"]
        r = 2 if c["res"] == "bf16" else 4
        b = n * (2 + 2 * r + (2 if c["gate"] == "token" else 0) + (2 if c["pre"] else 0))
        return {"bytes": float(b), "flops": 10.0 * n}
    ctx, new = _lengths(c)
    pairs = read = 0
    for a, n in zip(ctx, new):
        if n == 0:
            continue
        w = c["window"] or (a + n)
        m = max(0, min(n, w - a))              # rows that see everything before them
        pairs += m * a + m * (m + 1) // 2 + (n - m) * w
        read += min(a + n, w + n - 1)
    q = sum(new) * c["qheads"] * c["dim"]
    return {"bytes": 2.0 * 2 * q + read * c["heads"] * 2 * c["dim"] * 0.5625,
            "flops": 4.0 * pairs * c["qheads"] * c["dim"]}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 17)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(new):
    return _i32([0] + list(np.cumsum(np.array(new, dtype=np.int64))))


def _pages(ctx, new, page, g):
    """A pool's pages dealt out at random: (block table with -1 past the context's pages, pages still free, all)."""
    old = torch.tensor([-(-a // page) for a in ctx])
    need = torch.tensor([-(-(a + b) // page) for a, b in zip(ctx, new)])
    total = int(need.sum()) + 5
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
    width = max(1, int(need.max()))
    at = torch.cumsum(old, 0) - old
    col = torch.arange(width)[None, :]
    table = torch.where(col < old[:, None], perm[(at[:, None] + col).clamp(max=total - 1)], -1).to(torch.int32)
    return table.to(DEV), perm[int(old.sum()):].contiguous().to(DEV), total


def _kv_like(shape, g, keys):
    """Keys carry a few outlier channels, values do not."""
    x = torch.randn(shape, generator=g, device=DEV)
    if keys:
        gain = torch.ones(shape[-1], device=DEV)
        gain[3::29] = 4.0
        x *= gain
    return x


def prepare(c, seed):
    g = _gen(seed)
    st = {"case": c}
    if c["op"] == "norm":
        T, H = c["tokens"], c["hidden"]
        bf = torch.bfloat16
        st["x"] = (torch.randn(T, H, generator=g, device=DEV) * 0.7).to(bf)
        st["residual"] = (torch.randn(T, H, generator=g, device=DEV) * 3).to(bf if c["res"] == "bf16" else torch.float32)
        gate = None if c["gate"] == "none" else torch.rand((T, H) if c["gate"] == "token" else (H,), generator=g,
                                                           device=DEV)
        st["gate"] = None if gate is None else gate.to(bf)
        wp = (torch.rand(H, generator=g, device=DEV) + 0.5).to(bf)
        wn = (torch.rand(H, generator=g, device=DEV) + 0.5).to(bf)
        st["w_post"], st["w_pre"] = wp if c["post"] else None, wn if c["pre"] else None
        return st
    ctx, new = _lengths(c)
    P, T = c["page"], sum(new)
    table, free, total = _pages(ctx, new, P, g)
    if c["op"] == "step":
        # what the next step needs: lengths, the table so far, the free pages as a stack
        st.update(ctx=_i32(ctx), new=_i32(new), table=table, free=free, count=_i32([free.numel()]), tokens=T + c["pad"])
        if own:
            from nvfp4_mixture_experts_moe_gb300 import KvStep
            st["step"] = KvStep(c["batch"], T + c["pad"], P, table.shape[1])
        return st
    Hk, D = c["heads"], c["dim"]
    cu = _cu(new)
    ctx_t, new_t = _i32(ctx), _i32(new)
    slots = _plain_step(ctx_t, new_t, table, free, _i32([free.numel()]), P, T)
    table, slots = slots["block_table"], slots["slots"]
    if c["op"] == "append":
        # keys and values as the projections leave them: columns of a fused product, or their own
        if c["fused"]:
            qkv = torch.empty(T, (4 + 2) * Hk, D, dtype=torch.bfloat16, device=DEV)
            st["k"], st["v"] = qkv[:, 4 * Hk:5 * Hk], qkv[:, 5 * Hk:]
        else:
            st["k"], st["v"] = (torch.empty(T, Hk, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        st["k"].copy_(_kv_like((T, Hk, D), g, True))
        st["v"].copy_(_kv_like((T, Hk, D), g, False))
        st["slots"] = slots
        st["pool"] = torch.zeros(total, Hk, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
    else:
        st["q"] = torch.randn(T, c["qheads"], D, generator=g, device=DEV).to(torch.bfloat16)
        st["cu"], st["kv_len"], st["table"], st["max_q"] = cu, ctx_t + new_t, table, max(max(new), 1)
        pool = torch.empty(total, Hk, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
        half = 9 * D
        for at, keys in ((0, True), (half, False)):
            codes, sf = _quantise(_kv_like((total, Hk, P // 16, 16, D), g, keys), K_GS if keys else V_GS)
            pool[..., at:at + 8 * D] = codes.flatten(3)
            pool[..., at + 8 * D:at + half] = sf.flatten(3)
        st["pool"] = pool
    if own:
        # the handle on the pool and the workspace that a serving loop keeps
        from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
        st["cache"] = Kv4Cache(total, P, Hk, D, K_GS, V_GS, pool=st["pool"])
        if c["op"] == "attn":
            st["ws"] = st["cache"].attention_workspace(T, c["batch"], c["qheads"], st["max_q"])
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


def _plain_step(ctx, new, table, free, count, P, tokens):
    ctx, new, n = ctx.long(), new.long(), count.long()[0]
    old, want = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    need = want - old
    upto = torch.cumsum(need, 0)
    ok = (need == 0) | (upto <= n)
    need = torch.where(ok, need, 0)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (col >= old[:, None]) & (col < (old + need)[:, None])
    take = (n - 1 - (first[:, None] + col - old[:, None])).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[take], table)
    cu = torch.cat((torch.zeros_like(new[:1]), torch.cumsum(new, 0)))
    t = torch.arange(tokens, device=table.device)
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = req < len(new)
    req = req.clamp(max=len(new) - 1)
    pos = ctx[req] + t - cu[req]
    page = table[req, (pos // P).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(real & ok[req], page * P + pos % P, -1)
    return {"block_table": table, "cu_q": cu.int(), "kv_len": torch.where(ok, ctx + new, ctx).int(),
            "slots": slots.int(), "positions": torch.where(real, pos, 0).int(),
            "free_count": (n - need.sum()).int().reshape(1)}


def _plain_append(st):
    c = st["case"]
    P, Hk, D = c["page"], c["heads"], c["dim"]
    pool, s = st["pool"], st["slots"].long()
    kc, ks, vc, vs = _halves(pool, D)
    page, sub, tok = s // P, s % P // 16, s % 16
    at = (page[:, None], torch.arange(Hk, device=DEV)[None, :], sub[:, None], tok[:, None])
    codes, sf = _quantise(st["k"].float(), K_GS)
    kc[at], ks[at] = codes, sf
    codes, sf = _quantise(st["v"].float(), V_GS)
    vc[at], vs[at] = codes, sf
    return {"k": _dequantise(kc[at], ks[at], K_GS).to(torch.bfloat16),
            "v": _dequantise(vc[at], vs[at], V_GS).to(torch.bfloat16)}


def _plain_attention(st):
    c = st["case"]
    Hk, D, Hq, B = c["heads"], c["dim"], c["qheads"], c["batch"]
    cu, kv, Q = st["cu"].long(), st["kv_len"].long(), st["max_q"]
    nq = cu[1:] - cu[:-1]
    mine = st["pool"][st["table"].clamp(min=0).long()]                    # [B, pages, Hk, P/16, 18 D]
    parts = [p.permute(0, 2, 1, 3, 4, 5).flatten(2, 4) for p in _halves(mine, D)]
    del mine
    i = torch.arange(Q, device=DEV)[None, :]
    rows = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[rows].unflatten(2, (Hk, Hq // Hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = torch.matmul(q, _dequantise(parts[0], parts[1], K_GS).transpose(2, 3)).mul_(D ** -0.5)
    L = s.shape[-1]
    last = (kv - nq)[:, None] + i                                         # the position of each query
    t = torch.arange(L, device=DEV)
    see = (t <= last[..., None]) & (t < kv[:, None, None]) & (i < nq[:, None])[..., None]
    if c["window"]:
        see &= t > last[..., None] - c["window"]
    s = s.view(B, Hk, Hq // Hk, Q, L).masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), _dequantise(parts[2], parts[3], V_GS)).view(B, Hk, Hq // Hk, Q, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log()).squeeze(-1)
    n = torch.arange(st["q"].shape[0], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), n, right=True).clamp(max=B - 1)
    at = n - cu[b]
    out = {"out": o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, at].to(torch.bfloat16)}
    if c["lse"]:
        out["lse"] = lse.permute(0, 3, 1, 2).flatten(2, 3)[b, at]
    return out


def _plain_norm(st):
    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    n = st["x"].float()
    if st["w_post"] is not None:
        n = norm(n, st["w_post"])
    if st["gate"] is not None:
        n = n * st["gate"].float()
    r = 1.25 * st["residual"].float() + 0.75 * n
    out = {"residual": r.to(st["residual"].dtype)}
    if st["w_pre"] is not None:
        out["out"] = norm(r, st["w_pre"]).to(torch.bfloat16)
    return out


def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "step":
            return _plain_step(st["ctx"], st["new"], st["table"], st["free"], st["count"], c["page"], st["tokens"])
        return {"append": _plain_append, "norm": _plain_norm, "attn": _plain_attention}[c["op"]](st)
    if c["op"] == "step":
        s = st["step"].run(st["ctx"], st["new"], st["table"], st["free"], st["count"])
        return {"block_table": st["table"], "cu_q": s.cu_q, "kv_len": s.kv_len, "slots": s.slots,
                "positions": s.positions, "free_count": s.free_count}
    if c["op"] == "append":
        st["cache"].append(st["k"], st["v"], st["slots"])
        k, v = st["cache"].read(st["slots"])
        return {"k": k, "v": v}
    if c["op"] == "norm":
        from nvfp4_mixture_experts_moe_gb300 import block_norm
        r, y = block_norm(st["x"], st["residual"], gate=st["gate"], w_post=st["w_post"], w_pre=st["w_pre"],
                          residual_scale=1.25, branch_scale=0.75, eps=EPS)
        return {"residual": r} if y is None else {"residual": r, "out": y}
    o, lse = st["cache"].attention(st["q"], st["cu"], st["kv_len"], st["table"], max_q=st["max_q"],
                                   window=c["window"], want_lse=c["lse"], ws=st["ws"])
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


def _exact_append(x, gs):
    """The stored values: the quantiser's decisions are defined on correctly rounded fp32 steps, the value is not."""
    f = np.float32
    b = x.astype(f).reshape(x.shape[:-1] + (-1, 16))
    s = np.abs(b).max(-1) / f(6.0) * f(gs)
    grid = _e4m3_table()[:127]
    sf = grid[_nearest_even(s.astype(np.float64), grid)].astype(f)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(sf[..., None] > 0, b * (f(gs) / sf)[..., None], f(0))
    v = _E2M1[_nearest_even(np.abs(y).astype(np.float64), _E2M1)]
    return (np.copysign(v, y) * sf[..., None].astype(np.float64) / gs).reshape(x.shape)


def _exact_rows(pool, pages, h, P, D, at, gs, lo, hi):
    """Cached rows lo..hi of one request and head in float64, on the pool's device."""
    blk = pool[pages.long(), h].flatten(0, 1)                              # [pages * P/16, 18 D]
    codes = blk[:, at:at + 8 * D].reshape(-1, D // 2)[lo:hi]
    sf = blk[:, at + 8 * D:at + 9 * D].reshape(-1, D // 16)[lo:hi]
    dev = pool.device
    mag = torch.tensor(np.concatenate((_E2M1, -_E2M1)), device=dev)
    v = torch.empty(hi - lo, D, dtype=torch.float64, device=dev)
    v[:, 0::2], v[:, 1::2] = mag[(codes & 15).long()], mag[(codes >> 4).long()]
    scale = torch.tensor(_e4m3_table(), device=dev)[sf.long()]
    return v * scale.repeat_interleave(16, 1) / gs


def exact(c, seed):
    if c["op"] == "step":
        return None  # whole numbers
    st = prepare(c, seed)
    if c["op"] == "append":
        k, v = (st[n].float().cpu().numpy() for n in ("k", "v"))
        return {"k": _exact_append(k, K_GS), "v": _exact_append(v, V_GS)}
    if c["op"] == "norm":
        def rms(x):
            return (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        x, r = st["x"].double(), st["residual"].double()
        n = x if st["w_post"] is None else x / rms(x) * st["w_post"].double()
        r = 1.25 * r + 0.75 * (n if st["gate"] is None else n * st["gate"].double())
        return {"residual": r} if st["w_pre"] is None else {"residual": r, "out": r / rms(r) * st["w_pre"].double()}
    Hk, D, P, g = c["heads"], c["dim"], c["page"], c["qheads"] // c["heads"]
    ctx, new = _lengths(c)
    q = st["q"].double()
    out, lse, row = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV), 0
    for b, (a, n) in enumerate(zip(ctx, new)):
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            lo = max(0, a + i0 - c["window"] + 1) if c["window"] else 0
            hi = a + i1
            pos = torch.arange(a + i0, hi, device=DEV)[:, None]
            t = torch.arange(lo, hi, device=DEV)[None, :]
            hide = (t > pos) | ((t <= pos - c["window"]) if c["window"] else torch.zeros_like(t > pos))
            for h in range(Hk):
                pages = st["table"][b, :-(-hi // P)]
                key = _exact_rows(st["pool"], pages, h, P, D, 0, K_GS, lo, hi)
                val = _exact_rows(st["pool"], pages, h, P, D, 9 * D, V_GS, lo, hi)
                s = q[row + i0:row + i1, h * g:(h + 1) * g].transpose(0, 1) @ key.T / math.sqrt(D)
                s = s.masked_fill(hide, -math.inf)
                top = torch.logsumexp(s, -1)
                out[row + i0:row + i1, h * g:(h + 1) * g] = ((s - top[..., None]).exp() @ val).transpose(0, 1)
                lse[row + i0:row + i1, h * g:(h + 1) * g] = top.T
        row += n
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
