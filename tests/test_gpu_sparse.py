"""Rotation, block means, picks and sparse attention (include/moe_block.h) on the GPU against oracle/block.py.

Means and picks are compared bit for bit. Float bars, derived:

* rotation: the angle is off by at most 2^-31 turns of 2 pi (far positions) and the reduced angle by its rounding, 2^-24
  of at most pi / 4, twice (its conversion and its factor); the polynomials stop below 2^-28 and round a few times: sine
  and cosine are off by less than 2^-22, times the scale. Two products and a sum add 3 * 2^-24 of |a| + |b|: 2^-20
  (|a| + |b|) in all. bf16 outputs add 2^-8 |y|.
* stored keys: the quantiser is monotone in every step, so codes and scales lie between those of the true values moved
  by that error either way.
* attention: as in test_gpu_block.py.
"""
import numpy as np
import pytest
import torch

from oracle import block, nvfp4
from test_gpu_block import B, Scene, _bf16, _cuda

pytestmark = pytest.mark.gpu

ROPE_OFF = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _freq(R, theta=10000.0):
    return [theta ** (-2.0 * p / R) for p in range(R // 2)]


# ---------------------------------------------------------------- rotation

@pytest.mark.parametrize("pairs", ["half", "adjacent"])
@pytest.mark.parametrize("T,qh,kh,D,R,axes", [
    (1, 1, 0, 64, 64, 1), (1, 32, 8, 128, 128, 1), (3, 5, 1, 128, 64, 3), (7, 4, 2, 80, 80, 2), (5, 3, 3, 72, 72, 3),
    (9, 2, 1, 72, 48, 1), (4, 2, 2, 96, 34, 4), (6, 1, 1, 2, 2, 1), (130, 9, 3, 64, 32, 1), (2, 1, 1, 512, 512, 1),
    (33, 4, 1, 15, 6, 2)])
def test_rotation_matches_the_oracle(pairs, T, qh, kh, D, R, axes):
    from nvfp4_mixture_experts_moe_gb300 import Rope
    r = np.random.default_rng(T + D)
    axis = [int(a) for a in r.integers(0, axes, R // 2)]
    axis[-1] = axes - 1
    pos = r.integers(0, 200000, (axes, T))
    pos[:, 0] = 0
    pos[0, -1] = 2 ** 31 - 1
    if T > 2:
        pos[-1, 1] = -12345
    scale = 1.0 if T % 2 else 1.2079441
    q, k = _bf16((T, qh, D), 1, 3.0), _bf16((T, kh, D), 2)
    rope = Rope(R, inv_freq=_freq(R), axes=axis, pairs=pairs, scale=scale)
    p = _cuda(pos if axes > 1 else pos[0])
    for inverse in (False, True):
        got = rope(q.cuda(), p, k=k.cuda() if kh else None, inverse=inverse)
        for x, y in zip((q, k), got if kh else (got,)):
            want, size = block.rope(x.double().numpy(), pos, _freq(R), axis, pairs, float(np.float32(scale)), inverse)
            err = np.abs(y.double().cpu().numpy() - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + ROPE_OFF * size).all(), err.max()
            assert torch.equal(y[..., R:].cpu(), x[..., R:])


@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("D,R,pairs", [(128, 128, "half"), (128, 96, "adjacent"), (64, 20, "half"), (80, 80, "adjacent")])
def test_rotation_in_place_strided_and_on_a_stream(D, R, pairs, offset):
    """Columns of a fused product, in place, at any alignment, on another stream: the bits of the plain call."""
    from nvfp4_mixture_experts_moe_gb300 import Rope
    T, qh, kh = 37, 6, 2
    buf = torch.zeros(T * (qh + 2 * kh) * D + 8, dtype=torch.bfloat16, device="cuda")
    fused = buf[offset:offset + T * (qh + 2 * kh) * D].view(T, qh + 2 * kh, D)
    fused.copy_(_bf16((T, qh + 2 * kh, D), 5))
    before = fused.clone()
    rope = Rope(R, pairs=pairs)
    pos = torch.arange(1000, 1000 + T, dtype=torch.int32, device="cuda")
    q, k = rope(fused[:, :qh].contiguous(), pos, k=fused[:, qh:qh + kh].contiguous())
    q2, k2 = rope(fused[:, :qh], pos, k=fused[:, qh:qh + kh])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rope(fused[:, :qh], pos, k=fused[:, qh:qh + kh], out=fused[:, :qh], k_out=fused[:, qh:qh + kh], stream=s)
    torch.cuda.synchronize()
    for a, b, c in ((q, q2, fused[:, :qh]), (k, k2, fused[:, qh:qh + kh])):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert torch.equal(fused[:, qh + kh:], before[:, qh + kh:]) and not buf[:offset].any() and not buf[-8 + offset:].any()
    # a pair's NaN stays its own
    x = before[:, :qh].contiguous()
    x[3, 2, 1] = float("nan")
    y = rope(x, pos)
    i, j = (1, R // 2 + 1) if pairs == "half" else (0, 1)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[3, 2, i] = bad[3, 2, j] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], q[~bad])


def test_rotation_and_back_is_the_gradient():
    """<rope(x), y> = <x, inverse(y)> up to the two roundings: the backward pass is the rotation back."""
    from nvfp4_mixture_experts_moe_gb300 import Rope
    rope = Rope(128, sections=(16, 24, 24))
    x, y = _bf16((50, 3, 128), 1).cuda(), _bf16((50, 3, 128), 2).cuda()
    pos = torch.randint(0, 5000, (3, 50), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    a, b = (rope(x, pos).double() * y.double()).sum(-1), (x.double() * rope(y, pos, inverse=True).double()).sum(-1)
    bar = 2.0 ** -7 * (x.double().square().sum(-1) * y.double().square().sum(-1)).sqrt()   # 2^-8 of either, by Cauchy
    assert ((a - b).abs() <= bar).all()


# ------------------------------------------------- rotation into the cache

def _between(x, off, gs, codes, sf):
    """Whether stored codes and scales (of groups of 16 along the last axis) are those of values within ``off`` of x."""
    f = np.float32
    xg, og = x.reshape(x.shape[:-1] + (-1, 16)), off.reshape(off.shape[:-1] + (-1, 16))
    lo, hi = np.maximum(np.abs(xg) - og, 0).max(-1), (np.abs(xg) + og).max(-1)
    enc = lambda a: nvfp4.e4m3_encode((a.astype(f) / f(6.0) * f(gs)).astype(f)).astype(int)  # noqa: E731
    ok = (enc(lo * (1 - 2.0 ** -24)) <= sf) & (sf <= enc(hi * (1 + 2.0 ** -24)))
    s = nvfp4.e4m3_decode(sf).astype(f)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s > 0, f(gs) / s, f(0))[..., None]
    value = lambda v: nvfp4.e2m1_decode(nvfp4.e2m1_encode((v.astype(f) * r).astype(f)))  # noqa: E731
    got = nvfp4.e2m1_decode(codes).reshape(xg.shape)
    wide = og + 2.0 ** -24 * np.abs(xg)      # the fp32 rounding of the moved value
    return ok.all() and ((value(xg - wide) <= got) & (got <= value(xg + wide))).all()


@pytest.mark.parametrize("T,qh,kh,D,R,pairs,P,fused,axes", [
    (1, 1, 1, 64, 64, "half", 16, False, 1), (1, 32, 8, 128, 128, "half", 64, True, 1), (5, 6, 3, 64, 32, "half", 32, True, 3),
    (33, 4, 2, 128, 96, "half", 128, False, 2), (33, 4, 2, 128, 48, "adjacent", 16, True, 1), (130, 10, 5, 64, 16, "adjacent", 16, True, 3),
    (257, 8, 4, 128, 128, "adjacent", 32, True, 3), (70, 0, 2, 128, 64, "half", 16, False, 1), (600, 16, 8, 64, 64, "half", 64, False, 1)])
def test_rotated_append(T, qh, kh, D, R, pairs, P, fused, axes):
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, Rope
    r = np.random.default_rng(T)
    pages, k_gs, v_gs = -(-T // P) * 2 + 1, 150.0, 333.25
    qkv = _bf16((T, qh + 2 * kh, D), T, 2.0)
    qkv[0, qh, :16] = 0.0
    qkv[T // 2, qh] *= 1e4                             # past the calibrated range: saturates
    dev = qkv.cuda()
    parts = (dev[:, :qh], dev[:, qh:qh + kh], dev[:, qh + kh:])
    q, k, v = parts if fused else (x.contiguous() for x in parts)
    slots = r.permutation(pages * P)[:T]
    if T > 2:
        slots[T // 3] = -1
    pos = r.integers(0, 150000, (axes, T))
    axis = [i % axes for i in range(R // 2)]
    rope = Rope(R, inv_freq=_freq(R), axes=axis, pairs=pairs)
    c = Kv4Cache(pages, P, kh, D, k_gs, v_gs)
    c.pool.zero_()
    p = _cuda(pos if axes > 1 else pos[0])
    out = c.append_rotated(q if qh else None, k, v, _cuda(slots), p, rope)
    if qh:
        assert torch.equal(out, rope(q, p))            # the rotation by itself
    keep = slots >= 0
    ref = block.KvCache(pages, P, kh, D, k_gs, v_gs)
    kn, vn = qkv[:, qh:qh + kh].double().numpy(), qkv[:, qh + kh:].float().numpy()
    ref.append(np.zeros_like(vn), vn, slots)
    got = c.pool.cpu().numpy().reshape(pages, kh, P // 16, 18 * D)
    want = ref.pool()
    assert (got[..., 9 * D:] == want[..., 9 * D:]).all()      # values, bit for bit; nothing else written
    turned, size = block.rope(kn, pos, _freq(R), axis, pairs)
    codes = nvfp4.unpack(got[..., :8 * D].reshape(-1, D // 2)).reshape(pages, kh, P // 16, 16, D)
    sf = got[..., 8 * D:9 * D].reshape(pages, kh, P // 16, 16, D // 16)
    at = (slots[keep] // P, slice(None), slots[keep] % P // 16, slots[keep] % 16)
    assert _between(turned[keep], ROPE_OFF * size[keep], k_gs, codes[at], sf[at].astype(int))
    empty = np.ones((pages, P), bool)
    empty[slots[keep] // P, slots[keep] % P] = False
    assert not codes.transpose(0, 2, 3, 1, 4).reshape(pages, P, -1)[empty].any()
    assert int(c.status) == 0


def test_rotated_append_without_a_turn_stores_what_append_stores():
    """At position 0 nothing turns; NaNs and infinities are stored as append stores them; bad slots are reported."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, Rope
    T, kh, D, P = 20, 2, 128, 16
    k, v = _bf16((T, kh, D), 1).cuda(), _bf16((T, kh, D), 2).cuda()
    k[2, 0, 5], v[3, 1, 7], v[4, 0, 8] = float("nan"), float("nan"), float("-inf")
    slots = np.arange(T) + 3
    slots[5], slots[6] = -7, 64
    a, b = (Kv4Cache(4, P, kh, D, 400.0, 400.0) for _ in range(2))
    for c in (a, b):
        c.pool.fill_(0x55)
    a.append(k, v, _cuda(slots))
    out = torch.full((T, 4, D), 9.0, dtype=torch.bfloat16, device="cuda")
    q = _bf16((T, 4, D), 3).cuda()
    b.append_rotated(q, k, v, _cuda(slots), _cuda(np.zeros(T)), Rope(128), q_out=out)
    # the NaN's partner is spoilt too: 0 as well
    ka, va = a.read(_cuda(np.delete(slots, [2, 5, 6])))
    kb, vb = b.read(_cuda(np.delete(slots, [2, 5, 6])))
    assert torch.equal(ka, kb) and torch.equal(va, vb) and torch.equal(out, q)
    (k2, _), (k2a, _) = b.read(_cuda(slots[2:3])), a.read(_cuda(slots[2:3]))
    assert k2[0, 0, 5] == 0 and k2[0, 0, 69] == 0 and torch.equal(k2[0, 1], k2a[0, 1])
    assert int(a.status) == B().MOE_ERR_DEVICE and int(b.status) == B().MOE_ERR_DEVICE


# ------------------------------------------------------------ block means

def _index_of(scene, block_tokens):
    """An index whose unwritten rows are NaN, and the oracle's means per request: [blocks, heads, D]."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4BlockIndex
    index = Kv4BlockIndex(scene.cache, block_tokens)
    index.means.fill_(float("nan"))
    gs = scene.cache._fields[4]
    want = []
    for (kv, _), (keys, _) in zip(scene.lens, scene.vals):
        units = np.rint(keys * np.float64(np.float32(gs)) * 1024) / 1024     # code * scale, a whole number of 2^-10
        want.append(np.array([[block.block_mean(units[j * block_tokens:(j + 1) * block_tokens, h]) for h in range(scene.heads)]
                              for j in range(kv // block_tokens)]).reshape(-1, scene.heads, scene.D))
    return index, want


def _entry(scene, block_tokens, b, j):
    per = max(1, scene.P // block_tokens)
    tok = j * block_tokens
    return scene.table[b, tok // scene.P] * per + tok % scene.P // block_tokens


def _step_args(scene):
    return dict(cu_q=_cuda(scene.cu), kv_len=_cuda([kv for kv, _ in scene.lens]), block_table=_cuda(scene.table))


@pytest.mark.parametrize("block_tokens", [32, 64, 128])
@pytest.mark.parametrize("heads,D,P", [(1, 64, 16), (3, 128, 32), (9, 128, 64), (2, 64, 128)])
def test_means_match_the_oracle(block_tokens, heads, D, P):
    """Nothing new, one token that completes a block and one that does not, many blocks, a whole prompt, lengths of 0 and 1."""
    Bt = block_tokens
    lens = [(3 * Bt, 0), (3 * Bt, 1), (3 * Bt + 1, 1), (5 * Bt + 7, 3 * Bt), (4 * Bt, 4 * Bt), (0, 0), (1, 1), (Bt - 1, Bt - 1),
            (2 * Bt + 5, Bt + 6), (700, 1)]
    s = Scene(lens, heads, heads, D, P, seed=Bt)
    index, want = _index_of(s, Bt)
    index.update(**_step_args(s), max_q=s.max_q)
    means = index.means.double().cpu().numpy()
    new = np.zeros(len(means), bool)
    for b, (kv, n) in enumerate(lens):
        for j in range((kv - n) // Bt, kv // Bt):
            at = _entry(s, Bt, b, j)
            new[at] = True
            assert (means[at] == want[b][j]).all(), (b, j)
    assert np.isnan(means[~new]).all() and int(s.cache.status) == 0


def test_means_of_extreme_keys():
    """Saturated keys (the largest sums), zeros, one large element next to tiny ones: exact sums, ties to even."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4BlockIndex, Kv4Cache
    D, Bt = 64, 128
    k = torch.zeros(5, Bt, 1, D)
    k[0] = 1e30
    k[1, :, 0, 7] = -1e30
    k[1, 0, 0, 9] = 1e-3
    k[3] = torch.randn(Bt, 1, D, generator=torch.Generator().manual_seed(1)) * 1e-3
    k[4, :64, 0, :32] = 6.0
    k[4, 64:, 0, 3] = 0.5
    c = Kv4Cache(5, 128, 1, D, 448.0, 448.0)
    c.append(k.flatten(0, 1).to(torch.bfloat16).cuda(), k.flatten(0, 1).to(torch.bfloat16).cuda(), _cuda(np.arange(5 * Bt)))
    index = Kv4BlockIndex(c, Bt)
    index.update(_cuda([0, 5 * Bt]), _cuda([5 * Bt]), _cuda([range(5)]), max_q=5 * Bt)
    ref = block.KvCache(5, 128, 1, D, 448.0, 448.0)
    kn = k.flatten(0, 1).to(torch.bfloat16).float().numpy()
    ref.append(kn, kn, np.arange(5 * Bt))
    units = np.rint(ref.values(0, np.arange(5 * Bt))[:, 0] * 448.0 * 1024) / 1024
    want = np.array([block.block_mean(units[j * Bt:(j + 1) * Bt]) for j in range(5)])
    assert (index.means[:, 0].double().cpu().numpy() == want).all()


def test_means_report_bad_data():
    """Page ids outside the pool, lengths that cannot be: reported, and what is well is done."""
    lens = [(64, 64), (64, 64), (64, 64), (64, 64)]
    s = Scene(lens, 2, 2, 64, 32, seed=4)
    index, want = _index_of(s, 32)
    args = _step_args(s)
    table = args["block_table"].clone()
    table[0, 1], table[1, 0] = s.cache.num_pages, -1
    kv = _cuda([64, 64, 64, 10 ** 6])
    index.update(args["cu_q"], kv, table, max_q=64)
    assert int(s.cache.status) == B().MOE_ERR_DEVICE
    means = index.means.double().cpu().numpy()
    for b, j, good in ((0, 0, True), (0, 1, False), (1, 0, False), (1, 1, True), (2, 0, True), (2, 1, True), (3, 0, False)):
        got = means[_entry(s, 32, b, j)]
        assert (got == want[b][j]).all() if good else np.isnan(got).all(), (b, j)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.cache.status.zero_()
    index.update(**args, max_q=63, device_status=status)       # more new tokens than the bound
    assert int(status) == B().MOE_ERR_DEVICE and int(s.cache.status) == 0


# ----------------------------------------------------------------- picks

class Picker:
    """Random means on the index's grid under a table, no cache behind them."""

    def __init__(self, lens, qheads, heads, D, P, block_tokens, seed=0):
        from nvfp4_mixture_experts_moe_gb300 import Kv4BlockIndex, Kv4Cache
        r = np.random.default_rng(seed)
        self.lens, self.qheads, self.heads, self.D, self.P, self.Bt = lens, qheads, heads, D, P, block_tokens
        need = [-(-kv // P) for kv, _ in lens]
        self.W = max(need + [1]) + 1
        pages = sum(need) + 2
        perm, at = r.permutation(pages), 0
        self.table = np.full((len(lens), self.W), 2 ** 31 - 1)
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
        per = max(1, P // block_tokens)
        raw = r.normal(size=(pages * per, heads, D)) * 10.0 ** r.uniform(-2, 2, (pages * per, heads, 1))
        n = np.rint(raw / np.abs(raw).max(-1, keepdims=True) * r.integers(64, 129, (pages * per, heads, 1)))
        self.means = n * 2.0 ** r.integers(-4, 3, (pages * per, heads, 1))
        self.cache = Kv4Cache(pages, P, heads, D, 1.0, 1.0)
        self.index = Kv4BlockIndex(self.cache, block_tokens, means=torch.tensor(self.means).to(torch.float16).cuda())
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in lens])])
        self.total = int(self.cu[-1])
        self.q = _bf16((self.total, qheads, D), seed + 1)

    def args(self):
        return dict(cu_q=_cuda(self.cu), kv_len=_cuda([kv for kv, _ in self.lens]), block_table=_cuda(self.table),
                    max_q=max([n for _, n in self.lens] + [1]))

    def want(self, top, sink, local, rows=None):
        """Rows and their picks, [heads, top]."""
        per, g = max(1, self.P // self.Bt), self.qheads // self.heads
        for b, (kv, n) in enumerate(self.lens):
            pick = range(n) if rows is None or n <= rows else sorted(set(np.linspace(0, n - 1, rows).astype(int)))
            tok = np.arange(-(-kv // self.Bt)) * self.Bt
            page = self.table[b, tok // self.P]
            ok = (page >= 0) & (page < self.cache.num_pages)
            at = np.where(ok, page, 0) * per + tok % self.P // self.Bt
            for i in pick:
                row = int(self.cu[b]) + i
                q = self.q[row].double().numpy()
                out = np.full((self.heads, top), -1)
                for h in range(self.heads):
                    means = [self.means[e, h] if o else None for e, o in zip(at, ok)]
                    got = block.picks(q[h * g:(h + 1) * g], means, kv - n + i, self.Bt, top, sink, local)
                    out[h, :len(got)] = got
                yield row, out

    def check(self, top, sink, local, rows=None, **kw):
        got = self.index.select(self.q.cuda(), **self.args(), top=top, sink=sink, local=local, **kw).cpu().numpy()
        for row, want in self.want(top, sink, local, rows):
            assert (got[row] == want).all(), (row, got[row], want)


@pytest.mark.parametrize("qheads,heads,D,P,block_tokens", [
    (1, 1, 64, 16, 32), (8, 2, 128, 64, 64), (10, 2, 64, 128, 32), (16, 1, 128, 32, 128), (12, 4, 128, 16, 64)])
@pytest.mark.parametrize("top,sink,local", [(1, 0, 1), (4, 1, 2), (16, 2, 3), (64, 0, 1), (6, 3, 3)])
def test_single_queries_pick_the_oracles_blocks(qheads, heads, D, P, block_tokens, top, sink, local):
    """Lengths 1, around a block's end, as many blocks as are picked and one more, and long ones."""
    Bt = block_tokens
    lens = [(1, 1), (Bt, 1), (Bt + 1, 1), (0, 0), (top * Bt, 1), (top * Bt + 1, 1), ((top + 1) * Bt + 1, 1), (90 * Bt + 3, 1)]
    Picker(lens, qheads, heads, D, P, Bt, seed=top).check(top, sink, local)


@pytest.mark.parametrize("qheads,heads,D,P,block_tokens", [(4, 2, 128, 64, 64), (5, 1, 64, 16, 32), (16, 2, 64, 128, 128)])
@pytest.mark.parametrize("top,sink,local", [(8, 1, 2), (20, 0, 1)])
def test_prompts_pick_the_oracles_blocks(qheads, heads, D, P, block_tokens, top, sink, local):
    Bt = block_tokens
    lens = [(40 * Bt + 9, 150), (3, 3), (0, 0), (70 * Bt, 1), (30 * Bt, 65), (200, 200), (100 * Bt + 1, 4)]
    Picker(lens, qheads, heads, D, P, Bt, seed=top).check(top, sink, local, rows=24)


@pytest.mark.parametrize("n", [1, 40])
def test_a_long_context_is_ranked_whole(n):
    """More blocks than one pass of a CTA ranks."""
    Picker([(20011 * 32 + 5, n)], 2, 1, 64, 128, 32, seed=n).check(24, 1, 2, rows=3)


@pytest.mark.parametrize("n", [1, 33])
def test_equal_scores_take_the_lower_block(n):
    p = Picker([(60 * 32, n), (300 * 32, n)], 4, 2, 64, 32, 32)
    p.means[:] = 1.0
    p.means[::3] = 2.0
    p.index.means.copy_(torch.tensor(p.means))
    p.check(16, 1, 1)
    p.q.zero_()                      # every score 0
    p.check(16, 2, 1)
    p.q[:, :2] = float("nan")        # counts as 0
    p.q[:, 3, 5] = float("inf")
    p.q[:, 3, 6] = 3.0
    p.check(9, 0, 2)


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("mag", [1e-37, 1e-30, 1e30])
def test_queries_of_any_magnitude_pick_the_same(n, mag):
    """The largest sums of all (every product of the same sign) are exact too."""
    p = Picker([(200 * 32, n)], 16, 1, 128, 32, 32)
    p.means[:] = 128.0
    p.means[:, 0, 3] = np.arange(len(p.means)) % 128
    p.index.means.copy_(torch.tensor(p.means))
    p.q.fill_(1.999 * mag)
    p.check(12, 0, 1)


def test_picks_with_bad_device_data():
    """A page outside the pool scores lowest and is reported; impossible lengths are reported, their rows left alone."""
    p = Picker([(50 * 32, 1), (50 * 32, 3), (2000, 2)], 4, 2, 64, 32, 32)
    p.table[0, 7], p.table[1, 3] = -1, p.cache.num_pages
    p.check(16, 1, 1)
    assert int(p.cache.status) == B().MOE_ERR_DEVICE
    p = Picker([(50 * 32, 1), (50 * 32, 3), (2000, 2)], 4, 2, 64, 32, 32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    blocks = torch.full((p.total, 2, 16), 77, dtype=torch.int32, device="cuda")
    a = {**p.args(), "max_q": 2}
    p.index.select(p.q.cuda(), **a, top=16, sink=1, local=1, blocks=blocks, device_status=status)
    assert int(status) == B().MOE_ERR_DEVICE and int(p.cache.status) == 0
    got = blocks.cpu().numpy()
    for row, want in p.want(16, 1, 1):
        assert (got[row] == (77 if 1 <= row < 4 else want)).all()


def test_picks_of_strided_queries_and_padding():
    p = Picker([(50 * 32, 9), (90 * 32, 1)], 4, 2, 64, 32, 32)
    ref = p.index.select(p.q.cuda(), **p.args(), top=8, sink=1, local=1)
    wide = torch.full((p.total + 5, 7, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:p.total, 1:5] = p.q.cuda()
    blocks = torch.full((p.total + 5, 2, 8), 77, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.index.select(wide[:, 1:5], **p.args(), top=8, sink=1, local=1, blocks=blocks, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(blocks[:p.total], ref) and bool((blocks[p.total:] == 77).all())


# -------------------------------------------------------- sparse attention

def _lists(scene, block_tokens, top, seed=0, shuffle=False, drop=0.15):
    """Random lists: some places empty, neighbours share much; what a query cannot see is listed now and then."""
    r = np.random.default_rng(seed)
    out = np.full((scene.total, scene.heads, top), -1)
    for b, (kv, n) in enumerate(scene.lens):
        for h in range(scene.heads):
            base = r.permutation(-(-max(kv, 1) // block_tokens) + 1)
            for i in range(n):
                if i % 5 == 0:
                    r.shuffle(base[:max(2, len(base) // 2)])
                mine = base[:top].copy()
                mine[r.random(len(mine)) < drop] = -1
                mine = mine if shuffle else np.concatenate([np.sort(mine[mine >= 0]), mine[mine < 0]])
                out[scene.cu[b] + i, h, :len(mine)] = mine
    return out


def _check_sparse(scene, lists, block_tokens, out, lse=None, rows=None, scale=None):
    """As Scene.check, over the listed blocks' tokens."""
    g, scale = scene.qheads // scene.heads, scene.D ** -0.5 if scale is None else scale
    out = out.double().cpu().numpy()
    lse = None if lse is None else lse.double().cpu().numpy()
    for b, (kv, n) in enumerate(scene.lens):
        pick = range(n) if rows is None or n <= rows else sorted(set(np.linspace(0, n - 1, rows).astype(int)))
        for i in pick:
            row, pos = int(scene.cu[b]) + i, kv - n + i
            for h in range(scene.heads):
                tok = np.arange(max(pos + 1, 0))
                tok = tok[np.isin(tok // block_tokens, lists[row, h])]
                k, v = (x[tok, h] for x in scene.vals[b])
                for hh in range(h * g, (h + 1) * g):
                    o, l, pv, sabs = block.attention(scene.q[row, hh].double().numpy(), k, v, scale, len(tok) - 1)
                    ds = sabs * ((scene.D + 8) * 2.0 ** -22 + 2.0 ** -24) + 2.0 ** -20
                    vmax = np.abs(v).max() if len(tok) else 0.0
                    bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * ds) * pv + len(tok) * 2.0 ** -25 * vmax
                    err = np.abs(out[row, hh] - o)
                    assert (err <= bar).all(), (b, i, hh, err.max())
                    if lse is not None:
                        got = lse[row, hh]
                        assert (got == l) if l == -np.inf else abs(got - l) <= ds + 2.0 ** -22 * abs(l) + len(tok) * 2.0 ** -30


def _attend(scene, lists, block_tokens, **kw):
    kw = {"max_q": scene.max_q, "q": scene.q.cuda(), **kw}
    got = scene.cache.sparse_attention(kw.pop("q"), **_step_args(scene), blocks=_cuda(lists), block_tokens=block_tokens, **kw)
    assert int(scene.cache.status) == 0
    return got


@pytest.mark.parametrize("block_tokens,P", [(32, 16), (64, 128), (128, 32)])
@pytest.mark.parametrize("qheads,heads,D,top", [(1, 1, 64, 3), (8, 1, 128, 5), (8, 2, 64, 64), (12, 4, 128, 9), (10, 2, 128, 16),
                                                (16, 1, 64, 7), (24, 2, 128, 4)])
def test_sparse_single_tokens(block_tokens, P, qheads, heads, D, top):
    lens = [(1, 1), (0, 0), (block_tokens, 1), (block_tokens + 1, 1), (5 * block_tokens + 17, 1), (21 * block_tokens - 1, 1), (700, 1)]
    s = Scene(lens, qheads, heads, D, P, seed=top)
    lists = _lists(s, block_tokens, top, seed=top)
    out, lse = _attend(s, lists, block_tokens, want_lse=True)
    _check_sparse(s, lists, block_tokens, out, lse)


@pytest.mark.parametrize("shuffle", [False, True])
@pytest.mark.parametrize("qheads,heads,D,P,block_tokens,top", [
    (2, 2, 64, 16, 32, 40), (4, 1, 128, 64, 64, 6), (8, 2, 128, 16, 32, 12), (16, 2, 64, 32, 128, 5), (16, 1, 128, 128, 64, 9),
    (3, 1, 64, 64, 32, 17)])
def test_sparse_prompts(shuffle, qheads, heads, D, P, block_tokens, top):
    """Units that end at a request's end, units of several requests, rows that see nothing, single tokens among them."""
    lens = [(9 * block_tokens + 5, 30), (3, 3), (40, 1), (0, 0), (block_tokens * 20, 17), (64, 64), (300, 2), (1, 1)]
    s = Scene(lens, qheads, heads, D, P, seed=top + shuffle)
    lists = _lists(s, block_tokens, top, seed=top, shuffle=shuffle)
    out, lse = _attend(s, lists, block_tokens, want_lse=True)
    _check_sparse(s, lists, block_tokens, out, lse, rows=12)


def test_sparse_many_units():
    """More units than warps: each takes several in turn."""
    s = Scene([(1500, 700), (900, 900)], 8, 4, 64, 32, seed=3)
    lists = _lists(s, 32, 10, seed=1)
    out, _ = _attend(s, lists, 32)
    _check_sparse(s, lists, 32, out, rows=10)
    again, _ = _attend(s, lists, 32)
    assert torch.equal(out, again)


@pytest.mark.parametrize("n", [1, 7])
def test_all_blocks_listed_is_dense_attention(n):
    """Every block: the dense kernels' result up to the sum's order; listed twice or backwards: the same set."""
    s = Scene([(1000, n), (640, n), (31, min(n, 31))], 8, 2, 128, 64, seed=7)
    lists = np.tile(np.arange(16), (s.total, 2, 1))
    out, lse = _attend(s, lists, 64, want_lse=True)
    s.check(out, lse)
    twice = np.concatenate([lists, lists[..., ::-1]], -1)
    got, lse2 = _attend(s, twice, 64, want_lse=True)
    assert torch.equal(got, out) and torch.equal(lse, lse2)
    back, _ = _attend(s, lists[..., ::-1].copy(), 64)
    s.check(back)


def test_sparse_lists_with_nothing_and_with_nonsense():
    """Empty lists give zeros and -inf; ids past the position, past the table or negative are skipped."""
    s = Scene([(500, 4), (65, 1), (64, 64)], 4, 2, 64, 32, seed=2)
    lists = np.full((s.total, 2, 6), -1)
    lists[0, 0] = [2 ** 31 - 1, -2 ** 31, 10 ** 6, -1, 16, -5]
    lists[1, 1] = [3, 99, 3, -1, 0, 15]
    lists[4, 0] = [1, 2, 3, 4, 5, 6]
    out, lse = _attend(s, lists, 32, want_lse=True)
    _check_sparse(s, lists, 32, out, lse)
    assert not out[0].any() and bool((lse[0] == -float("inf")).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_query_spoils_its_own_sparse_row_only(value):
    s = Scene([(300, 5), (200, 1)], 8, 2, 64, 32, seed=9)
    lists = _lists(s, 32, 8, seed=2, drop=0.0)
    ref, ref_lse = _attend(s, lists, 32, want_lse=True)
    q = s.q.clone()
    q[2, 5, 3] = value
    out, lse = _attend(s, lists, 32, q=q.cuda(), want_lse=True)
    assert out[2, 5].isnan().all() and lse[2, 5].isnan()
    keep = torch.ones(s.total, 8, dtype=torch.bool)
    keep[2, 5] = False
    assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], ref_lse[keep])


def test_sparse_bad_device_data():
    """A page outside the pool hides its tokens; more rows than the bound are left alone; both are reported."""
    s = Scene([(320, 3), (320, 1), (320, 2)], 4, 2, 64, 32, seed=5)
    lists = np.tile(np.arange(10), (s.total, 2, 1))
    a = _step_args(s)
    a["block_table"][1, 4] = -3
    a["block_table"][2, 9] = s.cache.num_pages
    out, lse = s.cache.sparse_attention(s.q.cuda(), **a, blocks=_cuda(lists), block_tokens=32, max_q=3, want_lse=True)
    assert int(s.cache.status) == B().MOE_ERR_DEVICE
    cut = lists.copy()
    cut[3][cut[3] == 4] = -1
    cut[4:][cut[4:] == 9] = -1
    _check_sparse(s, cut, 32, out, lse)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.cache.status.zero_()
    out2 = torch.full_like(out, 5.0)
    s.cache.sparse_attention(s.q.cuda(), **_step_args(s), blocks=_cuda(lists), block_tokens=32, max_q=2, out=out2,
                             device_status=status)
    assert int(status) == B().MOE_ERR_DEVICE and int(s.cache.status) == 0
    assert bool((out2[:3] == 5.0).all())
    s.lens = [(320, 0), (320, 1), (320, 2)]
    s.cu = np.array([3, 3, 4, 6])
    _check_sparse(s, lists, 32, out2)


def test_sparse_strides_padding_and_streams():
    s = Scene([(500, 9), (90, 1)], 8, 2, 128, 64, seed=5, q_pad=3)
    lists = _lists(s, 64, 5, seed=3)
    ref, _ = _attend(s, lists, 64)
    wide = torch.full((s.total, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = s.q.cuda()
    out = torch.full((s.total, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    args = _step_args(s), _cuda(lists)
    torch.cuda.synchronize()
    s.cache.sparse_attention(wide[:, 2:10], **args[0], blocks=args[1], block_tokens=64, max_q=s.max_q, out=out, stream=other)
    torch.cuda.synchronize()
    n = int(s.cu[-1])
    assert torch.equal(out[:n], ref[:n]) and bool((out[n:] == 5.0).all())


def test_sparse_past_32_bit_offsets():
    """A pool of more than 2^32 bytes, its last pages in use."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4BlockIndex, Kv4Cache
    heads, D, P = 8, 128, 128
    pages = (1 << 32) // (P * heads * 144) + 50
    c = Kv4Cache(pages, P, heads, D, 448.0, 448.0)
    n = 3 * P
    table = np.array([[pages - 1, pages - 3, pages - 2]])
    k, v = _bf16((n, heads, D), 1), _bf16((n, heads, D), 2)
    slots = table[0, np.arange(n) // P] * P + np.arange(n) % P
    c.append(k.cuda(), v.cuda(), _cuda(slots))
    ref = block.KvCache(3, P, heads, D, 448.0, 448.0)
    ref.append(k.float().numpy(), v.float().numpy(), np.arange(n))
    vals = [ref.values(w, np.arange(n)) for w in (0, 1)]
    q = _bf16((1, heads, D), 3)
    lists = np.tile(np.array([0, 5, 7, 11]), (1, heads, 1))
    out, _ = c.sparse_attention(q.cuda(), _cuda([0, 1]), _cuda([n]), _cuda(table), _cuda(lists), block_tokens=32, max_q=1)
    tok = np.arange(n)[np.isin(np.arange(n) // 32, lists[0, 0])]
    for h in range(heads):
        o, _, pv, _ = block.attention(q[0, h].double().numpy(), vals[0][tok, h], vals[1][tok, h], D ** -0.5, len(tok))
        assert (np.abs(out[0, h].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -9 * pv).all()
    index = Kv4BlockIndex(c, 32)
    index.update(_cuda([0, n]), _cuda([n]), _cuda(table), max_q=n)
    units = np.rint(vals[0] * 448.0 * 1024) / 1024
    for j in (0, 5, 11):
        want = np.array([block.block_mean(units[j * 32:j * 32 + 32, h]) for h in range(heads)])
        assert (index.means[table[0, j // 4] * 4 + j % 4].double().cpu().numpy() == want).all()


# ------------------------------------------------------------- all together

def _serve(steps, graph):
    """Prompts, then single tokens: tables, rotated append, means, picks, attention. Outputs of each step."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4BlockIndex, Kv4Cache, KvStep, Rope
    Bn, qh, heads, D, P, W, T, Bt = 3, 8, 2, 64, 16, 60, 900, 32
    cache = Kv4Cache(Bn * W, P, heads, D, 400.0, 400.0)
    cache.pool.zero_()
    index, rope = Kv4BlockIndex(cache, Bt), Rope(D)
    index.means.zero_()
    t = KvStep(Bn, T, P, W)
    free = torch.arange(Bn * W, dtype=torch.int32, device="cuda")
    ctx, new = (torch.zeros(Bn, dtype=torch.int32, device="cuda") for _ in range(2))
    table, count = torch.zeros(Bn, W, dtype=torch.int32, device="cuda"), torch.full((1,), Bn * W, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(T, qh + 2 * heads, D, dtype=torch.bfloat16, device="cuda")

    def call():
        t.run(ctx, new, table, free, count)
        q = cache.append_rotated(qkv[:, :qh], qkv[:, qh:qh + heads], qkv[:, qh + heads:], t.slots, t.positions, rope)
        index.update(t.cu_q, t.kv_len, table, max_q=T)
        blocks = index.select(q, t.cu_q, t.kv_len, table, max_q=T, top=6, sink=1, local=2)
        o, lse = cache.sparse_attention(q, t.cu_q, t.kv_len, table, blocks, block_tokens=Bt, max_q=T, want_lse=True)
        ctx.copy_(t.kv_len)
        count.copy_(t.free_count)
        return q, blocks, o, lse
    g = None
    if graph:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = call()
        ctx.zero_(), count.fill_(Bn * W)
    got = []
    for i, n in enumerate(steps):
        qkv.copy_(_bf16(tuple(qkv.shape), 100 + i))
        new.copy_(_cuda(n))
        if graph:
            g.replay()
        else:
            outs = call()
        rows = sum(n)
        got.append([x[:rows].clone() for x in outs])
    assert int(cache.status) == 0 and int(t.status) == 0
    return got, (cache, table.clone(), ctx.clone())


STEPS = [[300, 7, 500], [1, 1, 1], [40, 0, 1], [1, 2, 1], [0, 300, 3]]


def test_operators_together_against_the_dense_oracle_rows():
    """Every step's rows, from the cache as it is: the oracle's attention over the blocks that were picked, and the picks
    of the index as it is."""
    got, (cache, table, _) = _serve(STEPS, False)
    ctx = np.zeros(3, int)
    P, D, heads, Bt = 16, 64, 2, 32
    ctxs = []
    for n in STEPS:
        ctxs.append(ctx.copy())
        ctx = ctx + n
    tb = table.cpu().numpy()
    vals = []
    for b in range(3):
        slots = _cuda(tb[b, np.arange(ctx[b]) // P] * P + np.arange(ctx[b]) % P)
        vals.append([x.double().cpu().numpy() for x in cache.read(slots)])   # bf16 of six-bit products / 400: off by 2^-8
    for n, c0, (q, blocks, o, lse) in zip(STEPS, ctxs, got):
        row = 0
        for b in range(3):
            for i in range(n[b]):
                if i in (0, n[b] - 1):
                    pos = c0[b] + i
                    for h in range(heads):
                        ids = blocks[row, h].cpu().numpy()
                        seen = pos // Bt + 1
                        assert (ids >= 0).sum() == min(6, seen) and (np.diff(ids[ids >= 0]) > 0).all()
                        assert 0 in ids and pos // Bt in ids and (seen < 2 or pos // Bt - 1 in ids)
                        tok = np.arange(pos + 1)
                        tok = tok[np.isin(tok // Bt, ids)]
                        k, v = vals[b][0][tok, h], vals[b][1][tok, h]
                        ref, l, pv, sabs = block.attention(q[row, 4 * h].double().cpu().numpy(), k, v, D ** -0.5, len(tok))
                        ds = 2.0 ** -8 * sabs      # the keys' rounding; the values' is 2^-8 of sum p |v|
                        assert (np.abs(o[row, 4 * h].double().cpu().numpy() - ref)
                                <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10 + 2 * ds) * pv).all()
                        assert abs(float(lse[row, 4 * h]) - l) <= ds + 2.0 ** -19
                row += 1


def test_operators_together_replay_from_a_graph():
    (a, _), (b, _) = _serve(STEPS, False), _serve(STEPS, True)
    for x, y in zip(a, b):
        assert all(torch.equal(i, j) for i, j in zip(x, y))
