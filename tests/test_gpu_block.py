"""The block operators (include/moe_block.h) on the GPU against oracle/block.py.

Tables and stored codes are compared bit for bit. Float bars, derived:

* attention: the output is rounded once to bf16 (half an ulp, 2^-9 |o|; 2^-8
  allows the binade's edge). A probability enters the second product as f16:
  2^-11 relative, at most 2^-25 absolute of the row's largest below f16's
  normal range (the largest is at least 2^-8 of the running maximum's 1). A
  score carries fp32 summation error, at most (D + 8) 2^-22 of |scale| sum |q k|
  (truncating accumulation included), plus 2^-20 for exp2 and its argument's
  rounding at |s| <= 16, 2^-24 |s| beyond; every probability then moves by
  twice that relative, and lse by once that.
* norms: fp32 sums of H squares in a tree (at most 2^-19 relative, the
  square root halves it) and a handful of rounded products; bf16 outputs add
  2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def B():
    from nvfp4_mixture_experts_moe_gb300 import binding
    return binding


def _cuda(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def _bf16(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


# ---------------------------------------------------------------- tables

@pytest.mark.parametrize("Bn,P,W,ctx,new,pad,short", [
    (1, 16, 4, 0, 1, 0, 0), (1, 64, 1, 63, 1, 5, 0), (64, 64, 70, 4000, 1, 0, 0), (33, 16, 40, 300, 200, 17, 0),
    (700, 32, 12, 200, 150, 100, 0), (4096, 16, 5, 40, 30, 3, 0), (50, 16, 30, 200, 100, 0, 40),
    (50, 16, 30, 200, 100, 9, 10 ** 6), (20, 128, 2, 250, 100, 0, 0)])
def test_step_matches_the_oracle(Bn, P, W, ctx, new, pad, short):
    from nvfp4_mixture_experts_moe_gb300 import KvStep
    r = np.random.default_rng(Bn + P)
    c = np.minimum(r.integers(0, ctx + 1, Bn), W * P)
    n = np.ones(Bn, int) if new == 1 else r.integers(0, new + 1, Bn)
    have = -(-c // P)
    pages = r.permutation(Bn * W + 7)
    table = np.full((Bn, W), -5)
    at = np.concatenate([[0], np.cumsum(have)])
    for b in range(Bn):
        table[b, :have[b]] = pages[at[b]:at[b + 1]]
    free = pages[at[-1]:]
    count = max(0, min(len(free), int(np.maximum(-(-(c + n) // P) - have, 0).sum()) + 2) - short)
    tokens = int(n.sum()) + pad
    ref = block.step(c, n, table, free, count, P, tokens)
    s = KvStep(Bn, tokens, P, W)
    tb = _cuda(table)
    for t in (s.slots, s.positions, s.kv_len, s.cu_q, s.free_count):
        t.fill_(-99)
    s.run(_cuda(c), _cuda(n), tb, _cuda(free), _cuda([count]))
    assert (tb.cpu().numpy() == ref["table"]).all()
    for name in ("kv_len", "cu_q", "slots", "positions"):
        assert (getattr(s, name).cpu().numpy() == ref[name]).all(), name
    assert int(s.free_count) == ref["free_count"]
    assert (int(s.status) == B().MOE_ERR_DEVICE) == ref["bad"]


def test_step_bad_lengths_and_short_bound():
    from nvfp4_mixture_experts_moe_gb300 import KvStep
    c, n = np.array([3, -4, 7, 2 ** 31 - 1, 0]), np.array([2, 1, -9, 2 ** 31 - 1, 6])
    table = np.arange(10).reshape(5, 2)
    ref = block.step(c[[0, 1, 2]], n[[0, 1, 2]], table[:3], np.arange(20, 40), 20, 16, 2)
    s = KvStep(3, 2, 16, 2)
    tb = _cuda(table[:3])
    s.run(_cuda(c[:3]), _cuda(n[:3]), tb, _cuda(np.arange(20, 40)), _cuda([20]))
    for name in ("kv_len", "cu_q", "slots", "positions"):
        assert (getattr(s, name).cpu().numpy() == ref[name]).all(), name
    assert int(s.status) == B().MOE_ERR_DEVICE and ref["bad"]
    # lengths whose sum passes 32 bits: that request is refused, the others are not
    s = KvStep(5, 8, 16, 2)
    tb = _cuda(table)
    s.run(_cuda(c), _cuda(n), tb, _cuda(np.arange(20, 40)), _cuda([20]))
    assert s.kv_len.cpu().tolist() == [5, 1, 7, 2 ** 31 - 1, 6]
    assert s.slots.cpu().tolist()[:3] == [0 * 16 + 3, 0 * 16 + 4, 20 * 0 + 39 * 16 + 0]
    assert int(s.free_count) == 18 and int(s.status) == B().MOE_ERR_DEVICE


def test_step_without_requests():
    from nvfp4_mixture_experts_moe_gb300 import KvStep
    s = KvStep(0, 3, 16, 2)
    s.run(_cuda([]), _cuda([]), _cuda(np.zeros((0, 2))), _cuda([4, 5]), _cuda([2]))
    assert s.cu_q.cpu().tolist() == [0] and s.slots.cpu().tolist() == [-1] * 3 and int(s.free_count) == 2
    assert int(s.status) == 0


# ----------------------------------------------------------------- cache

@pytest.mark.parametrize("T,heads,D,P,fused", [
    (1, 1, 64, 16, False), (1, 8, 128, 64, True), (5, 3, 64, 32, True), (33, 2, 128, 128, False),
    (130, 5, 64, 16, True), (257, 4, 128, 32, True)])
def test_append_stores_the_oracles_bytes_and_reads_back(T, heads, D, P, fused):
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
    pages = -(-T // P) * 2 + 1
    k_gs, v_gs = 150.0, 333.25
    qkv = _bf16((T, 4 * heads, D), T, 2.0)
    qkv[0, 0, :16] = 0.0                                   # an all-zero block
    qkv[0, 0, 16:32] = torch.linspace(-6, 6, 16).to(torch.bfloat16)
    qkv[-1, heads, 5] = float("nan")
    qkv[-1, -1, 7], qkv[-1, -1, 8] = float("inf"), float("-inf")
    qkv[T // 2, heads - 1] *= 1e4                          # past the calibrated range: saturates
    dev = qkv.cuda()
    k, v = (dev[:, :heads], dev[:, 3 * heads:]) if fused else (dev[:, :heads].contiguous(), dev[:, 3 * heads:].contiguous())
    r = np.random.default_rng(T)
    slots = r.permutation(pages * P)[:T] if T > 40 else np.arange(T) + 3
    slots[T // 3] = -1 if T > 2 else slots[T // 3]
    ref = block.KvCache(pages, P, heads, D, k_gs, v_gs)
    kn, vn = qkv[:, :heads].float().numpy(), qkv[:, 3 * heads:].float().numpy()
    with np.errstate(invalid="ignore"):
        ref.append(kn, vn, slots)
    c = Kv4Cache(pages, P, heads, D, k_gs, v_gs)
    c.pool.zero_()
    c.append(k, v, _cuda(slots))
    got = c.pool.cpu().numpy().reshape(pages, heads, P // 16, 18 * D)
    assert (got == ref.pool()).all()
    rk, rv = c.read(_cuda(slots))
    at = np.maximum(slots, 0)
    for out, which in ((rk, 0), (rv, 1)):
        want = np.where((slots >= 0)[:, None, None], ref.values(which, at), 0.0)
        # one fp32 reciprocal and product (2^-23), one rounding to bf16
        assert (np.abs(out.float().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()


def test_append_leaves_neighbours_alone_and_reports_bad_slots():
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
    c = Kv4Cache(2, 16, 2, 64, 10.0, 10.0)
    c.pool.fill_(0xA5)
    k = _bf16((3, 2, 64), 1).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(k, k, _cuda([-1, 32, 2 ** 31 - 1]), device_status=st)
    assert int(st) == B().MOE_ERR_DEVICE and bool((c.pool == 0xA5).all())
    st.zero_()
    c.append(k[:1], k[:1], _cuda([17]), device_status=st)
    assert int(st) == 0
    p = c.pool.cpu().numpy().reshape(2, 2, 18 * 64)
    touched = np.zeros_like(p, bool)
    for base, row in ((0, 32), (8 * 64, 4), (9 * 64, 32), (17 * 64, 4)):
        touched[1, :, base + row:base + 2 * row] = True    # token 1 of page 1
    assert (p[~touched] == 0xA5).all() and (p[touched] != 0xA5).any()
    rk, rv = c.read(_cuda([40, -3]), device_status=st)
    assert int(st) == B().MOE_ERR_DEVICE and not rk.any() and not rv.any()


def test_attention_past_32_bit_offsets():
    """A pool of more than 2^32 bytes, the request's pages at its end."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
    pages, P, heads, D = 30000, 128, 8, 128
    c = Kv4Cache(pages, P, heads, D, 100.0, 100.0)
    assert c.pool.numel() > 2 ** 32
    n = 200
    k, v = _bf16((n, heads, D), 1), _bf16((n, heads, D), 2)
    table = np.array([[pages - 1, pages - 2]])
    slots = table[0, np.arange(n) // P] * P + np.arange(n) % P
    c.append(k.cuda(), v.cuda(), _cuda(slots))
    ref = block.KvCache(2, P, heads, D, 100.0, 100.0)
    ref.append(k.float().numpy(), v.float().numpy(), np.arange(n))
    q = _bf16((1, heads, D), 3)
    out, _ = c.attention(q.cuda(), _cuda([0, 1]), _cuda([n]), _cuda(table), max_q=1)
    rk, rv = c.read(_cuda(slots[-3:]))
    assert np.allclose(rk.float().cpu().numpy(), ref.values(0, np.arange(n)[-3:]), rtol=2.0 ** -7)
    for h in range(heads):
        o, _, pv, _ = block.attention(q[0, h].double().numpy(), ref.values(0, np.arange(n))[:, h],
                                      ref.values(1, np.arange(n))[:, h], D ** -0.5, n - 1)
        assert (np.abs(out[0, h].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -9 * pv).all()


# ------------------------------------------------------------- attention

class Scene:
    """Requests (kv tokens, new tokens) with their pages, in the cache and in the oracle."""

    def __init__(self, lens, qheads, heads, D, P, seed=0, k_scale=1.0, q_pad=0, poison=True, q_scale=1.0):
        from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
        r = np.random.default_rng(seed)
        self.lens, self.qheads, self.heads, self.D, self.P = lens, qheads, heads, D, P
        k_gs, v_gs = 2688.0 / (6.0 * k_scale), 2688.0 / 5.5
        need = [-(-kv // P) for kv, _ in lens]
        self.W = max(need + [1]) + 1
        pages = sum(need) + 2
        perm = r.permutation(pages)
        self.table = np.full((len(lens), self.W), 2 ** 31 - 1)   # what lies past a request's pages is never used
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
        self.cache = Kv4Cache(pages, P, heads, D, k_gs, v_gs)
        # what was never appended decodes as NaN
        self.cache.pool.fill_(0xFF if poison else 0)
        self.vals = []
        for b, (kv, _) in enumerate(lens):
            k, v = _bf16((kv, heads, D), 7 * b + seed, k_scale), _bf16((kv, heads, D), 7 * b + seed + 1)
            k[:, :, 3] *= 3
            slots = self.table[b, np.arange(kv) // P] * P + np.arange(kv) % P
            if kv:
                self.cache.append(k.cuda(), v.cuda(), _cuda(slots))
            ref = block.KvCache(max(need[b], 1), P, heads, D, k_gs, v_gs)
            ref.append(k.float().numpy(), v.float().numpy(), np.arange(kv))
            self.vals.append((ref.values(0, np.arange(kv)), ref.values(1, np.arange(kv))))
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in lens])])
        self.total = int(self.cu[-1]) + q_pad
        self.max_q = max([n for _, n in lens] + [1])
        self.q = _bf16((self.total, qheads, D), seed + 99, q_scale)

    def run(self, q=None, **kw):
        kw = {"max_q": self.max_q, **kw}
        own = "ws" not in kw
        if own:
            kw["ws"] = self.cache.attention_workspace(self.total, len(self.lens), self.qheads, kw["max_q"], self.W)
        got = self.cache.attention(self.q.cuda() if q is None else q, _cuda(self.cu),
                                   _cuda([kv for kv, _ in self.lens]), _cuda(self.table), **kw)
        if own:   # no wait gave up, no bad data, and the workspace is as it has to be for the next call
            assert B().moe_get_device_status(kw["ws"]) == 0
            assert not kw["ws"][:B().MOE_KV4_WS_ZERO].any()
        return got

    def check(self, out, lse=None, scale=None, causal=True, window=0, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        g = self.qheads // self.heads
        out = out.double().cpu().numpy()
        lse = None if lse is None else lse.double().cpu().numpy()
        for b, (kv, n) in enumerate(self.lens):
            pick = range(n) if rows is None or n <= rows else sorted(set(np.linspace(0, n - 1, rows).astype(int)))
            for i in pick:
                pos = kv - n + i if causal else kv - 1
                for h in range(self.qheads):
                    k, v = (x[:, h // g] for x in self.vals[b])
                    row = self.cu[b] + i
                    o, l, pv, sabs = block.attention(self.q[row, h].double().numpy(), k, v, scale, pos, window)
                    ds = sabs * ((self.D + 8) * 2.0 ** -22 + 2.0 ** -24) + 2.0 ** -20
                    vmax = np.abs(v).max() if kv else 0.0
                    bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * ds) * pv + kv * 2.0 ** -25 * vmax
                    err = np.abs(out[row, h] - o)
                    assert (err <= bar).all(), (b, i, h, float((err - bar).max()), err.max())
                    if lse is not None:
                        got = lse[row, h]
                        assert (got == l) if l == -np.inf else abs(got - l) <= ds + 2.0 ** -22 * abs(l) + kv * 2.0 ** -30, \
                            (b, i, h, got, l)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("qheads,heads,D", [(1, 1, 64), (8, 1, 128), (8, 2, 64), (12, 4, 128), (10, 2, 128), (24, 1, 64)])
def test_single_tokens(P, qheads, heads, D):
    """One query each: lengths 0, 1, around a page's, a block's and a tile's end, and an idle slot."""
    lens = [(1, 1), (0, 0), (P, 1), (P + 1, 1), (15, 1), (16, 1), (17, 1), (31, 1), (33, 1), (127, 1), (129, 1),
            (300, 1), (64, 0), (1000, 1)]
    s = Scene(lens, qheads, heads, D, P, seed=P)
    out, lse = s.run(want_lse=True)
    s.check(out, lse)


@pytest.mark.parametrize("qheads,heads,D,P,n", [
    (8, 2, 128, 64, 2), (8, 2, 64, 16, 3), (4, 4, 128, 32, 7), (16, 2, 128, 128, 4), (5, 1, 64, 64, 6), (32, 1, 64, 16, 1),
    (40, 1, 128, 32, 1), (8, 1, 128, 16, 9)])
def test_drafted_tokens(qheads, heads, D, P, n):
    lens = [(n, n), (n + 1, n), (200, n), (513, n - 1), (64, n), (0, 0), (777, 1)]
    s = Scene(lens, qheads, heads, D, P, seed=n)
    out, lse = s.run(want_lse=True)
    s.check(out, lse)


@pytest.mark.parametrize("qheads,heads,D,P,lens,window", [
    (4, 1, 128, 64, [(130, 130)], 0), (4, 2, 64, 16, [(257, 257), (3, 3)], 0), (8, 8, 128, 32, [(300, 100), (129, 128)], 0),
    (2, 1, 64, 128, [(1000, 333), (64, 1), (0, 0), (500, 500)], 0), (6, 2, 128, 16, [(700, 200), (90, 90)], 64),
    (3, 3, 64, 64, [(520, 300)], 1), (7, 1, 128, 64, [(257, 129)], 130)])
def test_prompts(qheads, heads, D, P, lens, window):
    s = Scene(lens, qheads, heads, D, P, seed=len(lens) + D)
    out, lse = s.run(want_lse=True, window=window)
    s.check(out, lse, window=window, rows=40)


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
@pytest.mark.parametrize("window", [0, 200])
def test_row_tiles_of_every_kind_in_turn(D, P, window):
    """Few-row and many-row requests of one or a few tiles in one call, so that a CTA's range has pieces of all
    kinds one after another, single-tile ones among them."""
    lens = [((17 * b) % 390 + n, n) for b in range(36) for n in ((3, 5, 9, 20, 40, 70)[b % 6],)]
    s = Scene(lens, 8, 2, D, P, seed=D + window)
    for _ in range(3):
        out, lse = s.run(want_lse=True, window=window)
    s.check(out, lse, window=window, rows=3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[(700, 300), (130, 130)], [(3000, 9), (2000, 16)], [(400, 30), (5, 2), (999, 1)]])
def test_timeout_is_reported_and_the_next_call_is_exact(D, lens):
    """Every bounded wait gives up at once: the call records it, drains, frees its tensor memory and returns."""
    s = Scene(lens, 8, 2, D, 64, seed=D)
    ws = s.cache.attention_workspace(s.total, len(lens), 8, s.max_q, s.W)
    good = s.run(want_lse=True, ws=ws)
    assert B().moe_get_device_status(ws) == 0
    B().moe_debug_set(B().MOE_DEBUG_WAIT_LIMIT, 1)
    try:
        s.run(want_lse=True, ws=ws)
        torch.cuda.synchronize()
    finally:
        B().moe_debug_set(B().MOE_DEBUG_WAIT_LIMIT, 0)
    assert B().moe_get_device_status(ws) == B().MOE_ERR_TIMEOUT
    assert not ws[:B().MOE_KV4_WS_ZERO].any()
    again = s.run(want_lse=True, ws=ws)
    assert B().moe_get_device_status(ws) == 0
    assert all(torch.equal(x, y) for x, y in zip(good, again))


@pytest.mark.parametrize("D", [64, 128])
def test_long_context_is_split_and_joined(D):
    lens = [(20000, 1), (3, 1), (9999, 2)]
    s = Scene(lens, 8, 2, D, 64, seed=D)
    out, lse = s.run(want_lse=True)
    s.check(out, lse)
    again, lse2 = s.run(want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("window", [1, 5, 100])
def test_window_and_bidirectional(n, window):
    s = Scene([(333, n), (7, min(n, 7)), (100, n)], 8, 2, 128, 32, seed=window)
    out, lse = s.run(want_lse=True, window=window)
    s.check(out, lse, window=window)
    out, lse = s.run(want_lse=True, causal=False, scale=0.31)
    s.check(out, lse, causal=False, scale=0.31)


@pytest.mark.parametrize("n", [4, 70])
def test_rows_that_see_nothing(n):
    """More new tokens than the cache holds (a refused append): the first queries stand before position 0."""
    s = Scene([(2, n), (0, n), (150, n)], 8, 2, 64, 16, seed=n)
    out = torch.full((s.total, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = s.run(want_lse=True, out=out)
    s.check(out, lse)
    assert not out[:n - 2].any() and bool(torch.isneginf(lse[:n - 2]).all()) and not out[n:2 * n].any()


@pytest.mark.parametrize("qheads,heads,D,n", [(8, 2, 64, 1), (8, 2, 128, 4), (8, 2, 64, 9), (8, 2, 128, 40)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_query_spoils_its_own_row_only(qheads, heads, D, n, value):
    s = Scene([(300, n), (90, n)], qheads, heads, D, 32, seed=n)
    good, lse = s.run(want_lse=True)
    q = s.q.clone().cuda()
    row, head = n, 3                       # the second request's first token
    q[row, head, 5] = value
    out, lse2 = s.run(q=q, want_lse=True)
    keep = torch.ones(s.total, qheads, dtype=torch.bool, device="cuda")
    keep[row, head] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse2[keep], lse[keep])


@pytest.mark.parametrize("n,scale", [(1, 1.0), (1, 1e-3), (50, 2.0)])
def test_extreme_scores(n, scale):
    """Scores of hundreds (one token takes all) and scores near zero (all tokens alike)."""
    s = Scene([(400, n)], 8, 2, 128, 64, seed=3, k_scale=4.0)
    out, lse = s.run(want_lse=True, scale=scale)
    s.check(out, lse, scale=scale, rows=10)


@pytest.mark.parametrize("n", [1, 64])
@pytest.mark.parametrize("mag", [2.0 ** -30, 2.0 ** 20])
def test_queries_outside_f16_range(n, mag):
    s = Scene([(200, n)], 8, 2, 128, 64, seed=4, q_scale=mag)
    out, lse = s.run(want_lse=True, scale=0.088 / mag)
    s.check(out, lse, scale=float(np.float32(0.088 / mag)), rows=8)


@pytest.mark.parametrize("lens", [[(100, 1), (40, 1)], [(100, 60), (300, 1)]])
def test_strided_queries_padding_and_streams(lens):
    s = Scene(lens, 8, 2, 128, 64, seed=5, q_pad=3)
    ref, _ = s.run()
    wide = torch.full((s.total, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = s.q.cuda()
    out = torch.full((s.total, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    other = torch.cuda.Stream()
    args = [_cuda(s.cu), _cuda([kv for kv, _ in s.lens]), _cuda(s.table)]
    torch.cuda.synchronize()
    got, _ = s.cache.attention(wide[:, 2:10], *args, max_q=s.max_q, out=out, stream=other)
    torch.cuda.synchronize()
    n = int(s.cu[-1])
    assert torch.equal(got[:n], ref[:n]) and bool((got[n:] == 5.0).all())


def test_bad_device_data_is_reported():
    s = Scene([(100, 1), (50, 1), (70, 1)], 8, 2, 128, 16, seed=6)
    ws = s.cache.attention_workspace(s.total, 3, 8, 1)
    s.run(ws=ws)
    assert B().moe_get_device_status(ws) == 0
    good = s.table.copy()
    s.table[1, 2] = 10 ** 6                       # tokens 32..47 of request 1 count as hidden
    out, _ = s.run(ws=ws)
    assert B().moe_get_device_status(ws) == B().MOE_ERR_DEVICE
    k, v = s.vals[1]
    keep = np.r_[0:32, 48:50]
    for h in range(8):
        o, _, pv, _ = block.attention(s.q[1, h].double().numpy(), k[keep, h // 4], v[keep, h // 4], 128 ** -0.5, 99)
        assert (np.abs(out[1, h].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -9 * pv).all()
    s.table = good
    # more rows than the bound: that request's rows are left alone, the others are right
    t = Scene([(100, 3), (50, 1)], 8, 2, 128, 16, seed=7)
    out = torch.full((t.total, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    t.run(ws=ws, max_q=1, out=out)
    assert B().moe_get_device_status(ws) == B().MOE_ERR_DEVICE
    assert bool((out[:3] == 5.0).all())
    ref, _ = t.run()
    assert torch.equal(out[3:], ref[3:])
    # a length past the table is cut there
    u = Scene([(64, 1)], 8, 2, 128, 16, seed=8)
    lens = _cuda([10 ** 6])
    out, _ = u.cache.attention(u.q.cuda(), _cuda(u.cu), lens, _cuda(u.table[:, :4]), max_q=1, ws=ws)
    assert B().moe_get_device_status(ws) == B().MOE_ERR_DEVICE
    u.lens = [(64, 1)]
    u.check(out)


def test_workspace_serves_different_calls_in_turn():
    a = Scene([(3000, 1), (20, 1)], 8, 2, 128, 64, seed=9)
    b = Scene([(300, 120), (700, 5)], 8, 2, 64, 32, seed=10)
    wa = a.cache.attention_workspace(200, 4, 8, 200)
    wa[B().MOE_KV4_WS_ZERO:] = 0xFF
    ra, rb = a.run()[0], b.run()[0]
    for _ in range(3):
        assert torch.equal(a.run(ws=wa)[0], ra)
        assert torch.equal(b.run(ws=wa)[0], rb)
    assert B().moe_get_device_status(wa) == 0


def test_attention_in_a_cuda_graph():
    s = Scene([(500, 1), (40, 1)], 8, 2, 128, 64, seed=11)
    q, cu, kv, tb = s.q.cuda(), _cuda(s.cu), _cuda([k for k, _ in s.lens]), _cuda(s.table)
    ws = s.cache.attention_workspace(s.total, 2, 8, 1)
    out = torch.empty_like(q)
    ref, _ = s.cache.attention(q, cu, kv, tb, max_q=1, ws=ws, out=out)
    ref = ref.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.cache.attention(q, cu, kv, tb, max_q=1, ws=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_shapes_and_types_are_refused():
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, MoeError, block_norm
    c = Kv4Cache(2, 16, 2, 64, 1.0, 1.0)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (lambda: c.append(k.float(), k, i), lambda: c.append(k, k[:2], i), lambda: c.append(k, k, i.long()),
                lambda: c.append(k.cpu(), k, i), lambda: c.append(k[:, :1], k, i), lambda: c.read(i[::2]),
                lambda: c.append(k.transpose(1, 2).contiguous().transpose(1, 2), k, i),
                lambda: Kv4Cache(2, 8, 2, 64, 1.0, 1.0), lambda: Kv4Cache(2, 16, 2, 64, 1.0, 1.0, pool=c.pool[:-1]),
                lambda: c.attention(k, i[:2], i[:1], i[None], 3, out=k.float()),
                lambda: c.attention(k, i, i[:1], i[None], 3),
                lambda: block_norm(k[0], k[0].float().cpu()), lambda: block_norm(k[0, :1], k[0]),
                lambda: block_norm(k[0], k[0], gate=k[0, 0, :5])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(MoeError) as e:
        c.attention(torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda"), i[:2], i[:1], i[None], 1,
                    ws=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    assert e.value.status == B().MOE_ERR_UNSUPPORTED


# ----------------------------------------------------------------- norms

@pytest.mark.parametrize("T,H,gate,f32,post,pre,has_x", [
    (1, 64, None, False, True, True, True), (8, 4096, "channel", False, True, True, True),
    (3, 1000, "token", True, True, True, True), (5, 7168, "token", False, True, True, True),
    (2, 16384, "channel", True, True, True, True), (400, 2048, None, False, True, False, True),
    (7, 1, "token", False, True, True, True), (4, 333, "channel", False, False, True, True),
    (4, 12001, None, True, True, True, True), (9, 512, None, False, False, True, False),
    (320, 8192, "token", False, True, True, True), (310, 10240, "channel", False, True, True, True)])
def test_norm_matches_the_oracle(T, H, gate, f32, post, pre, has_x):
    from nvfp4_mixture_experts_moe_gb300 import block_norm
    x = _bf16((T, H), 1) if has_x else None
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(2)) * 2
    res = res if f32 else res.to(torch.bfloat16)
    g = None if gate is None else _bf16((T, H) if gate == "token" else (H,), 3)
    wp, wn = (_bf16((H,), 4) if post else None), (_bf16((H,), 5) if pre else None)
    dev = [None if t is None else t.cuda() for t in (x, res, g, wp, wn)]
    r, y = block_norm(dev[0], dev[1], gate=dev[2], w_post=dev[3], w_pre=dev[4], residual_scale=0.75,
                      branch_scale=-1.5, eps=1e-5, w_offset=1.0)
    n = [None if t is None else t.double().numpy() for t in (x, res, g, wp, wn)]
    rr, ry = block.block_norm(n[0], n[1], n[2], n[3], n[4], 0.75, -1.5, 1e-5, 1.0)
    size = 0.75 * np.abs(n[1]) + np.abs(rr - 0.75 * n[1])       # the terms the fp32 sum is made of
    err = np.abs(r.double().cpu().numpy() - rr)
    assert (err <= 2.0 ** -18 * size + (0 if f32 else 2.0 ** -8) * np.abs(rr)).all(), err.max()
    assert (y is None) == (not pre)
    if pre:
        gain = np.abs(ry) / np.maximum(np.abs(rr), 1e-30)
        err = np.abs(y.double().cpu().numpy() - ry)
        assert (err <= 2.0 ** -18 * (size * gain + np.abs(ry)) + 2.0 ** -8 * np.abs(ry) + 1e-30).all(), err.max()


# As many rows as make a CTA take several in turn, at widths that leave threads without a vector.
@pytest.mark.parametrize("T,H,gate,f32,post,pre,has_x", [
    (5000, 8, "token", True, True, True, True), (3001, 520, "channel", False, True, True, True),
    (1000, 2880, None, True, True, False, True), (997, 4096, "token", True, False, True, True),
    (913, 4104, "token", False, True, True, True), (640, 7168, "channel", False, True, True, True),
    (2000, 1536, None, False, False, True, False), (700, 8192, None, True, True, True, True),
    (3000, 77, "token", True, True, True, True), (1300, 2047, "token", False, True, True, True),
    (700, 5003, None, True, True, True, True), (400, 7001, "channel", False, False, True, True),
    (650, 4099, "token", True, True, False, True), (9, 8191, "token", True, True, True, True),
    (2500, 9, None, False, True, True, False), (1000, 130, "channel", True, False, False, True)])
def test_norm_of_many_rows_matches_the_oracle(T, H, gate, f32, post, pre, has_x):
    test_norm_matches_the_oracle(T, H, gate, f32, post, pre, has_x)


def test_norm_strides_alignment_in_place_and_stream():
    from nvfp4_mixture_experts_moe_gb300 import block_norm
    T, H = 6, 256
    x, res, w = _bf16((T, H), 1).cuda(), _bf16((T, H), 2).cuda(), _bf16((H,), 3).cuda()
    ref, refy = block_norm(x, res, w_post=w, w_pre=w)
    wide = torch.zeros(T, 2 * H + 24, dtype=torch.bfloat16, device="cuda")
    for at in (8, 1):   # 16-byte aligned rows, and rows that are not
        wide[:, at:at + H] = x
        wide[:, at + H + 8:at + 2 * H + 8] = res
        r, y = block_norm(wide[:, at:at + H], wide[:, at + H + 8:at + 2 * H + 8], w_post=w, w_pre=w)
        # the element-wise form sums in another order: fp32 rounding before the bf16 one
        assert torch.allclose(r.float(), ref.float(), rtol=2.0 ** -7) and torch.allclose(y.float(), refy.float(), rtol=2.0 ** -7)
    inplace = res.clone()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    r, y = block_norm(x, inplace, w_post=w, w_pre=w, residual_out=inplace, stream=other)
    torch.cuda.synchronize()
    assert r is inplace and torch.equal(r, ref) and torch.equal(y, refy)


@pytest.mark.parametrize("H,gap,at", [(130, 7, 1), (1001, 0, 0), (4095, 3, 5), (520, 1, 3), (64, 9, 2)])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_of_rows_at_any_offset(H, gap, at, f32):
    """Views into wider arrays, 2- or 4-byte aligned, the neighbours' bytes NaN; in place; against the copy's result."""
    from nvfp4_mixture_experts_moe_gb300 import block_norm
    T = 700
    wide = torch.full((T * (H + gap) + at + 3,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = lambda: wide.clone()[at:at + T * (H + gap)].view(T, H + gap)[:, :H]   # noqa: E731
    x, g = view(), view()
    x[:], g[:] = _bf16((T, H), 1).cuda(), _bf16((T, H), 2).cuda()
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(3)).cuda()
    wr = torch.full((T * (H + gap) + at,), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    r = wr[at:].view(T, H + gap)[:, :H]
    r[:] = res
    before = wr.clone()
    w = _bf16((H + 1,), 4).cuda()[1:]
    got, y = block_norm(x, r, gate=g, w_post=w, w_pre=w, eps=1e-5)
    n = [t.double().cpu().numpy() for t in (x, r, g, w)]
    rr, ry = block.block_norm(n[0], n[1], n[2], n[3], n[3], 1.0, 1.0, 1e-5, 0.0)
    size = np.abs(n[1]) + np.abs(rr - n[1])
    err = np.abs(got.double().cpu().numpy() - rr)
    assert (err <= 2.0 ** -18 * size + (0 if f32 else 2.0 ** -8) * np.abs(rr)).all(), err.max()
    gain = np.abs(ry) / np.maximum(np.abs(rr), 1e-30)
    err = np.abs(y.double().cpu().numpy() - ry)
    assert (err <= 2.0 ** -18 * (size * gain + np.abs(ry)) + 2.0 ** -8 * np.abs(ry) + 1e-30).all(), err.max()
    assert torch.equal(wr.view(torch.int32 if f32 else torch.int16), before.view(torch.int32 if f32 else torch.int16))
    if gap == 0 and at == 0:
        r2, y2 = block_norm(x, r, gate=g, w_post=w, w_pre=w, eps=1e-5, residual_out=r)
        assert r2 is r and torch.equal(r, got) and torch.equal(y2, y)


def test_norm_of_zero_rows_and_empty_batch():
    from nvfp4_mixture_experts_moe_gb300 import block_norm
    z = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    r, y = block_norm(z, z, w_post=w, w_pre=w)
    assert not r.any() and not y.any()
    r, y = block_norm(z[:0], z[:0], w_post=w, w_pre=w)
    assert r.shape == (0, 128) and y.shape == (0, 128)


# ----------------------------------------------------------------- all together

def test_calls_replay_from_a_graph():
    """A step's tables, rows in and out, attention of short and long requests, a norm: replays on other lengths give
    what direct calls give."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, KvStep, block_norm
    Bn, heads, D, P, W, T = 4, 2, 64, 16, 40, 400
    cache, plain = (Kv4Cache(Bn * W, P, heads, D, 400.0, 400.0) for _ in range(2))
    q, kv = _bf16((T, 8, D), 1).cuda(), _bf16((T, 2 * heads, D), 2).cuda()
    x, w = _bf16((T, 8 * D), 3).cuda(), _bf16((8 * D,), 4).cuda()
    free = torch.arange(Bn * W, dtype=torch.int32, device="cuda")

    def state():
        return dict(ctx=torch.zeros(Bn, dtype=torch.int32, device="cuda"), new=torch.zeros(Bn, dtype=torch.int32, device="cuda"),
                    table=torch.zeros(Bn, W, dtype=torch.int32, device="cuda"), step=KvStep(Bn, T, P, W),
                    count=torch.full((1,), Bn * W, dtype=torch.int32, device="cuda"))

    def call(c, s, ws):
        t = s["step"].run(s["ctx"], s["new"], s["table"], free, s["count"])
        c.append(kv[:, :heads], kv[:, heads:], t.slots)
        o, _ = c.attention(q, t.cu_q, t.kv_len, s["table"], max_q=300, ws=ws)
        r, y = block_norm(o.view(T, -1), x, w_post=w, w_pre=w)
        s["ctx"].copy_(t.kv_len)
        s["count"].copy_(t.free_count)
        return o, r, y
    got, ref = state(), state()
    ws, ws2 = (c.attention_workspace(T, Bn, 8, 300, W) for c in (cache, plain))
    call(cache, got, ws)   # once before the capture: kernels are loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(cache, got, ws)
    for s in (got, ref):
        s["ctx"].zero_()
        s["count"].fill_(Bn * W)
    for new in ([300, 3, 1, 90], [1, 1, 1, 1], [2, 130, 0, 4], [1, 0, 100, 1]):
        for s in (got, ref):
            s["new"].copy_(_cuda(new))
        graph.replay()
        want = call(plain, ref, ws2)
        torch.cuda.synchronize()
        n = sum(new)
        assert all(torch.equal(a[:n], b[:n]) for a, b in zip(outs, want)), new
    assert torch.equal(got["table"], ref["table"]) and B().moe_get_device_status(ws) == 0


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_blocks.py")
    spec = importlib.util.spec_from_file_location("decoder_blocks", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs_and_repeats():
    m = _example()
    new = [70, 0, 130]
    tokens = torch.randint(0, m.VOCAB, (200,), generator=torch.Generator().manual_seed(2)).cuda()
    runs = []
    for _ in range(2):
        s = m.Server(3, 256)
        t = s.step(tokens, new)
        got = [t]
        for _ in range(3):
            t = s.step(t, [1, 1, 1])
            got.append(t)
        assert int(s.tables.status) == 0 and s.length.cpu().tolist() == [73, 3, 133]
        assert all(B().moe_get_device_status(b.attn_ws) == 0 for b in s.blocks)
        runs.append(torch.stack(got).cpu())
    assert torch.equal(runs[0], runs[1])
    assert m.main() == 0


def test_prompt_in_pieces_gives_what_the_whole_prompt_gives():
    """The cached rows are the same bytes either way; the outputs differ by the roundings of two attention kernels
    (bf16 outputs, f16 probabilities, scores of at most some tens: 2^-6 of the largest value each element), carried
    through the projection, and by the bf16 roundings of the projection and of the residual."""
    m = _example()
    n = 150
    x = _bf16((n, m.HIDDEN), 5).cuda()
    h = _bf16((n, m.HIDDEN), 6).cuda()
    outs, rows = [], []
    for pieces in ([150], [100, 1, 1, 3, 45]):
        s = m.Server(1, 256)
        block_, at, hs = s.blocks[0], 0, []
        for c in pieces:
            t = s.tables.run(s.length, torch.tensor([c], dtype=torch.int32, device="cuda"), s.block_table, s.free_pages,
                             s.free_count)
            hs.append(block_.attend(h[at:at + c], x[at:at + c], t, s.block_table, c)[0])
            slots = t.slots[:c].clone()
            rows.append(block_.cache.read(slots))
            s.length.copy_(t.kv_len)
            s.free_count.copy_(t.free_count)
            at += c
        outs.append(torch.cat(hs).double())
    v = torch.cat([r[1] for r in rows[1:]])
    # a matrix product of another height may round its bf16 rows differently: rows that differ before quantisation
    same = [torch.equal(rows[0][i], torch.cat([r[i] for r in rows[1:]])) for i in (0, 1)]
    vmax = float(v.abs().max())
    da = block_.w_o.double().abs().sum(dim=1) * (2.0 ** -6 if all(same) else 2.0 ** -3) * vmax
    bar = da + 2.0 ** -7 * (outs[0] - h.double()).abs() + 2.0 ** -7 * outs[0].abs()
    assert ((outs[0] - outs[1]).abs() <= bar).all()
