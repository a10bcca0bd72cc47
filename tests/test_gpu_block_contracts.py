"""Corners of the block operators' contracts (include/moe_block.h) on the GPU."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block
from test_gpu_block import B, Scene, _bf16, _cuda, _example, built  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- bad queries

# Few rows in one range and cut across CTAs; many rows whole, of few rows (split over their tiles), and cut.
@pytest.mark.parametrize("qheads,heads,D,lens", [
    (8, 2, 64, [(300, 1), (90, 1)]), (8, 2, 128, [(90, 4), (300, 4)]), (8, 2, 128, [(3, 1), (20000, 1)]),
    (16, 1, 128, [(50, 1), (20000, 1)]), (16, 1, 64, [(9000, 1)]), (8, 2, 64, [(300, 40), (90, 40)]),
    (8, 2, 128, [(700, 300)]), (8, 2, 128, [(40, 9), (90, 9)]), (8, 2, 64, [(16000, 9)]), (8, 2, 128, [(16000, 70)])])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_query_gives_nan_rows(qheads, heads, D, lens, value):
    """A row with a NaN, or an infinity (inf * 0, inf - inf), is NaN in `out` and `lse`: zeros and -inf are what a row
    that sees nothing gives."""
    s = Scene(lens, qheads, heads, D, 32, seed=len(lens) + D)
    good, lse = s.run(want_lse=True)
    assert bool(torch.isfinite(good.float()).all()) and bool(torch.isfinite(lse).all())
    q = s.q.clone().cuda()
    row, head = s.total - 1, 3 % qheads        # the last request's last token
    q[row, head, 5] = value
    out, lse2 = s.run(q=q, want_lse=True)
    assert bool(torch.isnan(out[row, head]).all()) and bool(torch.isnan(lse2[row, head]))
    keep = torch.ones(s.total, qheads, dtype=torch.bool, device="cuda")
    keep[row, head] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse2[keep], lse[keep])


# ------------------------------------------------- tensors made for a stream

def _stream_of(other, handle):
    return other.cuda_stream if handle else other


def _queue_writes(*like):
    """Queues, behind some 50 ms of work on the current stream, writes over memory that is then given back to the
    allocator: tensors of these sizes made on this stream may take it, being ordered behind the writes."""
    torch.cuda.synchronize()
    made = [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in like for _ in range(8)]
    torch.cuda._sleep(100_000_000)
    for t in made:
        t.view(torch.uint8).fill_(0xFF)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("what", ["read", "attention", "block_norm"])
def test_outputs_on_another_stream_are_not_written_by_queued_work(what, handle):
    from nvfp4_mixture_experts_moe_gb300 import block_norm
    s = Scene([(100, 1), (300, 40)], 8, 2, 128, 64, seed=5)
    q, cu, kv, tb = s.q.cuda(), _cuda(s.cu), _cuda([k for k, _ in s.lens]), _cuda(s.table)
    ws = s.cache.attention_workspace(s.total, 2, 8, s.max_q, s.W)
    slots = _cuda(s.table[1, 0] * 64 + np.arange(50))
    x, w = _bf16((50, 1024), 1).cuda(), _bf16((1024,), 2).cuda()
    call = {"read": lambda st: s.cache.read(slots, stream=st),
            "attention": lambda st: s.cache.attention(q, cu, kv, tb, max_q=s.max_q, want_lse=True, ws=ws, stream=st),
            "block_norm": lambda st: block_norm(x, x, w_post=w, w_pre=w, stream=st)}[what]
    want = [t.clone() for t in call(None)]
    other = torch.cuda.Stream()
    _queue_writes(*want)
    got = call(_stream_of(other, handle))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("handle", [False, True])
def test_workspace_for_another_stream_is_not_written_by_queued_work(handle):
    s = Scene([(20000, 1), (300, 1)], 8, 2, 128, 64, seed=5)
    size = s.cache.attention_workspace(s.total, 2, 8, 1, s.W)
    other = torch.cuda.Stream()
    _queue_writes(size)
    ws = s.cache.attention_workspace(s.total, 2, 8, 1, s.W, stream=_stream_of(other, handle))
    torch.cuda.synchronize()
    assert not ws[:B().MOE_KV4_WS_ZERO].any()


@pytest.mark.parametrize("handle", [False, True])
def test_own_workspace_is_zeroed_on_the_calls_stream(handle):
    """Joins across CTAs count arrivals in the workspace: zeroed late, they never run."""
    s = Scene([(20000, 1), (300, 1)], 8, 2, 128, 64, seed=5)
    want, _ = s.run()
    args = (s.q.cuda(), _cuda(s.cu), _cuda([k for k, _ in s.lens]), _cuda(s.table))
    out = torch.zeros_like(want)
    used = [s.cache.attention_workspace(s.total, 2, 8, 1, s.W) for _ in range(8)]
    for t in used:
        t.fill_(0xFF)
    del used, t
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    s.cache.attention(*args, max_q=1, out=out, stream=_stream_of(other, handle))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_given_back_on_the_current_stream_are_not_reused_early(handle):
    """The caller waits for the other stream, queues a use and drops the tensors; the next call must not write them."""
    s = Scene([(300, 1)], 1, 1, 64, 64, seed=2)
    a, b = _cuda(s.table[0, 0] * 64 + np.arange(64)), _cuda(s.table[0, 1] * 64 + np.arange(64))
    other = torch.cuda.Stream()
    st = _stream_of(other, handle)
    want = [t.clone() for t in s.cache.read(a)]
    torch.cuda.synchronize()
    got = s.cache.read(a, stream=st)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(100_000_000)
    use = [t.clone() for t in got]
    del got
    for _ in range(4):
        s.cache.read(b, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(use, want))


def test_default_stream_by_its_handle():
    s = Scene([(300, 1)], 1, 1, 64, 64, seed=2)
    want, _ = s.run()
    args = (s.q.cuda(), _cuda(s.cu), _cuda([300]), _cuda(s.table))
    torch.cuda.synchronize()
    got, _ = s.cache.attention(*args, max_q=1, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------- windows

@pytest.mark.parametrize("n", [4, 100, 300])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 60, 2 ** 31 - 200])
def test_windows_near_the_largest_integer(n, window):
    """More query rows than cached tokens (a refused append) and a window that hides nothing."""
    s = Scene([(2, n), (0, n), (10, n), (150, n)], 8, 2, 64, 16, seed=n)
    ref, l0 = s.run(want_lse=True)
    out, lse = s.run(want_lse=True, window=window)
    s.check(out, lse, rows=20)
    assert torch.equal(out, ref) and torch.equal(lse, l0)


class Windowed(Scene):
    """Only what some query sees was ever appended: NaN lies before it in its page, and the pages before are given
    back: entry -1, or a page that nothing was appended to."""

    def __init__(self, lens, window, blank, *a, **kw):
        super().__init__(lens, *a, **kw)
        pool = self.cache.pool.view(-1, self.heads, self.P // 16, 18 * self.D)
        blank_page = sorted(set(range(pool.shape[0])) - set(self.table[self.table < pool.shape[0]].tolist()))[0]
        self.shown = 0
        for b, (kv, n) in enumerate(lens):
            first = max(0, kv - n + 1 - window)
            self.shown += first
            for j in range(first // self.P + 1):
                if (j + 1) * self.P <= first:
                    self.table[b, j] = blank_page if blank else -1
                    continue
                page = self.table[b, j]
                for t in range(j * self.P, first):
                    blk, r = t % self.P // 16, t % 16
                    for base, row in ((0, self.D // 2), (8 * self.D, self.D // 16), (9 * self.D, self.D // 2),
                                      (17 * self.D, self.D // 16)):
                        pool[page, :, blk, base + r * row:base + (r + 1) * row] = 0xFF


@pytest.mark.parametrize("qheads,heads,D,P", [(8, 2, 128, 16), (8, 2, 64, 16), (4, 4, 64, 32), (16, 2, 128, 32),
                                              (5, 1, 128, 64), (32, 2, 64, 64), (4, 1, 128, 128)])
@pytest.mark.parametrize("n,window", [(1, 1), (1, 100), (2, 37), (9, 100), (100, 100), (300, 333)])
@pytest.mark.parametrize("blank", [False, True])
def test_nothing_before_the_window_is_used(qheads, heads, D, P, n, window, blank):
    s = Windowed([(1000, n), (n + 3, n), (n + 555, n), (n + 129, n)], window, blank, qheads, heads, D, P, seed=n)
    assert s.shown
    out, lse = s.run(want_lse=True, window=window)   # and the status word stays clear
    s.check(out, lse, window=window, rows=5)


# ------------------------------------------------------------------- tables

def test_step_with_the_largest_bound_on_tokens():
    from nvfp4_mixture_experts_moe_gb300 import KvStep
    n = 2 ** 31 - 1
    s = KvStep(1, n, 16, 2)
    s.slots.fill_(7)
    s.positions.fill_(7)
    s.run(_cuda([5]), _cuda([3]), _cuda([[4, 0]]), _cuda([1]), _cuda([1]))
    assert s.slots[:4].tolist() == [69, 70, 71, -1] and s.positions[:4].tolist() == [5, 6, 7, 0]
    assert int(s.slots[3:].max()) == -1 and int(s.slots[3:].min()) == -1
    assert int(s.positions[3:].max()) == 0 and int(s.positions[3:].min()) == 0 and int(s.status) == 0


def test_step_reports_a_page_id_that_gives_no_slot():
    """A request whose last page has room, but whose entry is no page: its token has nowhere to go."""
    from nvfp4_mixture_experts_moe_gb300 import KvStep
    for entry in (-1, 2 ** 31 - 1):
        s = KvStep(2, 3, 16, 2)
        tb = _cuda([[entry, 0], [4, 0]])
        s.run(_cuda([5, 15]), _cuda([1, 2]), tb, _cuda([7]), _cuda([1]))
        assert s.slots.cpu().tolist() == [-1, 4 * 16 + 15, 7 * 16] and s.kv_len.cpu().tolist() == [6, 17]
        assert int(s.status) == B().MOE_ERR_DEVICE
    s = KvStep(1, 1, 16, 2)     # and one from the stack
    s.run(_cuda([16]), _cuda([1]), _cuda([[3, 0]]), _cuda([-2]), _cuda([1]))
    assert s.slots.cpu().tolist() == [-1] and int(s.status) == B().MOE_ERR_DEVICE


# ------------------------------------------------------------------ status

def test_cache_keeps_the_status_of_calls_that_were_given_no_place_for_it():
    s = Scene([(100, 1), (50, 1)], 8, 2, 128, 16, seed=6)
    c, k = s.cache, _bf16((2, 2, 128), 1).cuda()
    args = (s.q.cuda(), _cuda(s.cu), _cuda([100, 50]))
    c.attention(*args, _cuda(s.table), max_q=1)
    assert c.status.tolist() == [0]
    c.append(k, k, _cuda([-1, c.num_pages * 16]))
    assert c.status.tolist() == [B().MOE_ERR_DEVICE]
    c.attention(*args, _cuda(s.table), max_q=1)       # kept until the caller clears it
    assert c.status.tolist() == [B().MOE_ERR_DEVICE]
    c.status.zero_()
    c.read(_cuda([c.num_pages * 16]))
    assert c.status.tolist() == [B().MOE_ERR_DEVICE]
    c.status.zero_()
    s.table[1, 2] = 10 ** 6
    c.attention(*args, _cuda(s.table), max_q=1)
    assert c.status.tolist() == [B().MOE_ERR_DEVICE]
    c.status.zero_()
    own = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(k, k, _cuda([-1, c.num_pages * 16]), device_status=own)
    assert own.tolist() == [B().MOE_ERR_DEVICE] and c.status.tolist() == [0]


@pytest.mark.parametrize("group,n,launches", [(24, 1, 2), (17, 3, 2), (16, 1, 1), (16, 2, 3), (8, 2, 1), (8, 3, 3)])
def test_only_kernels_that_can_have_work_are_launched(group, n, launches):
    """One launch for at most 16 rows per key/value head, two for more, all three where a request may have either."""
    s = Scene([(100, n), (50, n)], group, 1, 64, 16, seed=6)
    args = (s.q.cuda(), _cuda(s.cu), _cuda([100, 50]), _cuda(s.table))
    ws = s.cache.attention_workspace(s.total, 2, group, n, s.W)
    before = B().lib().moe_kernel_launches()
    out, lse = s.cache.attention(*args, max_q=n, want_lse=True, ws=ws)
    assert B().lib().moe_kernel_launches() - before == launches
    s.check(out, lse)


def _to_bf16(x):
    """A Fraction to the nearest bf16 (normal range), ties to even."""
    if x == 0:
        return 0.0
    e = Fraction(2) ** (np.frexp(float(abs(x)))[1] - 8)
    return float(round(x / e) * e)      # round() of a Fraction is to even


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gs", [6.7855424880981445, 448.0, 333.25, 112.0])
def test_read_rounds_once(D, gs):
    """Every code with every scale: e2m1 * e4m3 / gs, exactly, to the nearest bf16."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
    from oracle import nvfp4
    gs = float(np.float32(gs))
    c = Kv4Cache(8, 16, 1, D, gs, gs)
    scale = (np.arange(128 * D // 16) % 127).astype(np.uint8).reshape(8, 16, D // 16)
    codes = np.tile(np.arange(16, dtype=np.uint8), (8, 16, D // 16))
    half = np.concatenate([nvfp4.pack(codes.reshape(-1, D)).reshape(8, -1), scale.reshape(8, -1)], axis=1)
    c.pool.copy_(torch.from_numpy(np.concatenate([half, half], axis=1).reshape(-1)))
    k, v = c.read(_cuda(np.arange(128)))
    mag = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    val = [Fraction(m) for m in mag] + [-Fraction(m) for m in mag]
    e4m3 = nvfp4.e4m3_decode(np.arange(127, dtype=np.uint8))
    want = {(s, i): _to_bf16(val[i] * Fraction(float(e4m3[s])) / Fraction(gs)) for s in range(127) for i in range(16)}
    ref = np.array([[want[int(s), i] for s in row for i in range(16)] for row in scale.reshape(128, -1)])
    assert (k[:, 0].double().cpu().numpy() == ref).all() and (v[:, 0].double().cpu().numpy() == ref).all()


# ------------------------------------------------------------------ example

def test_example_gives_idle_requests_no_token_and_takes_pages_back():
    m = _example()
    s = m.Server(3, 256)
    tokens = torch.randint(0, m.VOCAB, (200,), generator=torch.Generator().manual_seed(2)).cuda()
    first = s.step(tokens, [70, 0, 130])
    assert first[1].item() == -1 and (first[[0, 2]] >= 0).all()
    used = {0: set(s.block_table[0, :5].tolist()), 2: set(s.block_table[2, :9].tolist())}
    assert int(s.free_count) == m.NUM_PAGES - 5 - 9
    s.finish(2)
    assert s.length.cpu().tolist() == [70, 0, 0] and int(s.free_count) == m.NUM_PAGES - 5
    assert set(s.free_pages[:int(s.free_count)].tolist()) == set(range(m.NUM_PAGES)) - used[0]
    # the freed pages serve another request, whose tokens are those of a server that never held the first one
    again = s.step(tokens[:130], [0, 130, 0])
    assert again[0].item() == -1 and again[2].item() == -1 and int(s.free_count) == m.NUM_PAGES - 5 - 9
    alone = m.Server(3, 256).step(tokens[:130], [0, 130, 0])
    assert torch.equal(again, alone)
    s.finish(0)
    s.finish(1)
    assert int(s.free_count) == m.NUM_PAGES and sorted(s.free_pages.tolist()) == list(range(m.NUM_PAGES))
    assert int(s.tables.status) == 0


# --------------------------------------------------------- long contexts

@pytest.mark.parametrize("qheads,heads,D,n", [(16, 1, 128, 1), (12, 1, 128, 1), (8, 1, 128, 2), (16, 2, 128, 2),
                                              (16, 1, 64, 1), (24, 1, 128, 1), (32, 1, 64, 1), (32, 2, 128, 1)])
def test_long_contexts_of_wide_groups(qheads, heads, D, n):
    """Nine to sixteen rows (partials that do not fit a stage go to memory), and groups of more than sixteen heads:
    cut across warps and CTAs, whole beside them, twice the same."""
    lens = [(20000, n), (n, n), (7001, n), (333, n)]
    s = Scene(lens, qheads, heads, D, 64, seed=qheads + D)
    out, lse = s.run(want_lse=True)
    s.check(out, lse)
    again, lse2 = s.run(want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    out, lse = s.run(want_lse=True, window=5000)
    s.check(out, lse, window=5000)


# ------------------------------------------------------- prompts in pieces

def test_attention_of_a_prompt_in_pieces_row_by_row():
    """A prompt fed whole, and fed in pieces through a block's tables and cache: the cached bytes are equal, and every
    output element is within its own row's bar of the exact value. A piece that attended to itself alone, or to
    nothing, would be outside the same bars."""
    m = _example()
    n, P = 150, m.PAGE
    qkv = _bf16((n, m.Q_HEADS + 2 * m.KV_HEADS, m.DIM), 5).cuda()       # one projection for both
    ranges = lambda cuts: list(zip(np.cumsum([0] + cuts[:-1]), np.cumsum(cuts)))   # noqa: E731
    pieces = ranges([100, 1, 1, 3, 45])
    got, rows = [], []
    for cut in ([(0, n)], pieces):
        s = m.Server(1, 256)
        cache = s.blocks[0].cache
        outs, slots = [], []
        for a, b in cut:
            t = s.tables.run(s.length, _cuda([b - a]), s.block_table, s.free_pages, s.free_count)
            pos = t.positions[:b - a]
            assert pos.cpu().tolist() == list(range(a, b))
            k = m.rotate(qkv[a:b, m.Q_HEADS:m.Q_HEADS + m.KV_HEADS], pos)
            cache.append(k, qkv[a:b, m.Q_HEADS + m.KV_HEADS:], t.slots[:b - a])
            o, _ = cache.attention(m.rotate(qkv[a:b, :m.Q_HEADS], pos), t.cu_q, t.kv_len, s.block_table, max_q=int(b - a),
                                   ws=s.blocks[0].attn_ws)
            outs.append(o)
            slots.append(t.slots[:b - a].clone())
            s.length.copy_(t.kv_len)
            s.free_count.copy_(t.free_count)
        got.append(torch.cat(outs).double().cpu().numpy())
        rows.append([x.cpu() for x in cache.read(torch.cat(slots))])
        assert B().moe_get_device_status(s.blocks[0].attn_ws) == 0
    assert torch.equal(rows[0][0], rows[1][0]) and torch.equal(rows[0][1], rows[1][1])

    pos = torch.arange(n, device="cuda")
    ref = block.KvCache(-(-n // P), P, m.KV_HEADS, m.DIM, 2688 / 6, 2688 / 6)
    k = m.rotate(qkv[:, m.Q_HEADS:m.Q_HEADS + m.KV_HEADS], pos)
    ref.append(k.float().cpu().numpy(), qkv[:, m.Q_HEADS + m.KV_HEADS:].float().cpu().numpy(), np.arange(n))
    keys, vals = (ref.values(w, np.arange(n)) for w in (0, 1))
    q = m.rotate(qkv[:, :m.Q_HEADS], pos).double().cpu().numpy()
    start = np.zeros(n, int)
    for a, b in pieces:
        start[a:b] = a
    alone = 0                                  # later rows whose piece alone gives something else
    for i in range(n):
        for h in range(m.Q_HEADS):
            kv, v = keys[:, h * m.KV_HEADS // m.Q_HEADS], vals[:, h * m.KV_HEADS // m.Q_HEADS]
            o, _, pv, sabs = block.attention(q[i, h], kv, v, m.DIM ** -0.5, i)
            ds = sabs * ((m.DIM + 8) * 2.0 ** -22 + 2.0 ** -24) + 2.0 ** -20
            bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * ds) * pv + n * 2.0 ** -25 * np.abs(v).max()
            for g in got:
                assert (np.abs(g[i, h] - o) <= bar).all(), (i, h)
            if start[i]:
                own, *_ = block.attention(q[i, h], kv[start[i]:], v[start[i]:], m.DIM ** -0.5, i - start[i])
                assert (np.abs(o) > bar).any()          # nothing at all would be seen
                alone += (np.abs(own - o) > bar).any()
    assert alone == (n - 100) * m.Q_HEADS


@pytest.mark.parametrize("D,group,n,batch", [(64, 1, 1, 320), (128, 1, 1, 320), (128, 4, 4, 320), (64, 4, 40, 30), (128, 4, 40, 30)])
@pytest.mark.parametrize("gap", [14.3, 20.6, 24.6, 27.6])
def test_small_probabilities_are_kept(D, group, n, batch, gap):
    """One token 2^gap above 3000 others that are alike, with a value of zero: the output is the others' share. Enough
    requests (on the same pages) that a warp, or a CTA, goes through a context alone. A probability enters the second
    product as f16, the running maximum's as 2^7 or more: 2^-11 relative, at most 2^-25 / 2^7 absolute."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
    heads, kv, P = 8, 3000, 64
    W = -(-kv // P)
    k, v = torch.zeros(kv, heads, D), torch.full((kv, heads, D), 0.75)
    k[0], v[0] = 1.0, 0.0
    v[1:, :, 1::2] = _bf16((kv - 1, heads, D // 2), 3).float()
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c = Kv4Cache(W, P, heads, D, 448.0, 448.0)
    c.append(k.cuda(), v.cuda(), _cuda(np.arange(kv)))
    ref = block.KvCache(W, P, heads, D, 448.0, 448.0)
    ref.append(k.float().numpy(), v.float().numpy(), np.arange(kv))
    keys, vals = (ref.values(w, np.arange(kv)) for w in (0, 1))
    q = torch.ones(batch * n, heads * group, D, dtype=torch.bfloat16)
    scale = float(np.float32(gap * np.log(2) / keys[0, 0].sum()))
    table = _cuda(np.tile(np.arange(W), (batch, 1)))
    out, lse = c.attention(q.cuda(), _cuda(np.arange(batch + 1) * n), _cuda([kv] * batch), table, max_q=n, want_lse=True,
                           scale=scale)
    assert c.status.tolist() == [0]
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in {0, n // 2, n - 1}:
        for h in range(heads):
            o, l, pv, sabs = block.attention(q[i, 0].double().numpy(), keys[:, h], vals[:, h], scale, kv - n + i)
            ds = sabs * ((D + 8) * 2.0 ** -22 + 2.0 ** -24) + 2.0 ** -20
            bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * ds) * pv + kv * 2.0 ** -32 * np.abs(vals).max()
            rows = slice(i, batch * n, n), slice(h * group, (h + 1) * group)
            assert (np.abs(out[rows] - o) <= bar).all(), (i, h, np.abs(out[rows] - o).max(), bar.max(), np.abs(o).max())
            assert (np.abs(lse[rows] - l) <= ds + 2.0 ** -22 * abs(l) + kv * 2.0 ** -30).all()


# -------------------------------------------------------------------- norms

@pytest.mark.parametrize("T,H,gate,f32", [
    (152, 8192, "channel", False), (153, 8192, "token", False), (160, 5128, "token", True), (304, 5120, "token", True),
    (305, 5120, "token", True), (170, 6144, None, False), (400, 1024, "token", False), (1217, 1024, "channel", True),
    (600, 2048, "token", True), (153, 7688, "token", True), (170, 7688, "channel", True), (170, 8200, "token", False)])
def test_norm_on_either_side_of_each_variants_sizes(T, H, gate, f32):
    from test_gpu_block import test_norm_matches_the_oracle as check
    check(T, H, gate, f32, True, True, True)


# ------------------------------------------------------------- back to back

@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_steps_back_to_back_read_what_was_just_appended(D, P):
    """Tokens appended into blocks that the attention before has just read, with long and short requests in each call
    (two kernels that overlap): queued without a wait, and with one after each call."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, KvStep
    Bn, heads, W, steps = 6, 2, 64, 40
    new = np.random.default_rng(D).choice([1, 2, 3, 9, 17], (steps, Bn))
    new[:, 0], new[:, 1] = 1, 17                    # both kinds in every call
    total = new.sum(1)
    q, kv = _bf16((int(total.sum()), 8, D), 1).cuda(), _bf16((int(total.sum()), 2 * heads, D), 2).cuda()
    counts = _cuda(new)
    runs = []
    for wait in (False, True):
        c = Kv4Cache(Bn * W * 128 // P, P, heads, D, 400.0, 400.0)
        s = KvStep(Bn, int(total.max()), P, W * 128 // P)
        table = torch.zeros(Bn, W * 128 // P, dtype=torch.int32, device="cuda")
        free = torch.arange(c.num_pages, dtype=torch.int32, device="cuda")
        left, length = _cuda([c.num_pages]), _cuda([0] * Bn)
        ws = c.attention_workspace(int(total.max()), Bn, 8, 17, table.shape[1])
        at, outs = 0, []
        for i in range(steps):
            n = int(total[i])
            s.run(length, counts[i], table, free, left)
            c.append(kv[at:at + n, :heads], kv[at:at + n, heads:], s.slots[:n])
            if wait:
                torch.cuda.synchronize()
            outs.append(c.attention(q[at:at + n], s.cu_q, s.kv_len, table, max_q=17, ws=ws)[0])
            length.copy_(s.kv_len)
            left.copy_(s.free_count)
            at += n
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert int(s.status) == 0 and B().moe_get_device_status(ws) == 0
        runs.append(torch.cat(outs))
    assert torch.equal(*runs)
