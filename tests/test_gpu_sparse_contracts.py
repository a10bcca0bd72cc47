"""The kernels for many rows of selection and sparse attention, either side of the rules that choose a kernel, and what
callers may do between and around the calls. Bars as in test_gpu_sparse.py."""
import numpy as np
import pytest
import torch

from oracle import block
from test_gpu_block import B, Scene, _bf16, _cuda, _example
from test_gpu_sparse import Picker, _attend, _check_sparse, _index_of, _lists, _step_args

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _launches(f):
    """Kernels that a call launches."""
    before = B().moe_kernel_launches()
    f()
    return B().moe_kernel_launches() - before


# ------------------------------------------------- sparse attention, many rows

LENS = [(900, 320), (33, 33), (500, 1), (0, 0), (700, 24), (640, 25), (64, 64), (400, 2)]


@pytest.mark.parametrize("qheads,heads,D,P,block_tokens,top,shuffle", [
    (32, 8, 128, 64, 64, 6, False), (32, 8, 64, 16, 32, 11, True), (16, 8, 128, 32, 128, 4, False), (16, 8, 64, 128, 64, 16, True),
    (40, 8, 128, 16, 32, 9, False), (64, 8, 64, 64, 128, 3, False), (128, 8, 128, 128, 32, 7, True), (21, 7, 128, 32, 64, 64, False),
    (104, 8, 64, 64, 64, 5, False)])
def test_prompts_in_tiles_of_many_rows(qheads, heads, D, P, block_tokens, top, shuffle):
    """Groups that fill 128 rows and groups that do not, units that several requests share, requests of the other kernel
    among them, rows that see nothing, lists in any order."""
    s = Scene(LENS, qheads, heads, D, P, seed=top + shuffle)
    lists = _lists(s, block_tokens, top, seed=top, shuffle=shuffle)
    lists[5], lists[int(s.cu[1]) + 3] = -1, -1
    lists[int(s.cu[6]):int(s.cu[7]), 0] = -1            # a whole unit that has nothing
    got = []
    assert _launches(lambda: got.append(_attend(s, lists, block_tokens, want_lse=True))) == 2
    out, lse = got[0]
    keep = range(0, heads, 3)                           # of the heads, every third (the oracle takes its time)
    s2 = Scene.__new__(Scene)
    s2.__dict__.update(s.__dict__)
    g = qheads // heads
    s2.heads, s2.qheads = len(keep), len(keep) * g
    rows = [h * g + i for h in keep for i in range(g)]
    s2.q = s.q[:, rows]
    s2.vals = [(k[:, list(keep)], v[:, list(keep)]) for k, v in s.vals]
    _check_sparse(s2, lists[:, list(keep)], block_tokens, out[:, rows], lse[:, rows], rows=9)
    again, _ = _attend(s, lists, block_tokens, want_lse=True)
    assert torch.equal(out, again)


@pytest.mark.parametrize("n,many", [(24, False), (25, True), (383, False), (384, True)])
def test_which_kernel_takes_sparse_rows(n, many):
    """Either side of the rules, the same rows to the same bars."""
    lens = [(1000, n)] * (16 if n < 100 else 1)
    s = Scene(lens, 32, 8, 64, 64, seed=n)
    lists = _lists(s, 32, 8, seed=1)
    got = []
    assert _launches(lambda: got.append(_attend(s, lists, 32))) == (2 if many else 1)
    s.lens, s.cu = lens[:1], s.cu[:2]
    _check_sparse(s, lists, 32, got[0][0], rows=2)


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_bad_pages_queries_padding_and_strides(D):
    s = Scene([(700, 450), (300, 60)], 32, 8, D, 32, seed=8, q_pad=5)
    lists = _lists(s, 64, 6, seed=2, drop=0.0)
    q = s.q.clone()
    q[70, 9, 3], q[200, 17, 5], q[460, 0, 1] = float("nan"), float("inf"), float("nan")
    lists[460, 0] = -1                                   # nothing listed: zeros all the same
    ref, ref_lse = _attend(s, lists, 64, want_lse=True)
    wide = torch.full((s.total, 40, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:35] = q.cuda()
    out = torch.full((s.total, 32, D), 5.0, dtype=torch.bfloat16, device="cuda")
    out, lse = _attend(s, lists, 64, q=wide[:, 3:35], out=out, want_lse=True)
    spoilt = torch.zeros(s.total, 32, dtype=torch.bool, device="cuda")
    spoilt[70, 9] = spoilt[200, 17] = True
    n = int(s.cu[-1])
    assert out[70, 9].isnan().all() and lse[70, 9].isnan() and out[200, 17].isnan().all()
    assert not out[460, :4].any() and bool((lse[460, :4] == -float("inf")).all())
    spoilt[460, :4] = True
    keep = ~spoilt
    keep[n:] = False
    assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], ref_lse[keep]) and bool((out[n:] == 5.0).all())
    # pages outside the pool hide their tokens
    a = _step_args(s)
    a["block_table"][0, 4], a["block_table"][1, 1] = -3, s.cache.num_pages
    out, lse = s.cache.sparse_attention(s.q.cuda(), **a, blocks=_cuda(lists), block_tokens=64, max_q=s.max_q, want_lse=True)
    assert int(s.cache.status) == B().MOE_ERR_DEVICE
    pages = [[4], [1]]

    def cut(b, row, h):
        pos = s.lens[b][0] - s.lens[b][1] + row - int(s.cu[b])
        tok = np.arange(pos + 1)
        return tok[np.isin(tok // 64, lists[row, h]) & ~np.isin(tok // 32, pages[b])]
    for b, i in ((0, 0), (0, 449), (0, 200), (1, 0), (1, 59)):
        row = int(s.cu[b]) + i
        for h in (0, 5):
            tok = cut(b, row, h)
            k, v = (x[tok, h] for x in s.vals[b])
            o, l, pv, sabs = block.attention(s.q[row, 4 * h].double().numpy(), k, v, D ** -0.5, len(tok))
            ds = sabs * ((D + 8) * 2.0 ** -22 + 2.0 ** -24) + 2.0 ** -20
            bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * ds) * pv + len(tok) * 2.0 ** -25 * (np.abs(v).max() if len(tok) else 0)
            assert (np.abs(out[row, 4 * h].double().cpu().numpy() - o) <= bar).all()
    # more rows than the bound: left alone, reported; the others as before
    s.cache.status.zero_()
    out = torch.full((s.total, 32, D), 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.sparse_attention(s.q.cuda(), **_step_args(s), blocks=_cuda(lists), block_tokens=64, max_q=449, out=out)
    assert int(s.cache.status) == B().MOE_ERR_DEVICE and bool((out[:450] == 5.0).all())
    assert torch.equal(out[450:460], ref[450:460])


@pytest.mark.parametrize("n,heads", [(1, 1), (5, 2), (400, 8)])
def test_blocks_of_a_very_long_context(n, heads):
    """More blocks than a union is built of at once, over pages that come up again and again."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache
    D, P, Bt, pages, kv = 64, 128, 32, 7, 600011
    c = Kv4Cache(pages, P, heads, D, 448.0, 448.0)
    k, v = _bf16((pages * P, heads, D), 1), _bf16((pages * P, heads, D), 2)
    c.append(k.cuda(), v.cuda(), _cuda(np.arange(pages * P)))
    ref = block.KvCache(pages, P, heads, D, 448.0, 448.0)
    ref.append(k.float().numpy(), v.float().numpy(), np.arange(pages * P))
    vals = [ref.values(w, np.arange(pages * P)) for w in (0, 1)]
    r = np.random.default_rng(n)
    table = r.integers(0, pages, -(-kv // P))
    q = _bf16((n, 4 * heads, D), 3)
    last = (kv - 1) // Bt
    lists = np.sort(r.integers(0, last + 1, (n, heads, 9)), -1)
    lists[..., 0], lists[..., 4], lists[..., 5], lists[..., 8] = 0, 8191, 8192, last
    out, lse = c.sparse_attention(q.cuda(), _cuda([0, n]), _cuda([kv]), _cuda(table[None]), _cuda(lists), block_tokens=Bt,
                                  max_q=n, want_lse=True)
    assert int(c.status) == 0
    for i in sorted({0, n // 2, n - 1}):
        pos = kv - n + i
        for h in range(0, heads, 3):
            tok = (np.unique(lists[i, h])[:, None] * Bt + np.arange(Bt)).ravel()
            tok = tok[tok <= pos]
            at = table[tok // P] * P + tok % P
            o, l, pv, sabs = block.attention(q[i, 4 * h].double().numpy(), vals[0][at, h], vals[1][at, h], D ** -0.5, len(tok))
            ds = sabs * ((D + 8) * 2.0 ** -22 + 2.0 ** -24) + 2.0 ** -20
            bar = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * ds) * pv + len(tok) * 2.0 ** -25 * np.abs(vals[1]).max()
            assert (np.abs(out[i, 4 * h].double().cpu().numpy() - o) <= bar).all(), (i, h)
            assert abs(float(lse[i, 4 * h]) - l) <= ds + 2.0 ** -22 * abs(l) + len(tok) * 2.0 ** -30


@pytest.mark.parametrize("scale", [30.0, -1.0, 0.0])
def test_many_rows_of_extreme_scores(scale):
    """Maxima that grow late (the sums are rescaled), scores of the other sign, none at all."""
    s = Scene([(1200, 420)], 32, 8, 128, 64, seed=3, k_scale=2.0)
    lists = _lists(s, 64, 8, seed=4)
    out, lse = _attend(s, lists, 64, scale=scale, want_lse=True)
    s2 = Scene.__new__(Scene)
    s2.__dict__.update(s.__dict__)
    s2.heads, s2.qheads, s2.q = 1, 4, s.q[:, :4]
    s2.vals = [(k[:, :1], v[:, :1]) for k, v in s.vals]
    _check_sparse(s2, lists[:, :1], 64, out[:, :4], lse[:, :4], rows=12, scale=scale)


# ------------------------------------------------------------ picks, many rows

@pytest.mark.parametrize("qheads,heads,D,P,block_tokens", [
    (16, 4, 128, 64, 64), (40, 8, 64, 16, 32), (4, 4, 128, 128, 128), (64, 4, 64, 32, 64), (32, 4, 128, 16, 128)])
@pytest.mark.parametrize("top,sink,local", [(8, 1, 2), (64, 0, 1), (33, 3, 5), (5, 4, 1)])
def test_many_rows_pick_the_oracles_blocks(qheads, heads, D, P, block_tokens, top, sink, local):
    """Runs of 128 rows and what is left of them, requests that rank nothing, requests of the other kernel."""
    Bt = block_tokens
    lens = [(90 * Bt + 9, 290), (3, 3), (0, 0), (70 * Bt, 1), (100 * Bt + 3, 128), (200, 200), (40 * Bt + 1, 9), (80 * Bt, 8)]
    p = Picker(lens, qheads, heads, D, P, Bt, seed=top)
    assert _launches(lambda: p.check(top, sink, local, rows=7)) == 2


@pytest.mark.parametrize("n,heads,launches", [(8, 8, 1), (9, 8, 1), (81, 8, 2), (640, 1, 1), (641, 1, 2)])
def test_which_kernel_takes_picks(n, heads, launches):
    p = Picker([(150 * 32, n)], 2 * heads, heads, 64, 32, 32, seed=n)
    assert _launches(lambda: p.check(12, 1, 2, rows=3)) == launches


@pytest.mark.parametrize("top", [2, 14, 26, 27, 28, 45, 64])
@pytest.mark.parametrize("kind", ["random", "rising", "falling", "equal", "few", "signs", "gone"])
def test_many_rows_pick_whatever_the_order_of_scores(top, kind):
    """Ranges either side of the one where a first pass finds a bound, picks either side of what it finds in registers;
    scores in every order, mostly equal, of both signs around zero, of pages that are not there."""
    lens = [((259 + top // 2) * 32, 420), (700 * 32, 150), (34 * 32, 30), (66 * 32 + 5, 200)]
    p = Picker(lens, 2, 1, 64, 64, 32, seed=top)
    if kind in ("rising", "falling", "few", "equal", "signs"):
        p.q[:] = 0
        p.q[:, :, 0] = 1.0
        p.means[:] = 0.0
        r = np.random.default_rng(top)
        for b, (kv, _) in enumerate(lens):
            for j in range(-(-kv // 32)):
                x = {"rising": j / 8, "falling": 100 - j / 8, "equal": 3.0, "few": float(r.integers(0, 2)),
                     "signs": float(r.integers(-1, 2))}[kind]
                p.means[p.table[b, j // 2] * 2 + j % 2, 0, 0] = x
        p.index.means.copy_(torch.tensor(p.means))
    elif kind == "gone":
        p.table[0, 5:100:3], p.table[1, 1:349], p.table[3, 2:30] = -1, p.cache.num_pages, -7
    p.check(top, 0, 1, rows=6)
    p.check(top, 1, 1, rows=4)


def test_many_rows_of_equal_scores_and_bad_pages():
    p = Picker([(120 * 32, 400), (90 * 32, 60)], 4, 2, 64, 32, 32)
    p.means[:] = 1.0
    p.means[::3] = 2.0
    p.index.means.copy_(torch.tensor(p.means))
    p.check(16, 1, 1, rows=9)
    p.q.zero_()                                   # every score 0
    p.check(64, 2, 1, rows=9)
    p.q[:, :2] = float("nan")                     # counts as 0
    p.q[::2, 3, 5] = float("-inf")
    p.q[:, 3, 6] = 3.0
    p.check(9, 0, 2, rows=9)
    # a page that is not in the pool scores lowest; with nothing else left it is picked
    p = Picker([(70 * 32, 700)], 4, 2, 64, 32, 32, seed=3)
    p.table[0, 20], p.table[0, 45] = -1, p.cache.num_pages
    p.check(16, 1, 1, rows=9)
    assert int(p.cache.status) == B().MOE_ERR_DEVICE
    p.table[0, 3:69] = -5
    p.check(16, 1, 1, rows=9)


@pytest.mark.parametrize("n", [1, 500])
def test_means_that_are_no_numbers_do_no_harm(n):
    """An index that was never updated: any picks, in range and ascending, and the call ends."""
    p = Picker([(300 * 32, n)], 4, 2, 64, 32, 32)
    raw = torch.randint(-32768, 32767, p.index.means.shape, dtype=torch.int16, generator=torch.Generator().manual_seed(1))
    p.index.means.copy_(raw.view(torch.float16))
    p.index.means[::5] = float("inf")
    p.index.means[1::5] = float("-inf")
    got = p.index.select(p.q.cuda(), **p.args(), top=20, sink=1, local=2).cpu().numpy()
    assert (got >= 0).all() and (np.diff(got, axis=-1) > 0).all() and (got[..., -1] == (300 * 32 - n + np.arange(n))[:, None] // 32).all()


def test_scores_far_apart_are_ranked():
    """Scores of every magnitude that f16 means give: outliers, thousands of equal ones, steps of a factor."""
    for n in (1, 700):
        p = Picker([(4000 * 32, n)], 2, 1, 64, 128, 32, seed=1)
        j = np.arange(len(p.means))
        p.means[:] = 0.0
        p.means[:, 0, 0] = np.where(j % 7 == 0, 2.0 ** (j % 40 - 20.0), np.where(j % 11 == 0, -(2.0 ** (j % 15)), 0.0))
        p.index.means.copy_(torch.tensor(p.means))
        p.means[:] = p.index.means.double().cpu().numpy()
        p.q[:] = 0
        p.q[:, :, 0] = 1.0
        p.check(64, 1, 1, rows=3)


# ----------------------------------------------------------------- timeouts

@pytest.mark.parametrize("which", ["select", "sparse"])
def test_waits_that_give_up_are_reported(which):
    """Every wait at one cycle: MOE_ERR_TIMEOUT, and the next call is exact."""
    if which == "select":
        p = Picker([(300 * 32, 700)], 4, 2, 64, 32, 32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call = lambda: p.index.select(p.q.cuda(), **p.args(), top=12, sink=1, local=1, device_status=status)  # noqa: E731
    else:
        s = Scene([(900, 500)], 32, 8, 64, 64, seed=3)
        lists = _lists(s, 64, 6, seed=1)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(**_step_args(s), blocks=_cuda(lists), block_tokens=64, max_q=500)
        call = lambda: s.cache.sparse_attention(s.q.cuda(), **args, device_status=status)[0]  # noqa: E731
    ref = call().clone()
    assert int(status) == 0
    B().moe_debug_set(B().MOE_DEBUG_WAIT_LIMIT, 1)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        B().moe_debug_set(B().MOE_DEBUG_WAIT_LIMIT, 0)
    assert int(status) == B().MOE_ERR_TIMEOUT
    status.zero_()
    for _ in range(3):
        assert torch.equal(call(), ref)
    assert int(status) == 0


# ------------------------------------------------------- calls and their order

def test_two_calls_at_once():
    """No state between calls: two streams at the same time give what one after the other gives."""
    s = Scene([(800, 420), (300, 1)], 32, 8, 64, 64, seed=5)
    index, _ = _index_of(s, 32)
    index.means.zero_()
    index.update(**_step_args(s), max_q=s.max_q)
    a, q = _step_args(s), s.q.cuda()

    def call(top, stream=None):
        blocks = index.select(q, **a, max_q=s.max_q, top=top, sink=1, local=1, stream=stream)
        return (blocks,) + s.cache.sparse_attention(q, **a, blocks=blocks, block_tokens=32, max_q=s.max_q, want_lse=True,
                                                    stream=stream)
    want = {top: [x.clone() for x in call(top)] for top in (6, 13)}
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[call(top, st) for top, st in zip((6, 13), streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for top, x in zip((6, 13), pair):
            assert all(torch.equal(i, j) for i, j in zip(x, want[top]))


def test_many_rows_replay_from_a_graph():
    """Selection and attention of long and short requests captured once, replayed on other lengths."""
    s = Scene([(900, 450), (600, 30), (500, 1)], 32, 8, 64, 64, seed=6)
    index, _ = _index_of(s, 32)
    index.means.zero_()
    a, q = _step_args(s), s.q.cuda()
    index.update(cu_q=_cuda([0, 900, 1500, 2000]), kv_len=a["kv_len"], block_table=a["block_table"], max_q=900)

    def call():
        blocks = index.select(q, **a, max_q=460, top=7, sink=1, local=1)
        return (blocks,) + s.cache.sparse_attention(q, **a, blocks=blocks, block_tokens=32, max_q=460, want_lse=True)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = call()
    for cu, kv in (([0, 450, 480, 481], [900, 600, 500]), ([0, 1, 460, 481], [17, 600, 333]), ([0, 100, 100, 400], [900, 0, 500]),
                   ([0, 3, 6, 9], [3, 600, 40])):
        a["cu_q"].copy_(_cuda(cu))
        a["kv_len"].copy_(_cuda(kv))
        g.replay()
        torch.cuda.synchronize()
        got = [x[:cu[-1]].clone() for x in outs]
        want = [x[:cu[-1]] for x in call()]
        assert all(torch.equal(x, y) for x, y in zip(got, want)), cu
    assert int(s.cache.status) == 0


def test_requests_that_share_pages_share_means():
    """A prefix in the same pages: either request's update serves both, and a page given to another is its."""
    s = Scene([(256, 256), (256, 256)], 2, 2, 64, 64, seed=7)
    s.table[1, :2] = s.table[0, :2]
    index, _ = _index_of(s, 64)
    a = _step_args(s)
    index.update(**a, max_q=256)
    m = index.means.clone()
    assert not m[_cuda(s.table[0, :4]).long()].isnan().any() and not m[_cuda(s.table[1, :4]).long()].isnan().any()
    k = _bf16((64, 2, 64), 5).cuda()
    slots = s.table[0, 1] * 64 + np.arange(64)
    s.cache.append(k, k, _cuda(slots))            # the page holds other tokens now
    index.update(cu_q=_cuda([0, 64, 64]), kv_len=_cuda([128, 128]), block_table=a["block_table"], max_q=64)
    changed = (index.means != m).flatten(1).any(1)
    want = torch.zeros_like(changed)
    want[int(s.table[0, 1])] = True
    assert torch.equal(changed | m.isnan().flatten(1).all(1), want | m.isnan().flatten(1).all(1))


def test_calls_with_nothing_to_do():
    from nvfp4_mixture_experts_moe_gb300 import Kv4BlockIndex, Kv4Cache, Rope
    c = Kv4Cache(4, 16, 2, 64, 400.0, 400.0)
    index, rope = Kv4BlockIndex(c, 32), Rope(64)
    e = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    assert rope(e(0, 4, 64), i(0)).shape == (0, 4, 64)
    assert c.append_rotated(e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), i(0), i(0), rope).shape == (0, 4, 64)
    index.update(i(1), i(0), i(0, 3), max_q=1)
    index.update(i(3), i(2), i(2, 0), max_q=1)                       # requests without tokens or pages
    assert index.select(e(0, 4, 64), i(3), i(2), i(2, 3), max_q=1, top=4).shape == (0, 2, 4)
    assert (index.select(e(5, 4, 64), i(3), i(2), i(2, 3), max_q=1, top=4, blocks=i(5, 2, 4) + 7) == 7).all()
    out, lse = c.sparse_attention(e(0, 4, 64), i(3), i(2), i(2, 3), i(0, 2, 4), block_tokens=32, max_q=1, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    cu = _cuda([0, 1, 2])
    out, lse = c.sparse_attention(e(2, 4, 64).zero_(), cu, i(2), i(2, 0), i(2, 2, 4), block_tokens=32, max_q=1, want_lse=True)
    assert not out.any() and bool((lse == -float("inf")).all())     # queries of requests that hold nothing: reported below
    assert int(c.status) == 0


# ---------------------------------------------------------------- the example

def test_example_with_chosen_blocks_runs_and_repeats():
    m = _example()
    tokens = torch.randint(0, m.VOCAB, (200,), generator=torch.Generator().manual_seed(2)).cuda()
    runs = []
    for _ in range(2):
        s = m.Server(3, 256, top=3)
        t = s.step(tokens, [70, 0, 130])
        got = [t]
        for _ in range(3):
            t = s.step(t, [1, 1, 1])
            got.append(t)
        assert int(s.tables.status) == 0 and s.length.cpu().tolist() == [73, 3, 133]
        assert all(int(b.cache.status) == 0 for b in s.blocks)
        runs.append(torch.stack(got).cpu())
    assert torch.equal(runs[0], runs[1])
    assert m.main(top=3) == 0


def test_example_with_every_block_attends_as_without_blocks():
    """The cached rows are the same bytes; the outputs differ by the roundings of two attention kernels (bf16 outputs, f16
    probabilities, scores of at most some tens: 2^-6 of the largest value each element), carried through the projection, and
    by the bf16 roundings of the projection and of the residual."""
    m = _example()
    n = 200
    x, h = _bf16((n, m.HIDDEN), 5).cuda(), _bf16((n, m.HIDDEN), 6).cuda()
    outs, rows = [], []
    for top in (0, 64):
        s = m.Server(2, 256, top=top)
        b = s.blocks[0]
        t = s.tables.run(s.length, _cuda([150, 50]), s.block_table, s.free_pages, s.free_count)
        outs.append(b.attend(h, x, t, s.block_table, 150)[0].double())
        rows.append(b.cache.read(t.slots[:n]))
    assert torch.equal(rows[0][0], rows[1][0]) and torch.equal(rows[0][1], rows[1][1])
    da = b.w_o.double().abs().sum(dim=1) * 2.0 ** -6 * float(rows[0][1].abs().max())
    bar = da + 2.0 ** -7 * (outs[0] - h.double()).abs() + 2.0 ** -7 * outs[0].abs()
    assert ((outs[0] - outs[1]).abs() <= bar).all()


def test_example_turns_as_its_torch_form():
    """Two roundings to bf16, and the torch form's angles: up to 256, rounded twice, 2^-15 of a pair's magnitudes."""
    m = _example()
    x, pos = _bf16((256, m.Q_HEADS, m.DIM), 3).cuda(), torch.arange(256, dtype=torch.int32, device="cuda")
    rope = m.Server(1, 256).blocks[0].rope
    got, want = rope(x, pos).double(), m.rotate(x, pos).double()
    a, b = x.double().abs().chunk(2, dim=-1)
    bar = 2.0 ** -7 * want.abs() + 2.0 ** -14 * torch.cat((a + b, a + b), dim=-1)
    assert ((got - want).abs() <= bar).all()
