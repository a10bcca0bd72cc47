"""Corners of the contracts of positions, block means, selection and sparse attention (include/moe_block.h) on the GPU.
Bars as in test_gpu_sparse.py."""
import numpy as np
import pytest
import torch

from oracle import block
from test_gpu_block import Scene, _bf16, _cuda, built  # noqa: F401
from test_gpu_sparse import Picker, _attend, _check_sparse, _index_of
from test_gpu_sparse_contracts import _launches

pytestmark = pytest.mark.gpu


# --------------------------------------------------- many rows, end of a unit

@pytest.mark.parametrize("D,block_tokens", [(64, 64), (128, 64), (128, 128), (64, 32)])
def test_units_whose_last_step_is_most_of_them(D, block_tokens):
    """Units of one step or two: an output that is read before the last products are in it is no near miss."""
    s = Scene([(1500, 520), (900, 200)], 32, 8, D, 32, seed=D + block_tokens)
    lists = np.full((s.total, 8, 2), -1)
    t = np.arange(s.total)
    lists[:, :, 0] = (t // 32 % 5)[:, None]
    lists[t // 32 % 2 == 1, :, 1] = 5
    ref, lse = _attend(s, lists, block_tokens, want_lse=True)
    _check_sparse(s, lists, block_tokens, ref, lse, rows=12)
    for _ in range(20):
        assert torch.equal(_attend(s, lists, block_tokens)[0], ref)


# ----------------------------------------- blocks of several pages, shared starts

P = 16


def _share(scene, b, tokens):
    """Request b's first tokens are request 0's, in the same pages."""
    scene.table[b, :tokens // P] = scene.table[0, :tokens // P]
    for mine, first in zip(scene.vals[b], scene.vals[0]):
        mine[:tokens] = first[:tokens]


def _update(scene, index, who):
    """Makes all blocks of the requests ``who``, the others bring nothing."""
    n = [kv if b in who else 0 for b, (kv, _) in enumerate(scene.lens)]
    index.update(_cuda(np.concatenate([[0], np.cumsum(n)])), _cuda([kv for kv, _ in scene.lens]), _cuda(scene.table),
                 max_q=max(n))


def _toward(scene, want, blocks):
    """Queries that look for one block of their request's each, the others at random."""
    g = scene.qheads // scene.heads
    q = scene.q.clone()
    for b, (_, n) in enumerate(scene.lens):
        for i in range(0, n, 2):
            m = torch.tensor(np.repeat(want[b][blocks[b]], g, 0))
            q[int(scene.cu[b]) + i] = (m / m.abs().amax()).to(torch.bfloat16)
    return q


def _check_picks(scene, index, want, q, top, who=None, rows=9):
    got = index.select(q.cuda(), _cuda(scene.cu), _cuda([kv for kv, _ in scene.lens]), _cuda(scene.table), max_q=scene.max_q,
                       top=top, sink=0, local=1).cpu().numpy()
    assert int(scene.cache.status) == 0
    g, missed = scene.qheads // scene.heads, []
    for b, (kv, n) in enumerate(scene.lens):
        if who is not None and b not in who:
            continue
        for i in sorted(set(np.linspace(0, n - 1, rows).astype(int))):
            for h in range(scene.heads):
                row = int(scene.cu[b]) + i
                means = [want[b][j][h] for j in range(len(want[b]))]
                means += [np.zeros(scene.D)]      # the last block may be incomplete: never ranked
                ref = block.picks(q[row, h * g:(h + 1) * g].double().numpy(), means, kv - n + i, index.block_tokens, top, 0, 1)
                if got[row, h].tolist() != ref + [-1] * (top - len(ref)):
                    missed.append((b, i, h, got[row, h].tolist(), ref))
    assert not missed, missed[:4]


def _check_rows(scene, index, want, who):
    """Means where the header says they are."""
    means, owners = index.means.double().cpu().numpy(), index.owners.cpu().numpy()
    Bt = index.block_tokens
    for b in who:
        for j in range(scene.lens[b][0] // Bt):
            first, last = scene.table[b, j * Bt // P], scene.table[b, (j * Bt + Bt - 1) // P]
            assert owners[first] >= 0
            assert (means[first if owners[first] == last else last] == want[b][j]).all(), (b, j)


@pytest.mark.parametrize("n", [1, 330])
@pytest.mark.parametrize("order", [((0, 1, 2),), ((0,), (1,), (2,)), ((2,), (1,), (0,)), ((1,), (0, 2), (1,))])
@pytest.mark.parametrize("block_tokens", [32, 64, 128])
def test_blocks_that_start_in_a_shared_page_keep_their_own_means(block_tokens, order, n):
    """Requests 0, 1 and 2 have a prefix in common that ends inside block 1 (request 2: block 3)."""
    Bt = block_tokens
    s = Scene([(12 * Bt + n, n), (11 * Bt + n + 7, n), (14 * Bt + n, n)], 8, 2, 64, P, seed=Bt)
    _share(s, 1, Bt + P)
    _share(s, 2, 3 * Bt + Bt // 2)
    index, want = _index_of(s, Bt)
    for who in order:
        _update(s, index, who)
    q = _toward(s, want, (1, 1, 3))
    for top in (2, 6):
        _check_picks(s, index, want, q, top)
    q = _toward(s, want, (3, 0, 1))
    _check_picks(s, index, want, q, 2)
    _check_rows(s, index, want, (0, 1, 2))


def test_pages_given_back_and_taken_again_need_no_care():
    """Request 0 ends; request 2 takes its pages, in another order, behind the prefix that request 1 still has."""
    Bt, heads, D, n = 64, 2, 64, 3
    s = Scene([(9 * Bt, n), (9 * Bt + 3, n), (9 * Bt, n)], 8, heads, D, P, seed=1)
    _share(s, 1, Bt + P)
    _share(s, 2, Bt + P)
    index, want = _index_of(s, Bt)
    _update(s, index, (0, 1))
    have = (Bt + P) // P
    freed = s.table[0, have:9 * Bt // P].copy()
    s.table[2, have:9 * Bt // P] = freed[::-1]
    k, v = _bf16((9 * Bt, heads, D), 7 * 2 + 1), _bf16((9 * Bt, heads, D), 7 * 2 + 2)     # request 2's rows, as Scene made them
    k[:, :, 3] *= 3
    tok = np.arange(Bt + P, 9 * Bt)
    s.cache.append(k[tok].cuda(), v[tok].cuda(), _cuda(s.table[2, tok // P] * P + tok % P))
    s.lens[0], s.cu = (0, 0), np.array([0, 0, n, 2 * n])
    s.table[0] = -1
    s.q = s.q[n:]
    _update(s, index, (2,))
    q = _toward(s, want, (1, 1, 1))
    _check_picks(s, index, want, q, 2, who=(1, 2))
    _check_rows(s, index, want, (1, 2))
    # and the other way round: pages in their first order again, request 1 ends
    s.table[2, have:9 * Bt // P] = freed
    s.cache.append(k[tok].cuda(), v[tok].cuda(), _cuda(s.table[2, tok // P] * P + tok % P))
    _update(s, index, (2,))
    _check_picks(s, index, want, q, 2, who=(1, 2))
    _check_rows(s, index, want, (1, 2))


def test_a_block_with_a_bad_last_page_scores_lowest():
    s = Scene([(9 * 64, 1)], 8, 2, 64, P, seed=2)
    index, want = _index_of(s, 64)
    _update(s, index, (0,))
    q = _toward(s, want, (2,)).cuda()
    pick = lambda: index.select(q, _cuda([0, 1]), _cuda([9 * 64]), _cuda(s.table), max_q=1, top=2, sink=0, local=1)  # noqa: E731
    assert pick()[0, :, 0].tolist() == [2, 2] and int(s.cache.status) == 0
    s.table[0, 11] = -1
    assert 2 not in pick()[0].tolist()[0] and int(s.cache.status) != 0


# ------------------------------------------------------- infinite queries

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[(40, 1), (300, 2)], [(300, 40), (90, 40)], [(700, 400), (20, 20)]])
def test_an_infinity_whose_scores_are_all_minus_infinity_gives_nan(D, lens):
    """exp(-inf + inf) is no number: zeros and -inf are what a row that sees nothing gives. All cached keys are negative
    where the query is infinite."""
    s = Scene(lens, 32, 8, D, 32, seed=D)
    for b, (kv, _) in enumerate(lens):
        k = _bf16((kv, 8, D), b)
        k[:, :, 3] = -5.0
        s.cache.append(k.cuda(), k.cuda(), _cuda(s.table[b, np.arange(kv) // 32] * 32 + np.arange(kv) % 32))
    lists = np.tile(np.arange(24), (s.total, 8, 1))
    row, head = int(s.cu[1]), 5                  # the second request's first token
    lists[row + 1, 1] = -1                       # the next row sees nothing
    q = s.q.clone()
    q[row, head, 3] = q[row + 1, head, 3] = float("inf")
    spoilt = torch.zeros(s.total, 32, dtype=torch.bool, device="cuda")
    spoilt[row, head] = True
    for name, call in (("sparse", lambda q: _attend(s, lists, 32, q=q.cuda(), want_lse=True)),
                       ("dense", lambda q: s.run(q=q.cuda(), want_lse=True))):
        spoilt[row + 1, head] = name == "dense"
        (good, good_lse), (out, lse) = call(s.q), call(q)
        assert bool(out.isnan().all(-1).eq(spoilt).all()) and bool(lse.isnan().eq(spoilt).all()), name
        assert torch.equal(out[~spoilt], good[~spoilt]) and torch.equal(lse[~spoilt], good_lse[~spoilt]), name
    assert bool((_attend(s, lists, 32, q=q.cuda(), want_lse=True)[1][row + 1, 4:8] == -float("inf")).all())


# ------------------------------------------------------- the largest rotation

def test_rotation_of_as_many_elements_as_the_limit_allows():
    """2^32 elements of heads of three: two threads a head, more of them than 2^31."""
    from nvfp4_mixture_experts_moe_gb300 import MoeError, Rope
    n, few = (1 << 32) // 3, 1000
    rope = Rope(2)
    x, pos = torch.zeros(n + 1, 1, 3, dtype=torch.bfloat16, device="cuda"), torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    spots = (0, (1 << 31) // 3 - few // 2, (1 << 31) // 2 - few // 2, n - few)
    for i, at in enumerate(spots):
        x[at:at + few] = _bf16((few, 1, 3), i).cuda()
        pos[at:at + few] = torch.arange(at, at + few, dtype=torch.int32, device="cuda")
    y = rope(x[:n], pos[:n])
    for at in spots:
        assert torch.equal(y[at:at + few], rope(x[at:at + few], pos[at:at + few]))
    with pytest.raises(MoeError):
        rope(x, pos, out=x)


# ------------------------------------------------- which kernel takes picks

@pytest.mark.parametrize("n,heads,launches", [(76, 8, 1), (77, 8, 2), (80, 8, 2), (608, 1, 1), (609, 1, 2)])
def test_which_kernel_takes_picks_of_wide_heads(n, heads, launches):
    p = Picker([(150 * 32, n)], 2 * heads, heads, 128, 32, 32, seed=n)
    assert _launches(lambda: p.check(12, 1, 2, rows=3)) == launches


# ------------------------------------------------------------- stored bytes

@pytest.mark.parametrize("D,pairs", [(64, "half"), (128, "half"), (128, "adjacent")])
def test_groups_whose_scale_is_zero_store_zero_codes(D, pairs):
    """Elements of either sign too small for a scale: the pool's bytes are the append's, keys (unturned ones) and values."""
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, Rope
    T, heads = 40, 2
    k, v = _bf16((T, heads, D), 1), _bf16((T, heads, D), 2)
    for x in (k, v):
        x[3:7, :, 16:48] *= 1e-30
        x[9, 1] = -0.0
        x[11, 0, 32:] = -1e-38
    k[:, :, D // 2:] = 0.0 if pairs == "half" else k[:, :, D // 2:]
    pools = []
    for turned in (False, True):
        c = Kv4Cache(3, 16, heads, D, 300.0, 300.0)
        c.pool.fill_(0xA5)
        at = _cuda(np.arange(T) + 5)
        if turned:
            c.append_rotated(None, k.cuda(), v.cuda(), at, _cuda(np.zeros(T)), Rope(D, pairs=pairs))
        else:
            c.append(k.cuda(), v.cuda(), at)
        pools.append(c.pool.view(3, heads, 1, 18 * D))
    assert torch.equal(pools[0][..., 9 * D:], pools[1][..., 9 * D:])
    a, b = (x[..., :9 * D] for x in pools)
    assert torch.equal(a[..., 8 * D:], b[..., 8 * D:])
    zero = (a[..., 8 * D:] == 0).view(3, heads, 1, 16, D // 16, 1).expand(-1, -1, -1, -1, -1, 8).reshape(3, heads, 1, 8 * D)
    assert bool(zero.any()) and torch.equal(a[..., :8 * D][zero], b[..., :8 * D][zero])
