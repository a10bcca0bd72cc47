"""Pins of the block operators' oracle (oracle/block.py) and host-side checks
of their entry points: no GPU needed."""
import ctypes
import shutil
import subprocess
import os

import numpy as np
import pytest
import torch

from oracle import block, nvfp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("P,B,seed", [(16, 1, 0), (32, 7, 1), (64, 40, 2), (1, 5, 3)])
def test_step_hands_out_pages_once_and_in_order(P, B, seed):
    r = np.random.default_rng(seed)
    ctx, new = r.integers(0, 5 * P + 1, B), r.integers(0, 3 * P + 1, B)
    W = 9
    have = -(-ctx // P)
    pages = r.permutation(4 * W * B)
    table = np.full((B, W), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = pages[at:at + have[b]]
        at += have[b]
    free = pages[at:]
    need = -(-(ctx + new) // P) - have
    for count in (len(free), int(need.sum()), int(need.sum()) // 2, 0):
        o = block.step(ctx, new, table, free, count, P, int(new.sum()) + 3)
        grant = o["kv_len"] == ctx + new
        # granted requests are those whose running need fits, plus those that need nothing
        assert (grant == ((need == 0) | (np.cumsum(need) <= count))).all()
        assert o["free_count"] == count - need[grant].sum()
        used = [p for b in range(B) for p in o["table"][b, :-(-o["kv_len"][b] // P)]]
        assert len(set(used)) == len(used) and set(free[:o["free_count"]]).isdisjoint(used)
        assert o["bad"] == (not grant.all())
        for b in range(B):
            for i in range(new[b]):
                s, p = o["slots"][o["cu_q"][b] + i], ctx[b] + i
                assert o["positions"][o["cu_q"][b] + i] == p
                assert s == (o["table"][b, p // P] * P + p % P if grant[b] else -1)
        assert (o["slots"][new.sum():] == -1).all()


def test_cache_rows_and_layout():
    g = np.random.default_rng(5)
    c = block.KvCache(3, 32, 2, 64, 100.0, 50.0)
    k, v = (torch.tensor(g.normal(size=(5, 2, 64))).to(torch.bfloat16).float().numpy() for _ in range(2))
    k[1, 0, 3] = np.nan
    slots = np.array([95, 3, -1, 40, 0])
    c.append(k, v, slots)
    k0 = np.where(np.isnan(k), 0, k)
    for which, x in ((0, k0), (1, v)):
        got = c.values(which, [95, 3, 40, 0])
        ref = x[[0, 1, 3, 4]]
        amax = np.abs(ref.reshape(4, 2, 4, 16)).max(-1, keepdims=True)
        # half the widest e2m1 step (1 of 6) of the block's largest value, widened by the scale's rounding
        assert (np.abs(got - ref).reshape(4, 2, 4, 16) <= amax / 6 * (1 + 2.0 ** -4)).all()
    pool = c.pool()
    assert pool.shape == (3, 2, 2, 18 * 64)
    row = pool[2, 1, 1]     # slot 95: page 2, block 1, token 15
    assert (nvfp4.unpack(row[15 * 32:16 * 32][None])[0] == c.codes[0, 95, 1]).all()
    assert (row[8 * 64 + 15 * 4:8 * 64 + 16 * 4] == c.sf[0, 95, 1]).all()
    assert (nvfp4.unpack(row[9 * 64 + 15 * 32:9 * 64 + 16 * 32][None])[0] == c.codes[1, 95, 1]).all()
    assert (row[17 * 64 + 15 * 4:17 * 64 + 16 * 4] == c.sf[1, 95, 1]).all()


@pytest.mark.parametrize("position,window", [(9, 0), (4, 0), (9, 3), (-1, 0), (0, 1)])
def test_attention_is_masked_softmax(position, window):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(s, 16, generator=g, dtype=torch.float64) for s in (1, 10, 10))
    out, lse, pv, sabs = block.attention(q[0].numpy(), k.numpy(), v.numpy(), 0.25, position, window)
    s = (q @ k.T * 0.25)[0]
    for j in range(10):
        if j > position or (window and j <= position - window):
            s[j] = -torch.inf
    if position < 0:
        assert lse == -np.inf and (out == 0).all()
        return
    assert np.allclose(out, (torch.softmax(s, 0) @ v).numpy(), atol=1e-14)
    assert np.isclose(lse, float(torch.logsumexp(s, 0)), atol=1e-14)
    assert (np.abs(out) <= pv + 1e-15).all() and sabs >= float(s[torch.isfinite(s)].abs().max())


def test_block_norm_against_torch():
    g = torch.Generator().manual_seed(2)
    x, res, gate = (torch.randn(3, 24, generator=g, dtype=torch.float64) for _ in range(3))
    w1, w2 = (torch.rand(24, generator=g, dtype=torch.float64) for _ in range(2))
    r, out = block.block_norm(*(t.numpy() for t in (x, res, gate, w1, w2)), a=0.5, b=2.0, eps=1e-5, offset=1.0)
    n = torch.nn.functional.rms_norm(x, (24,), w1 + 1, 1e-5)
    ref = 0.5 * res + 2.0 * gate * n
    assert np.allclose(r, ref.numpy(), atol=1e-13)
    assert np.allclose(out, torch.nn.functional.rms_norm(ref, (24,), w2 + 1, 1e-5).numpy(), atol=1e-13)
    assert np.array_equal(block.block_norm(None, res.numpy(), a=3.0)[0], 3.0 * res.numpy())


# ------------------------------------------------ entry points, on the host

@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from nvfp4_mixture_experts_moe_gb300 import binding
    return binding.lib()


def _cache(B, **kw):
    d = dict(num_pages=4, page_tokens=64, kv_heads=2, head_dim=128, k_gs=1.0, v_gs=1.0, pool=256)
    d.update(kw)
    return B.MoeKv4Cache(**d)


def test_pool_sizes(L):
    assert L.moe_kv4_pool_size(4, 64, 2, 128) == 4 * 64 * 2 * 2 * 72
    assert L.moe_kv4_pool_size(4, 64, 2, 64) == 4 * 64 * 2 * 2 * 36
    assert L.moe_kv4_pool_size(1 << 24, 64, 8, 128) == (1 << 24) * 64 * 8 * 144   # far past 32 bits
    for bad in ((0, 64, 2, 128), (4, 48, 2, 128), (4, 64, 0, 128), (4, 64, 2, 96), (1 << 25, 64, 2, 128),
                (4, 64, 2000, 128)):
        assert L.moe_kv4_pool_size(*bad) == 0


def test_cache_calls_refuse_on_the_host(L):
    from nvfp4_mixture_experts_moe_gb300 import binding as B
    ok = dict(k=256, v=256, ks=256, vs=256, slots=256, n=4)

    def append(cache=None, **kw):
        a = {**ok, **kw}
        return L.moe_kv4_append(ctypes.byref(cache or _cache(B)), a["k"], a["v"], a["ks"], a["vs"], a["slots"],
                                a["n"], None, None)
    assert append(n=0) == B.MOE_OK
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(k=264), dict(v=258), dict(ks=255), dict(vs=260),
                dict(ks=128), dict(n=-1)):
        assert append(**bad) == B.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(k_gs=0.0), dict(v_gs=float("inf")), dict(k_gs=float("nan")), dict(pool=None), dict(pool=264),
                dict(num_pages=0), dict(kv_heads=-1)):
        assert append(cache=_cache(B, **bad)) == B.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(page_tokens=8), dict(head_dim=96), dict(head_dim=256), dict(num_pages=1 << 26)):
        assert append(cache=_cache(B, **bad)) == B.MOE_ERR_UNSUPPORTED, bad
    c = ctypes.byref(_cache(B))
    assert L.moe_kv4_read(c, None, 0, None, None, None, None) == B.MOE_OK
    assert L.moe_kv4_read(c, 256, 3, None, None, None, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_kv4_read(c, 256, 3, 264, None, None, None) == B.MOE_ERR_INVALID_ARG


def _attn(B, cache=None, **kw):
    d = dict(cache=cache or _cache(B), batch=2, q_heads=8, total_q=5, max_q=3, max_pages=3, q=256, q_stride=1024,
             cu_q=256, kv_len=256, block_table=256, scale=0.1, causal=1, window=0, out=256, lse=None)
    d.update(kw)
    return B.MoeKv4AttnArgs(**d)


def test_attention_refuses_on_the_host(L):
    from nvfp4_mixture_experts_moe_gb300 import binding as B

    def call(a, ws=256, nbytes=1 << 40):
        return L.moe_kv4_attention(ctypes.byref(a), ws, nbytes, None)
    need = B.moe_kv4_attention_workspace_size(_attn(B))
    assert need >= B.MOE_KV4_WS_ZERO
    assert call(_attn(B), ws=None) == B.MOE_ERR_WORKSPACE
    assert call(_attn(B), ws=264) == B.MOE_ERR_WORKSPACE
    assert call(_attn(B), nbytes=need - 1) == B.MOE_ERR_WORKSPACE
    assert call(_attn(B, batch=0)) == B.MOE_OK and call(_attn(B, total_q=0)) == B.MOE_OK
    for bad in (dict(q=None), dict(cu_q=None), dict(kv_len=None), dict(out=None), dict(block_table=None),
                dict(q=264), dict(out=264), dict(q_stride=1023), dict(q_stride=512), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(window=-1), dict(window=4, causal=0), dict(batch=-1), dict(total_q=-1),
                dict(max_q=-1), dict(max_q=0), dict(max_pages=-1), dict(q_heads=0), dict(cache=_cache(B, k_gs=-1.0))):
        assert call(_attn(B, **bad)) == B.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(q_heads=7), dict(batch=5000), dict(cache=_cache(B, head_dim=80)), dict(max_pages=1 << 25),
                dict(max_pages=1 << 24, batch=4096), dict(total_q=1 << 30),
                dict(batch=1, total_q=1 << 22, max_q=1 << 22, max_pages=1 << 18)):
        assert call(_attn(B, **bad)) == B.MOE_ERR_UNSUPPORTED, bad
        assert B.moe_kv4_attention_workspace_size(_attn(B, **bad)) == 0


def test_step_and_norm_refuse_on_the_host(L):
    from nvfp4_mixture_experts_moe_gb300 import binding as B
    step = dict(batch=3, page_tokens=16, max_pages=4, tokens=5, free_capacity=8, ctx_len=256, new_len=512,
                block_table=256, free_pages=256, free_count=256, free_count_out=512, kv_len=1024, cu_q=256, slots=256,
                positions=256, device_status=None)
    for bad in (dict(batch=-1), dict(page_tokens=0), dict(max_pages=0), dict(tokens=-1), dict(free_capacity=-1),
                dict(ctx_len=None), dict(new_len=None), dict(block_table=None), dict(free_pages=None),
                dict(free_count=None), dict(free_count_out=None), dict(kv_len=None), dict(cu_q=None),
                dict(slots=None), dict(positions=None), dict(free_count_out=256), dict(kv_len=256),
                dict(page_tokens=1 << 16, max_pages=1 << 16)):
        assert L.moe_kv_step(ctypes.byref(B.MoeKvStepArgs(**{**step, **bad})), None) == B.MOE_ERR_INVALID_ARG, bad
    assert L.moe_kv_step(ctypes.byref(B.MoeKvStepArgs(**{**step, "batch": 4097})), None) == B.MOE_ERR_UNSUPPORTED
    norm = dict(T=2, H=64, x=256, x_stride=64, gate=256, gate_stride=0, residual=256, residual_stride=64,
                residual_f32=0, w_post=256, w_pre=256, residual_scale=1.0, branch_scale=1.0, eps=1e-6, w_offset=0.0,
                residual_out=512, out=512)
    assert L.moe_block_norm(ctypes.byref(B.MoeBlockNormArgs(**{**norm, "T": 0})), None) == B.MOE_OK
    for bad in (dict(T=-1), dict(H=0), dict(residual=None), dict(out=None), dict(w_pre=None, residual_out=None),
                dict(x_stride=63), dict(residual_stride=63), dict(gate_stride=63), dict(eps=-1.0),
                dict(eps=float("nan")), dict(residual_scale=float("inf")), dict(x=257), dict(residual_f32=1, residual=258),
                dict(residual=512, residual_stride=72)):
        assert L.moe_block_norm(ctypes.byref(B.MoeBlockNormArgs(**{**norm, **bad})), None) == B.MOE_ERR_INVALID_ARG, bad
    assert L.moe_block_norm(ctypes.byref(B.MoeBlockNormArgs(**{**norm, "H": 16385, "x_stride": 16385,
                                                               "residual_stride": 16385})), None) == B.MOE_ERR_UNSUPPORTED


def test_structs_match_the_header(tmp_path):
    from nvfp4_mixture_experts_moe_gb300 import binding as B
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = {"moe_kv4_cache": B.MoeKv4Cache, "moe_kv4_attn_args": B.MoeKv4AttnArgs,
               "moe_kv_step_args": B.MoeKvStepArgs, "moe_block_norm_args": B.MoeBlockNormArgs}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "moe_block.h"', "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {n} %zu\\n", offsetof({cname}, {n}));' for n, _ in py._fields_]
    lines += [f'  printf("zero bytes %d\\n", MOE_KV4_WS_ZERO);', "  return 0;", "}"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    assert got.pop(("zero", "bytes")) == B.MOE_KV4_WS_ZERO
    # the packed forms are the structs' bytes
    for pack, py in ((B.PACK_KV4_ATTN, B.MoeKv4AttnArgs), (B.PACK_KV_STEP, B.MoeKvStepArgs),
                     (B.PACK_BLOCK_NORM, B.MoeBlockNormArgs)):
        assert pack.size == ctypes.sizeof(py)
        n = len(pack.unpack(bytes(pack.size)))
        vals = list(range(1, n + 1))
        a = py.from_buffer_copy(pack.pack(*vals))
        flat = []
        for name, _ in py._fields_:
            v = getattr(a, name)
            flat += [getattr(v, f) for f, _ in v._fields_] if isinstance(v, ctypes.Structure) else [v]
        assert flat == vals, py
    for cname, py in structs.items():
        assert got.pop((cname, "size")) == ctypes.sizeof(py), cname
        for name, _ in py._fields_:
            assert got.pop((cname, name)) == getattr(py, name).offset, (cname, name)
    assert not got
