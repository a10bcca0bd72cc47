"""Pins of the oracle of rotation, block means and picks (oracle/block.py), and host-side limits and checks of their
entry points (include/moe_block.h, block.py): no GPU needed."""
import ctypes
import math
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block
from test_block_host import BF, Fake, I32, U8
from test_oracle_block import L, _cache  # noqa: F401


def bind():
    from nvfp4_mixture_experts_moe_gb300 import binding
    return binding


# ------------------------------------------------------------------- oracle

@pytest.mark.parametrize("pairs", ["half", "adjacent"])
def test_oracle_rotation(pairs):
    """Against a plain 2 x 2 product at small positions, relative angles, and back again."""
    g = np.random.default_rng(3)
    x = g.normal(size=(4, 2, 10))
    freq, axis = [1.0, 0.37, 0.011], [0, 1, 1]
    pos = np.array([[0, 1, 5, 9], [0, 2, 3, 40]])
    y, _ = block.rope(x, pos, freq, axis, pairs)
    for t in range(4):
        for p in range(3):
            i, j = (p, p + 3) if pairs == "half" else (2 * p, 2 * p + 1)
            a = pos[axis[p]][t] * freq[p]
            assert np.allclose(y[t, :, i], x[t, :, i] * math.cos(a) - x[t, :, j] * math.sin(a), atol=1e-12)
            assert np.allclose(y[t, :, j], x[t, :, i] * math.sin(a) + x[t, :, j] * math.cos(a), atol=1e-12)
    assert (y[..., 6:] == x[..., 6:]).all() and (y[0] == x[0]).all()
    back, _ = block.rope(y, pos, freq, axis, pairs, inverse=True)
    assert np.allclose(back, x, atol=1e-12)
    # a product of two turned vectors goes by the difference of their positions
    far, _ = block.rope(x, pos + 10 ** 9, freq, axis, pairs)
    assert np.allclose((far[1] * far[2]).sum(-1), (y[1] * y[2]).sum(-1), atol=1e-9)


def test_two_pi():
    assert abs(float(block.TWO_PI) - 2 * math.pi) == 0.0
    # Machin: pi = 16 atan(1/5) - 4 atan(1/239)
    def atan(n, terms):
        return sum(Fraction((-1) ** k, (2 * k + 1) * n ** (2 * k + 1)) for k in range(terms))
    pi = 16 * atan(5, 50) - 4 * atan(239, 20)
    assert abs(2 * pi - block.TWO_PI) < Fraction(1, 10 ** 59)


def test_oracle_means_and_picks():
    rows = np.array([[1.0, -3.0, 0.0], [2.0, -4.0, 0.03]])
    m = block.block_mean(rows)          # means 1.5, -3.5, 0.015: steps of 2^(1 - 6)
    assert m.tolist() == [1.5, -3.5, 0.0]
    assert (block.block_mean(np.zeros((4, 3))) == 0).all()
    q = np.array([[1.0, 0.0, 0.0], [0.0, 0.0, np.nan]])
    means = [np.array([v, 0.0, 0.0]) for v in (0.0, 5.0, 7.0, 7.0, 1.0, 9.0, 0.0)]
    pick = lambda pos, **kw: block.picks(q, means, pos, 32, **{**dict(top=4, sink=1, local=1), **kw})  # noqa: E731
    assert pick(6 * 32) == [0, 2, 5, 6] and pick(6 * 32, top=3) == [0, 5, 6]
    assert pick(4 * 32 + 5) == [0, 2, 3, 4] and pick(3 * 32) == [0, 1, 2, 3] and pick(-1) == []
    assert pick(6 * 32, top=3, sink=0, local=2) == [2, 5, 6]      # equal scores: the lower block
    means[5] = None
    assert pick(6 * 32, top=3) == [0, 2, 6]


# -------------------------------------------------------------------- tables

@pytest.mark.parametrize("f", [0.0, 1.0, -1.0, 1024.0, -0.3, 1e-4, 10000.0 ** (-63 / 64), 2.0 ** -60, 5e-324, 0.1, math.pi])
def test_turns_are_the_nearest_multiples(L, f):  # noqa: F811
    """inv_freq / (2 pi) modulo one turn, to half of 2^-62 and what truncating below 2^-64 loses."""
    for axis in range(4):
        t, = bind().moe_rope_turns([f], [axis])
        assert t & 3 == axis
        off = (Fraction(t & ~3, 2 ** 64) - block.turns(f, 1)) % 1
        assert min(off, 1 - off) <= Fraction(3, 2 ** 64)


def test_turns_refuse(L):  # noqa: F811
    for f, axis in ((math.nan, 0), (math.inf, 0), (1024.5, 0), (1.0, 4), (1.0, -1)):
        with pytest.raises(bind().MoeError):
            bind().moe_rope_turns([f], [axis])
    assert L.moe_rope_turns(None, None, 1, None) == bind().MOE_ERR_INVALID_ARG
    assert L.moe_rope_turns(None, None, 0, None) == bind().MOE_OK
    f, t = (ctypes.c_double * 1)(0.5), (ctypes.c_uint64 * 1)()
    assert L.moe_rope_turns(f, None, 1, t) == bind().MOE_OK and t[0] & 3 == 0


def test_a_table_of_many_positions(L):  # noqa: F811
    """The fixed-point product modulo 2^64 is the angle at any 32-bit position, to 2^-31 turns and a little."""
    for f in (1.0, 0.7498942093324559, 1e-4):
        t, = bind().moe_rope_turns([f], [0])
        for pos in (0, 1, 131071, 10 ** 6 + 3, 2 ** 31 - 1, -1, -2 ** 31):
            off = (Fraction(t * pos % 2 ** 64, 2 ** 64) - block.turns(f, pos)) % 1
            assert min(off, 1 - off) <= Fraction(3 * abs(pos), 2 ** 64)


# ------------------------------------------------------------------ refusals

def _plan(B, **kw):
    return B.MoeRopePlan(**{**dict(rotary_dim=64, axes=1, adjacent=0, scale=1.0, turns=256), **kw})


def _rope(B, plan=None, **kw):
    M = 1 << 20
    d = dict(plan=plan or _plan(B), tokens=5, head_dim=64, q_heads=4, k_heads=2, inverse=0, q=M, q_stride=256, k=2 * M,
             k_stride=128, positions=256, q_out=3 * M, q_out_stride=256, k_out=4 * M, k_out_stride=128)
    return B.MoeRopeArgs(**{**d, **kw})


def _reaches_device(status, B):
    """The checks passed: the call ended at the device that is not there."""
    return status not in (B.MOE_OK, B.MOE_ERR_INVALID_ARG)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU, where a call "
                                                                    "that passes the checks ends at the device")


@needs_no_gpu
def test_rope_refuses_on_the_host(L):  # noqa: F811
    B = bind()
    call = lambda *a, **kw: L.moe_rope(ctypes.byref(_rope(B, *a, **kw)), None)  # noqa: E731
    assert L.moe_rope(None, None) == B.MOE_ERR_INVALID_ARG
    assert call(tokens=0) == B.MOE_OK
    assert _reaches_device(call(), B) and _reaches_device(call(k_heads=0, k=None, k_out=None), B)
    for bad in (dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(positions=None), dict(tokens=-1),
                dict(head_dim=0), dict(q_heads=0), dict(k_heads=-1), dict(q_stride=255), dict(k_stride=127),
                dict(q_out_stride=255), dict(k_out_stride=127), dict(q=(1 << 20) + 1)):
        assert call(**bad) == B.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=66), dict(axes=0), dict(axes=5), dict(turns=None),
                dict(scale=math.nan), dict(scale=math.inf), dict(turns=260)):
        assert call(_plan(B, **bad)) == B.MOE_ERR_INVALID_ARG, bad
    assert call(head_dim=514, q_stride=4096, k_stride=4096, q_out_stride=4096, k_out_stride=4096) == B.MOE_ERR_UNSUPPORTED
    assert call(q_heads=65535, q_stride=1 << 30) == B.MOE_ERR_UNSUPPORTED


@needs_no_gpu
def test_rope_outputs_overlap_nothing_but_their_own_input(L):  # noqa: F811
    B, M = bind(), 1 << 20
    call = lambda **kw: L.moe_rope(ctypes.byref(_rope(B, **kw)), None)  # noqa: E731
    assert _reaches_device(call(q_out=M), B) and _reaches_device(call(q_out=M, k_out=2 * M), B)
    q_bytes, k_bytes = 5 * 256 * 2, 5 * 128 * 2
    for bad in (dict(q_out=M + 2), dict(q_out=M - 2), dict(q_out=M + q_bytes - 2), dict(q_out=M - q_bytes + 2),
                dict(q_out=2 * M), dict(k_out=M), dict(k_out=2 * M + 2), dict(k_out=3 * M), dict(q_out=M, q_out_stride=300)):
        assert call(**bad) == B.MOE_ERR_INVALID_ARG, bad
    for fine in (dict(q_out=M + q_bytes), dict(q_out=M - q_bytes), dict(k_out=2 * M + k_bytes)):
        assert _reaches_device(call(**fine), B), fine
    # columns of one buffer: rows 512 wide, queries 0..255, keys 256..383
    cols = dict(q=M, q_stride=512, k=M + 512, k_stride=512, q_out=M, q_out_stride=512, k_out=M + 512, k_out_stride=512)
    assert _reaches_device(call(**cols), B)
    assert _reaches_device(call(**{**cols, "k_out": M + 768}), B)                  # 384..511
    assert call(**{**cols, "k_out": M + 770}) == B.MOE_ERR_INVALID_ARG             # the last one meets the next row's first
    assert call(**{**cols, "k_out": M + 510}) == B.MOE_ERR_INVALID_ARG


def _append(B, cache=None, plan=None, **kw):
    M = 1 << 20
    d = dict(cache=cache or _cache(B), plan=plan or _plan(B, rotary_dim=128), tokens=5, q_heads=4, q=M, q_stride=512, k=2 * M,
             k_stride=256, v=3 * M, v_stride=256, slots=256, positions=256, q_out=4 * M, q_out_stride=512,
             device_status=None)
    return B.MoeKv4AppendRopeArgs(**{**d, **kw})


@needs_no_gpu
def test_append_refuses_on_the_host(L):  # noqa: F811
    B, M = bind(), 1 << 20
    call = lambda *a, **kw: L.moe_kv4_append_rope(ctypes.byref(_append(B, *a, **kw)), None)  # noqa: E731
    assert call(tokens=0) == B.MOE_OK and L.moe_kv4_append_rope(None, None) == B.MOE_ERR_INVALID_ARG
    assert _reaches_device(call(), B) and _reaches_device(call(q_heads=0, q=None, q_out=None), B)
    assert _reaches_device(call(q_out=M), B)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(slots=None), dict(positions=None), dict(q_out=None),
                dict(q=M + 8), dict(k=M + 8), dict(v=M + 8), dict(q_out=M + 8), dict(tokens=-1), dict(q_heads=-1),
                dict(q_stride=504), dict(q_stride=516), dict(k_stride=252), dict(v_stride=248), dict(q_out_stride=511),
                dict(q_out=2 * M), dict(q_out=3 * M), dict(q_out=M + 16)):
        assert call(**bad) == B.MOE_ERR_INVALID_ARG, bad
    assert call(_cache(B, k_gs=0.0)) == B.MOE_ERR_INVALID_ARG
    assert call(None, _plan(B, rotary_dim=130)) == B.MOE_ERR_INVALID_ARG
    for plan in (dict(rotary_dim=48), dict(rotary_dim=16), dict(rotary_dim=24, adjacent=1)):
        assert call(None, _plan(B, **plan)) == B.MOE_ERR_UNSUPPORTED, plan
    assert _reaches_device(call(None, _plan(B, rotary_dim=48, adjacent=1)), B)


def _index(B, cache=None, **kw):
    return B.MoeKv4Index(**{**dict(cache=cache or _cache(B), block_tokens=64, means=256), **kw})


def test_index_sizes(L):  # noqa: F811
    assert L.moe_kv4_index_size(10, 64, 2, 128, 64) == 10 * 2 * 128 * 2
    assert L.moe_kv4_index_size(10, 128, 2, 64, 32) == 40 * 2 * 64 * 2
    assert L.moe_kv4_index_size(10, 16, 2, 64, 128) == 10 * 2 * 64 * 2
    for bad in ((0, 64, 2, 128, 64), (10, 64, 2, 128, 16), (10, 64, 2, 128, 0), (10, 64, 2, 128, 256), (10, 48, 2, 128, 64)):
        assert L.moe_kv4_index_size(*bad) == 0


@needs_no_gpu
def test_index_update_refuses_on_the_host(L):  # noqa: F811
    B = bind()

    def call(index=None, **kw):
        d = {**dict(batch=2, max_q=3, max_pages=4, cu=256, kv=256, table=256), **kw}
        return L.moe_kv4_index_update(ctypes.byref(index or _index(B)), d["batch"], d["max_q"], d["max_pages"], d["cu"],
                                      d["kv"], d["table"], None, None)
    assert call(batch=0) == B.MOE_OK and _reaches_device(call(), B)
    for bad in (dict(batch=-1), dict(max_q=0), dict(max_q=-1), dict(max_pages=-1), dict(cu=None), dict(kv=None),
                dict(table=None)):
        assert call(**bad) == B.MOE_ERR_INVALID_ARG, bad
    for bad in (_index(B, means=None), _index(B, means=264), _index(B, block_tokens=0), _index(B, _cache(B, pool=None))):
        assert call(bad) == B.MOE_ERR_INVALID_ARG
    for bad in (dict(batch=4097), dict(max_pages=1 << 25)):
        assert call(**bad) == B.MOE_ERR_UNSUPPORTED, bad
    for bad in (_index(B, block_tokens=48), _index(B, _cache(B, head_dim=96))):
        assert call(bad) == B.MOE_ERR_UNSUPPORTED


def _select(B, index=None, **kw):
    d = dict(index=index or _index(B), batch=2, q_heads=8, total_q=5, max_q=3, max_pages=3, q=256, q_stride=1024, cu_q=256,
             kv_len=256, block_table=256, top=8, sink=1, local=2, blocks=256, device_status=None)
    return B.MoeKv4SelectArgs(**{**d, **kw})


def _sparse(B, cache=None, **kw):
    d = dict(cache=cache or _cache(B), block_tokens=64, batch=2, q_heads=8, total_q=5, max_q=3, max_pages=3, top=8, q=256,
             q_stride=1024, cu_q=256, kv_len=256, block_table=256, blocks=256, scale=0.1, out=256, lse=None,
             device_status=None)
    return B.MoeKv4SparseArgs(**{**d, **kw})


@needs_no_gpu
@pytest.mark.parametrize("which", ["select", "sparse"])
def test_selection_and_attention_refuse_on_the_host(L, which):  # noqa: F811
    B = bind()
    make, fn = (_select, L.moe_kv4_select) if which == "select" else (_sparse, L.moe_kv4_sparse_attention)
    call = lambda *a, **kw: fn(ctypes.byref(make(B, *a, **kw)), None)  # noqa: E731
    assert fn(None, None) == B.MOE_ERR_INVALID_ARG
    assert call(batch=0) == B.MOE_OK and call(total_q=0) == B.MOE_OK and _reaches_device(call(), B)
    bad = [dict(q=None), dict(cu_q=None), dict(kv_len=None), dict(block_table=None), dict(blocks=None), dict(q=264),
           dict(q_stride=1020), dict(q_stride=1016), dict(batch=-1), dict(total_q=-1), dict(max_q=0), dict(max_pages=-1),
           dict(q_heads=0), dict(top=0), dict(top=-3)]
    if which == "select":
        bad += [dict(sink=-1), dict(local=0), dict(sink=9), dict(local=8), dict(sink=7, local=2), dict(local=2 ** 31 - 1)]
    else:
        bad += [dict(out=None), dict(out=264), dict(scale=math.nan), dict(scale=math.inf)]
    for b in bad:
        assert call(**b) == B.MOE_ERR_INVALID_ARG, b
    for b in (dict(q_heads=9), dict(q_heads=34, q_stride=1 << 16), dict(top=65), dict(batch=4097), dict(max_pages=(1 << 22) + 1),
              dict(total_q=1 << 30)):
        assert call(**b) == B.MOE_ERR_UNSUPPORTED, b
    assert _reaches_device(call(q_heads=32, q_stride=4096), B) and _reaches_device(call(top=64), B)
    for index in (dict(block_tokens=16), dict(block_tokens=256)):
        if which == "select":
            assert call(_index(B, **index)) == B.MOE_ERR_UNSUPPORTED
        else:
            assert call(**index) == B.MOE_ERR_UNSUPPORTED
    for c in (dict(pool=None), dict(v_gs=0.0), dict(num_pages=0)):
        assert call(_index(B, _cache(B, **c)) if which == "select" else _cache(B, **c)) == B.MOE_ERR_INVALID_ARG


def test_structs_match_the_header(tmp_path):
    """Field offsets and sizes, also of the packed bytes, against the host C compiler."""
    B = bind()
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = {"moe_rope_plan": (B.MoeRopePlan, None), "moe_rope_args": (B.MoeRopeArgs, B.PACK_ROPE),
               "moe_kv4_append_rope_args": (B.MoeKv4AppendRopeArgs, B.PACK_KV4_APPEND_ROPE),
               "moe_kv4_index": (B.MoeKv4Index, None), "moe_kv4_select_args": (B.MoeKv4SelectArgs, B.PACK_KV4_SELECT),
               "moe_kv4_sparse_args": (B.MoeKv4SparseArgs, B.PACK_KV4_SPARSE)}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "moe_block.h"', "int main(void) {"]
    for cname, (py, _) in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {n} %zu\\n", offsetof({cname}, {n}));' for n, _ in py._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["  return 0;", "}", ""]))
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-std=c99", "-I", inc, str(tmp_path / "layout.c"), "-o", str(tmp_path / "layout")], check=True)
    got = {}
    for line in subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.splitlines():
        cname, field, value = line.split()
        got[cname, field] = int(value)

    def leaves(py, at=0):
        for name, kind in py._fields_:
            if issubclass(kind, ctypes.Structure):
                yield from leaves(kind, at + getattr(py, name).offset)
            else:
                yield at + getattr(py, name).offset, kind
    for cname, (py, pack) in structs.items():
        assert got[cname, "size"] == ctypes.sizeof(py)
        for name, _ in py._fields_:
            assert got[cname, name] == getattr(py, name).offset, (cname, name)
        if pack is not None:
            values = [i + 1 for i in range(len(list(leaves(py))))]
            raw = pack.pack(*values)
            raw += bytes(ctypes.sizeof(py) - len(raw))
            for (at, kind), v in zip(leaves(py), values):
                assert kind.from_buffer_copy(raw, at).value == v, (cname, at)


# -------------------------------------------------------------------- Python

def _objects(module, gpu=0):
    cache = module.Kv4Cache(4, 16, 2, 64, 1.0, 1.0, pool=Fake(gpu, U8, 4 * 16 * 2 * 72))
    cache.status = Fake(gpu, I32, 1)
    rope = module.Rope(64, device="cpu")
    rope._dev = gpu
    index = module.Kv4BlockIndex(cache, 32, means=Fake(gpu, torch.float16, 4, 2, 64))
    return cache, rope, index


def _calls(module, objects_gpu=0, **where):
    def f(name, dtype, *shape):
        return Fake(where.get(name, 0), dtype, *shape)
    cache, rope, index = _objects(module, objects_gpu)
    step = dict(cu_q=lambda: f("cu_q", I32, 3), kv_len=lambda: f("kv_len", I32, 2), block_table=lambda: f("block_table", I32, 2, 4))
    step = {k: v() for k, v in step.items()}
    status = f("device_status", I32, 1)
    return {
        "rope": lambda: rope(f("q", BF, 5, 4, 64), f("positions", I32, 5), k=f("k", BF, 5, 2, 64), out=f("out", BF, 5, 4, 64),
                             k_out=f("k_out", BF, 5, 2, 64)),
        "append": lambda: cache.append_rotated(f("q", BF, 5, 4, 64), f("k", BF, 5, 2, 64), f("v", BF, 5, 2, 64),
                                               f("slots", I32, 5), f("positions", I32, 5), rope, q_out=f("q_out", BF, 5, 4, 64),
                                               device_status=status),
        "update": lambda: index.update(**step, max_q=3, device_status=status),
        "select": lambda: index.select(f("q", BF, 5, 4, 64), **step, max_q=3, top=4, blocks=f("blocks", I32, 5, 2, 4),
                                       device_status=status),
        "sparse": lambda: cache.sparse_attention(f("q", BF, 5, 4, 64), **step, blocks=f("blocks", I32, 5, 2, 4),
                                                 block_tokens=32, max_q=3, out=f("out", BF, 5, 4, 64),
                                                 lse=f("lse", torch.float32, 5, 4), device_status=status)}


@pytest.fixture
def module(monkeypatch, L):  # noqa: F811
    """block.py with GPU 0 the current one and the C calls replaced by a record of them."""
    from nvfp4_mixture_experts_moe_gb300 import block as m
    reached = []
    for name in ("moe_rope", "moe_kv4_append_rope", "moe_kv4_index_update", "moe_kv4_select", "moe_kv4_sparse_attention"):
        monkeypatch.setattr(m.B, name, lambda *a, name=name: reached.append(name))
    monkeypatch.setattr(m, "_where", lambda stream: (0, 0))
    m.reached = reached
    yield m
    del m.reached


@pytest.mark.parametrize("call,names", [
    ("rope", ("q", "k", "positions", "out", "k_out")), ("append", ("q", "k", "v", "slots", "positions", "q_out", "device_status")),
    ("update", ("cu_q", "kv_len", "block_table", "device_status")),
    ("select", ("q", "cu_q", "kv_len", "block_table", "blocks", "device_status")),
    ("sparse", ("q", "cu_q", "kv_len", "block_table", "blocks", "out", "lse", "device_status"))])
@pytest.mark.parametrize("gpu", [1, -1])
def test_tensors_elsewhere_are_refused(module, call, names, gpu):
    _calls(module)[call]()
    for name in names:
        with pytest.raises(ValueError):
            _calls(module, **{name: gpu})[call]()
    with pytest.raises(ValueError):
        _calls(module, objects_gpu=1)[call]()
    assert len(module.reached) == 1


def test_wrong_shapes_and_numbers_are_value_errors(module):
    cache, rope, index = _objects(module)
    two = module.Rope(64, sections=(12, 20), device="cpu")
    two._dev = 0
    F = lambda dtype, *shape: Fake(0, dtype, *shape)  # noqa: E731
    q, k, s = F(BF, 5, 4, 64), F(BF, 5, 2, 64), F(I32, 5)
    step = dict(cu_q=F(I32, 3), kv_len=F(I32, 2), block_table=F(I32, 2, 4))
    blocks = F(I32, 5, 2, 4)
    bad = [
        lambda: rope(F(BF, 5, 256), s), lambda: rope(F(torch.float32, 5, 4, 64), s), lambda: rope(q, F(I32, 6)),
        lambda: rope(q, F(torch.int64, 5)), lambda: rope(q, s, k=F(BF, 6, 2, 64)), lambda: rope(q, s, k=F(BF, 5, 2, 32)),
        lambda: rope(q, s, out=F(BF, 6, 4, 64)), lambda: rope(q, F(I32, 2, 5)), lambda: two(q, s), lambda: two(q, F(I32, 3, 5)),
        lambda: cache.append_rotated(q, k, F(BF, 4, 2, 64), s, s, rope), lambda: cache.append_rotated(F(BF, 4, 4, 64), k, k, s, s, rope),
        lambda: cache.append_rotated(q, k, k, s, F(I32, 4), rope, q_out=q), lambda: cache.append_rotated(q, k, k, F(I32, 4), s, rope, q_out=q),
        lambda: cache.append_rotated(q, k, k, s, s, rope, q_out=F(BF, 6, 4, 64)), lambda: cache.append_rotated(F(BF, 5, 4, 32), k, k, s, s, rope),
        lambda: index.update(**{**step, "cu_q": F(I32, 2)}, max_q=3), lambda: index.update(**step, max_q=2.5),
        lambda: index.update(**step, max_q=2 ** 40), lambda: index.update(**{**step, "kv_len": F(I32, 2, 1)}, max_q=3),
        lambda: index.select(q, **step, max_q=3, top=4, blocks=F(I32, 5, 2, 5)), lambda: index.select(q, **step, max_q=3, top=4.5, blocks=blocks),
        lambda: index.select(q, **step, max_q=2 ** 40, top=4, blocks=blocks), lambda: index.select(q, **step, max_q=3, top=4, sink="1", blocks=blocks),
        lambda: index.select(F(BF, 5, 4, 128), **step, max_q=3, top=4, blocks=blocks),
        lambda: cache.sparse_attention(q, **step, blocks=F(I32, 4, 2, 4), block_tokens=32, max_q=3, out=q),
        lambda: cache.sparse_attention(q, **step, blocks=F(I32, 5, 3, 4), block_tokens=32, max_q=3, out=q),
        lambda: cache.sparse_attention(q, **step, blocks=F(I32, 5, 2), block_tokens=32, max_q=3, out=q),
        lambda: cache.sparse_attention(q, **step, blocks=blocks, block_tokens=32, max_q=None, out=q),
        lambda: cache.sparse_attention(q, **step, blocks=blocks, block_tokens=32, max_q=3, scale="x", out=q),
        lambda: module.Rope(63), lambda: module.Rope(64.0), lambda: module.Rope(64, pairs="both"), lambda: module.Rope(64, sections=(1, 2)),
        lambda: module.Rope(64, inv_freq=[1.0]), lambda: module.Rope(64, axes=[4] * 32), lambda: module.Rope(0),
        lambda: module.Rope(64, sections=(32,), axes=[0] * 32), lambda: module.Rope(10, sections=(1, 1, 1, 1, 1)),
        lambda: module.Kv4BlockIndex(cache, 48), lambda: module.Kv4BlockIndex(cache, 2 ** 32 + 64),
        lambda: module.Kv4BlockIndex(cache, 32, means=F(torch.float16, 8, 2, 64)),
        lambda: module.Kv4BlockIndex(cache, 32, means=F(BF, 4, 2, 64))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(str(i))
    assert not module.reached
