"""Host-side limits and checks of the block operators' entry points (include/moe_block.h, block.py): no GPU needed."""
import ctypes

import pytest
import torch

from test_oracle_block import L, _attn, _cache  # noqa: F401


# ------------------------------------------------------------- 32-bit sizes

@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_tables_whose_lengths_round_past_32_bits_are_refused(L, page):  # noqa: F811
    from nvfp4_mixture_experts_moe_gb300 import binding as B

    def size(max_pages):
        c = _cache(B, page_tokens=page, kv_heads=1)
        return B.moe_kv4_attention_workspace_size(_attn(B, cache=c, batch=1, q_heads=1, max_pages=max_pages))
    most = (2 ** 31 - 129) // page          # a length up to here rounds up to a multiple of 128 below 2^31
    assert size(most) > 0
    assert all(size(p) == 0 for p in (most + 1, (2 ** 31 - 1) // page))


# ------------------------------------------------------------------ overlaps

def _step(**kw):
    from nvfp4_mixture_experts_moe_gb300 import binding as B
    d = dict(batch=3, page_tokens=16, max_pages=4, tokens=5, free_capacity=8, device_status=0xB000)
    d.update({n: 0x1000 * (i + 1) for i, n in enumerate(
        ("ctx_len", "new_len", "block_table", "free_pages", "free_count", "free_count_out", "kv_len", "cu_q", "slots",
         "positions"))})
    d.update(kw)
    return d, B.MoeKvStepArgs(**d)


STEP_SIZES = dict(ctx_len=3, new_len=3, block_table=12, free_pages=8, free_count=1, free_count_out=1, kv_len=3, cu_q=4,
                  slots=5, positions=5, device_status=1)
STEP_OUTPUTS = ("block_table", "free_count_out", "kv_len", "cu_q", "slots", "positions", "device_status")


@pytest.mark.parametrize("out", STEP_OUTPUTS)
@pytest.mark.parametrize("other", STEP_SIZES)
def test_step_refuses_outputs_that_overlap(L, out, other):  # noqa: F811
    """Equal addresses, and one element shared at either end; arrays that touch are fine as far as this check goes."""
    from nvfp4_mixture_experts_moe_gb300 import binding as B
    if out == other:
        return
    d, args = _step()
    call = lambda a: L.moe_kv_step(ctypes.byref(a), None)   # noqa: E731
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only without a GPU, where a call that passes the checks ends at the device")
    assert call(args) not in (B.MOE_OK, B.MOE_ERR_INVALID_ARG)
    for at in (d[other], d[other] + 4 * (STEP_SIZES[other] - 1), d[other] - 4 * (STEP_SIZES[out] - 1)):
        assert call(_step(**{out: at})[1]) == B.MOE_ERR_INVALID_ARG, at
    for at in (d[other] + 4 * STEP_SIZES[other], d[other] - 4 * STEP_SIZES[out]):
        assert call(_step(**{out: at})[1]) not in (B.MOE_OK, B.MOE_ERR_INVALID_ARG), at


def test_step_arrays_of_no_length_overlap_nothing(L):  # noqa: F811
    from nvfp4_mixture_experts_moe_gb300 import binding as B
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    d, _ = _step()
    _, a = _step(tokens=0, slots=d["ctx_len"], positions=d["ctx_len"], device_status=None)
    assert L.moe_kv_step(ctypes.byref(a), None) not in (B.MOE_OK, B.MOE_ERR_INVALID_ARG)


# ------------------------------------------------------------------- devices

class Fake:
    """Answers as a contiguous tensor on a GPU would."""
    is_cuda, device = True, torch.device("cpu")

    def __init__(self, gpu, dtype, *shape):
        self.gpu, self.dtype, self.shape = gpu, dtype, torch.Size(shape)

    def get_device(self):
        return self.gpu

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 256


BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def _calls(block, gpu=0, cache_gpu=0, **where):
    """Every call of block.py with the named arguments on another GPU."""
    def f(name, dtype, *shape):
        return Fake(where.get(name, gpu), dtype, *shape)
    cache = block.Kv4Cache(4, 16, 2, 64, 1.0, 1.0, pool=Fake(cache_gpu, U8, 4 * 16 * 2 * 72))
    cache.status = Fake(cache_gpu, I32, 1)
    step = block.KvStep(2, 5, 16, 4, device="cpu")
    step._dev = cache_gpu
    return {
        "append": lambda: cache.append(f("k", BF, 5, 2, 64), f("v", BF, 5, 2, 64), f("slots", I32, 5),
                                       device_status=f("device_status", I32, 1)),
        "read": lambda: cache.read(f("slots", I32, 5), device_status=f("device_status", I32, 1)),
        "attention": lambda: cache.attention(
            f("q", BF, 5, 4, 64), f("cu_q", I32, 3), f("kv_len", I32, 2), f("block_table", I32, 2, 4), max_q=3,
            out=f("out", BF, 5, 4, 64), lse=f("lse", torch.float32, 5, 4), ws=f("ws", U8, 1 << 30)),
        "step": lambda: step.run(f("ctx_len", I32, 2), f("new_len", I32, 2), f("block_table", I32, 2, 4),
                                 f("free_pages", I32, 9), f("free_count", I32, 1)),
        "norm": lambda: block.block_norm(f("x", BF, 3, 8), f("residual", BF, 3, 8), gate=f("gate", BF, 3, 8),
                                         w_post=f("w", BF, 8), w_pre=f("w_pre", BF, 8), out=f("out", BF, 3, 8),
                                         residual_out=f("residual_out", BF, 3, 8)),
        "norm, gate per channel": lambda: block.block_norm(f("x", BF, 3, 8), f("residual", BF, 3, 8), gate=f("gate", BF, 8),
                                                           w_pre=f("w_pre", BF, 8))}


@pytest.fixture
def block(monkeypatch, L):  # noqa: F811
    """The module, with GPU 0 the current one and the C calls replaced by a record of them."""
    from nvfp4_mixture_experts_moe_gb300 import block as module
    reached = []
    for name in ("moe_kv4_append", "moe_kv4_read", "moe_kv4_attention", "moe_kv_step", "moe_block_norm"):
        monkeypatch.setattr(module.B, name, lambda *a, name=name: reached.append(name))
    monkeypatch.setattr(module, "_where", lambda stream: (0, 0), raising=False)
    module.reached = reached
    yield module
    del module.reached


@pytest.mark.parametrize("call,names", [
    ("append", ("k", "v", "slots", "device_status")), ("read", ("slots", "device_status")),
    ("attention", ("q", "cu_q", "kv_len", "block_table", "out", "lse", "ws")),
    ("step", ("ctx_len", "new_len", "block_table", "free_pages", "free_count")),
    ("norm", ("x", "residual", "gate", "w", "w_pre", "out", "residual_out")), ("norm, gate per channel", ("gate",))])
@pytest.mark.parametrize("gpu", [1, -1])
def test_tensors_elsewhere_are_refused(block, call, names, gpu):
    """On another GPU, or on the CPU."""
    _calls(block)[call]()
    for name in names:
        with pytest.raises(ValueError):
            _calls(block, **{name: gpu})[call]()
    assert len(block.reached) == 1      # the one above


@pytest.mark.parametrize("call", ["append", "read", "attention", "step"])
def test_a_cache_or_step_of_another_gpu_is_refused(block, call):
    with pytest.raises(ValueError):
        _calls(block, cache_gpu=1)[call]()
    assert not block.reached


def test_cpu_tensors_are_refused(L):  # noqa: F811
    from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, KvStep, block_norm
    x, i = torch.zeros(3, 64, dtype=BF), torch.zeros(3, dtype=I32)
    for bad in (lambda: block_norm(x, x), lambda: KvStep(3, 3, 16, 1, device="cpu").run(i, i, i[:, None], i, i[:1]),
                lambda: Kv4Cache(2, 16, 2, 64, 1.0, 1.0, device="cpu")):
        with pytest.raises(ValueError):
            bad()


# -------------------------------------------------------------------- shapes

def _attention(block, **kw):
    cache = block.Kv4Cache(4, 16, 2, 64, 1.0, 1.0, pool=Fake(0, U8, 4 * 16 * 2 * 72))
    cache.status = Fake(0, I32, 1)
    a = dict(q=Fake(0, BF, 5, 4, 64), cu_q=Fake(0, I32, 3), kv_len=Fake(0, I32, 2), block_table=Fake(0, I32, 2, 4), max_q=3,
             ws=Fake(0, U8, 1 << 30))
    return cache.attention(**{**a, **kw})


def test_wrong_shapes_and_numbers_are_value_errors(block):
    _attention(block)
    for bad in (dict(q=Fake(0, BF, 5)), dict(q=Fake(0, BF, 5, 256)), dict(q=Fake(0, BF)), dict(q=Fake(0, BF, 5, 4, 64, 1)),
                dict(kv_len=Fake(0, I32)), dict(kv_len=Fake(0, I32, 2, 1)), dict(kv_len=Fake(0, I32, 3)),
                dict(cu_q=Fake(0, I32)), dict(cu_q=Fake(0, I32, 2)), dict(block_table=Fake(0, I32, 2)),
                dict(block_table=Fake(0, I32, 1, 4)), dict(max_q=2 ** 31), dict(max_q=1.5), dict(window=2 ** 31),
                dict(window=-2 ** 32), dict(scale="1")):
        with pytest.raises(ValueError):
            _attention(block, **bad)
    f = Fake(0, BF, 3, 8)
    for bad in (dict(eps="1"), dict(branch_scale=None), dict(gate=Fake(0, BF)),
                dict(gate=Fake(0, BF, 3, 8, 1)), dict(x=Fake(0, BF, 8))):
        with pytest.raises(ValueError):
            block.block_norm(**{**dict(x=f, residual=f), **bad})
    for bad in (Fake(0, BF), Fake(0, BF, 8)):
        with pytest.raises(ValueError):
            block.block_norm(f, bad)
    assert block.reached == ["moe_kv4_attention"]
    with pytest.raises(ValueError):
        block.Kv4Cache(4, 16, 2, 64, 1.0, 1.0, pool=Fake(0, U8, 4 * 16 * 2 * 72)).append(
            Fake(0, BF, 5, 2, 64), Fake(0, BF, 5, 2, 64), Fake(0, I32))
    for shape in ((), (3, 1)):
        with pytest.raises(ValueError):
            block.Kv4Cache(4, 16, 2, 64, 1.0, 1.0, pool=Fake(0, U8, 4 * 16 * 2 * 72)).read(Fake(0, I32, *shape))


def test_a_workspace_serves_every_smaller_call(L):  # noqa: F811
    from nvfp4_mixture_experts_moe_gb300 import binding as B

    def size(batch, heads, max_q, dim):
        return B.moe_kv4_attention_workspace_size(
            _attn(B, cache=_cache(B, kv_heads=1, head_dim=dim), batch=batch, q_heads=heads, max_q=max_q, total_q=batch * max_q))
    for dim in (64, 128):
        for batch in (1, 2, 9):
            for heads in (1, 8, 12, 16, 17, 32, 64):
                for max_q in (1, 2, 3, 16, 17, 100):
                    most = size(batch, heads, max_q, dim)
                    assert all(0 < size(b, h, m, dim) <= most for b in (1, 2, 9) if b <= batch
                               for h in (1, 4, 8, 16, 17, 24, 32) if h <= heads for m in (1, 2, 5, 16, 40) if m <= max_q)
