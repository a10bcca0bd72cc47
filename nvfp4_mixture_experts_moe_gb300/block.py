"""What a decoder block runs around the MoE layer when it serves tokens.

``KvStep`` places a step's new tokens in pages (``moe_kv_step``), ``Kv4Cache``
keeps one layer's keys and values as NVFP4 pages, appends to them, reads rows
back and attends over them (``moe_kv4_append``, ``moe_kv4_read``,
``moe_kv4_attention``), ``block_norm`` fuses the norm after a block, its gate,
the residual and the norm before the next block (``moe_block_norm``). The C
calls and their contracts are in ``include/moe_block.h``; torch only
allocates. A call runs on the current stream, or on ``stream=`` (a Stream or
a raw handle), on which its outputs and its own workspace are then made; what
the caller passes in has to be ready there. Wrong shapes, types or devices
raise ``ValueError``; what the C call refuses raises ``MoeError``.
"""
from __future__ import annotations

import struct

import torch

from . import binding as B


_UNPACKABLE = (struct.error, OverflowError)   # a number of the caller's that is none, or does not fit its field
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_C = torch._C


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _where(stream):
    """The current GPU, where kernels are launched, and the call's stream there as a handle (looked up once a call:
    each of these takes a good part of a launch's time). Every tensor of the call has to lie on that GPU."""
    try:
        dev = _C._cuda_getDevice()
    except (RuntimeError, AttributeError):   # no driver, or torch without CUDA: no tensor passes (the CPU's are -1)
        return -2, 0
    if stream is None:
        return dev, _C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != dev:
            raise ValueError(f"stream: one of GPU {stream.device_index}, the current one is {dev}")
        return dev, stream.cuda_stream
    return dev, int(stream)


def _ints(t, shape, what, dev):
    if not (t.get_device() == dev and t.dtype is _I32 and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{what}: a contiguous int32 tensor of shape {tuple(shape)} on the current GPU is needed")
    return t.data_ptr()


def _rows(t, heads, dim, what, dev):
    """Address and row stride of a bf16 [n, heads, dim] tensor whose rows' heads are contiguous."""
    shape = t.shape
    n = shape[0] if len(shape) == 3 else -1
    if not (t.get_device() == dev and t.dtype is _BF16 and shape == (n, heads, dim)):
        raise ValueError(f"{what}: a bf16 tensor [rows, {heads}, {dim}] on the current GPU is needed")
    st = t.stride()
    if n > 0 and not (st[2] == 1 and (heads == 1 or st[1] == dim)):
        raise ValueError(f"{what}: a row's heads have to be contiguous")
    return t.data_ptr(), (st[0] if n > 1 else heads * dim)


def _like(t, shape, dtype, what, dev):
    if not (t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{what}: a contiguous {dtype} tensor of shape {tuple(shape)} on the current GPU is needed")
    return t.data_ptr()


def _status(t, dev):
    """A ``device_status``: an int32 tensor (its first element is set) or an address."""
    if not isinstance(t, int) and not (t.get_device() == dev and t.dtype is _I32 and t.numel() > 0):
        raise ValueError("device_status: an int32 tensor on the current GPU is needed")
    return t


def _on(stream):
    """A context in which torch works on the stream of a call (None: the current one; a Stream; a raw handle)."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream, zeros=0):
    """An output or workspace (its first ``zeros`` elements zero) of a call on ``stream``.

    It is made on that stream: memory of the current one may still be used by work queued there, which the call does
    not wait for. It stays reserved for what the current stream has queued when the caller gives it back.
    """
    if stream is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        if zeros:
            t[:zeros].zero_()
        return t
    here = torch.cuda.current_stream()
    with _on(stream):
        t = _empty(shape, dtype, device, None, zeros)
        if torch.cuda.current_stream().cuda_stream != here.cuda_stream:
            t.record_stream(here)
    return t


class Kv4Cache:
    """Paged NVFP4 keys and values of one layer.

    ``k_gs`` and ``v_gs`` are the calibrated global scales in the quant
    convention (2688 / amax). ``pool`` may be given (uint8, layout in
    ``include/moe_block.h``); otherwise it is allocated, uninitialised. What
    the constructor makes is made on the current stream: a call on another one
    comes after it (``stream.wait_stream``).

    ``status`` (int32 ``[1]``) keeps what calls without a ``device_status`` or
    workspace of their own report (MOE_ERR_DEVICE: a slot or page id outside
    the pool, lengths past a bound; MOE_ERR_TIMEOUT); the caller clears it.
    """

    def __init__(self, num_pages, page_tokens, kv_heads, head_dim, k_gs, v_gs, device="cuda", pool=None):
        nbytes = B.moe_kv4_pool_size(num_pages, page_tokens, kv_heads, head_dim)
        _need(nbytes > 0, "cache sizes: page_tokens 16, 32, 64 or 128, head_dim 64 or 128, 1 to 1024 kv heads, "
                          "num_pages * page_tokens < 2^31")
        if pool is None:
            pool = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _need(pool.is_cuda and pool.dtype == torch.uint8 and pool.is_contiguous() and pool.numel() == nbytes,
              f"pool: a contiguous CUDA uint8 tensor of {nbytes} bytes is needed")
        self.num_pages, self.page_tokens = num_pages, page_tokens
        self.kv_heads, self.head_dim = kv_heads, head_dim
        self.pool = pool
        self.status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self._dev, self._scale = pool.get_device(), head_dim ** -0.5
        self._fields = (num_pages, page_tokens, kv_heads, head_dim, float(k_gs), float(v_gs), pool.data_ptr())
        self.desc = B.MoeKv4Cache(*self._fields)

    def append(self, k, v, slots, device_status=None, stream=None):
        """bf16 ``[tokens, kv_heads, head_dim]`` rows into the slots (int32; negative ones are skipped)."""
        dev, handle = _where(stream)
        if dev != self._dev:
            raise ValueError(f"the cache lies on GPU {self._dev}, the current one is {dev}")
        kp, ks = _rows(k, self.kv_heads, self.head_dim, "k", dev)
        vp, vs = _rows(v, self.kv_heads, self.head_dim, "v", dev)
        n = k.shape[0]
        if v.shape[0] != n:
            raise ValueError("k and v have different lengths")
        B.moe_kv4_append(self.desc, kp, vp, ks, vs, _ints(slots, (n,), "slots", dev), n,
                         self.status if device_status is None else _status(device_status, dev), handle)

    def read(self, slots, stream=None, device_status=None):
        """The slots' rows as bf16 (k, v) ``[n, kv_heads, head_dim]``; negative slots give zeros."""
        dev, handle = _where(stream)
        if dev != self._dev:
            raise ValueError(f"the cache lies on GPU {self._dev}, the current one is {dev}")
        n = slots.shape[0] if slots.dim() == 1 else -1
        at = _ints(slots, (n,), "slots", dev)
        shape = (n, self.kv_heads, self.head_dim)
        k = _empty(shape, _BF16, self.pool.device, stream)
        v = _empty(shape, _BF16, self.pool.device, stream)
        B.moe_kv4_read(self.desc, at, n, k.data_ptr(), v.data_ptr(),
                       self.status if device_status is None else _status(device_status, dev), handle)
        return k, v

    def attention_workspace(self, total_q, batch, q_heads, max_q, max_pages=1, stream=None):
        """A workspace for calls of up to these sizes on ``stream``; its leading bytes start at zero."""
        a = B.MoeKv4AttnArgs(cache=self.desc, batch=batch, q_heads=q_heads, total_q=total_q, max_q=max_q,
                             max_pages=max_pages, scale=1.0, causal=1)
        n = B.moe_kv4_attention_workspace_size(a)
        _need(n > 0, "attention sizes outside the limits")
        return _empty(n, torch.uint8, self.pool.device, stream, B.MOE_KV4_WS_ZERO)

    def attention(self, q, cu_q, kv_len, block_table, max_q, scale=None, causal=True, window=0, want_lse=False,
                  out=None, lse=None, ws=None, stream=None):
        """Attention of ``q`` (bf16 ``[total_q, q_heads, head_dim]``) over the cached tokens.

        ``cu_q`` int32 ``[batch + 1]``, ``kv_len`` int32 ``[batch]`` (new
        tokens included, already appended), ``block_table`` int32 ``[batch,
        max_pages]``, ``max_q`` a bound on every request's query rows.
        Returns (out, lse); lse (fp32 ``[total_q, q_heads]``) is None unless
        wanted or given. Bad device data and waits that gave up are reported
        in ``ws`` (``moe_get_device_status``), or without one in ``status``.
        """
        dev, handle = _where(stream)
        if dev != self._dev:
            raise ValueError(f"the cache lies on GPU {self._dev}, the current one is {dev}")
        try:
            total_q, heads, _ = q.shape
            batch, = kv_len.shape
            _, max_pages = block_table.shape
        except ValueError:
            raise ValueError("q [rows, heads, dim], kv_len [batch] and block_table [batch, max_pages] are needed") from None
        qp, qs = _rows(q, heads, self.head_dim, "q", dev)
        shape = (total_q, heads, self.head_dim)
        if out is None:
            out = _empty(shape, _BF16, q.device, stream)
            op = out.data_ptr()
        else:
            op = _like(out, shape, _BF16, "out", dev)
        if lse is None and want_lse:
            lse = _empty((total_q, heads), _F32, q.device, stream)
        lp = 0 if lse is None else _like(lse, (total_q, heads), _F32, "lse", dev)
        own = ws is None
        if own:
            ws = self.attention_workspace(total_q, batch, heads, max_q, max_pages, stream)
        elif ws.get_device() != dev:
            raise ValueError("ws: a tensor on the current GPU is needed")
        try:
            a = B.PACK_KV4_ATTN.pack(*self._fields, batch, heads, total_q, max_q, max_pages, qp, qs,
                                     _ints(cu_q, (batch + 1,), "cu_q", dev), _ints(kv_len, (batch,), "kv_len", dev),
                                     _ints(block_table, (batch, max_pages), "block_table", dev),
                                     self._scale if scale is None else scale, 1 if causal else 0, window, op, lp)
        except _UNPACKABLE as e:
            raise ValueError(f"max_q, scale or window: {e}") from None
        B.moe_kv4_attention(a, ws, handle)
        if own:
            with _on(stream):
                torch.maximum(self.status, ws[:4].view(_I32), out=self.status)
        return out, lse


class KvStep:
    """One step's tables for up to ``batch`` requests and ``tokens`` new tokens.

    Holds the outputs, rewritten by every ``run``: ``kv_len`` ``[batch]``,
    ``cu_q`` ``[batch + 1]``, ``slots`` and ``positions`` ``[tokens]``,
    ``free_count`` ``[1]``, and ``status`` ``[1]``, which ``run`` sets to
    MOE_ERR_DEVICE when a request was refused, or its lengths or a page id were
    bad (the caller clears it). They are made on the current stream: a run on
    another one comes after it (``stream.wait_stream``).
    """

    def __init__(self, batch, tokens, page_tokens, max_pages, device="cuda"):
        self.batch, self.tokens, self.page_tokens, self.max_pages = batch, tokens, page_tokens, max_pages
        made = [torch.empty(n, dtype=torch.int32, device=device) for n in (batch, batch + 1, tokens, tokens, 1)]
        self.kv_len, self.cu_q, self.slots, self.positions, self.free_count = made
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._dev = self.status.get_device()
        self._outs = [t.data_ptr() for t in (self.free_count, self.kv_len, self.cu_q, self.slots, self.positions,
                                             self.status)]

    def run(self, ctx_len, new_len, block_table, free_pages, free_count, stream=None):
        """Extends ``block_table`` (int32 ``[batch, max_pages]``) in place and fills the outputs.

        ``free_pages[:free_count]`` is the stack of free pages, taken from its
        top; ``self.free_count`` says how many are left. The next step's
        ``ctx_len`` and ``free_count`` are copies of ``kv_len`` and
        ``self.free_count`` (they may not be these very tensors).
        """
        dev, handle = _where(stream)
        if dev != self._dev:
            raise ValueError(f"the step's outputs lie on GPU {self._dev}, the current one is {dev}")
        b = self.batch
        cap = free_pages.shape[0] if free_pages.dim() == 1 else -1
        a = B.PACK_KV_STEP.pack(b, self.page_tokens, self.max_pages, self.tokens, cap,
                                _ints(ctx_len, (b,), "ctx_len", dev), _ints(new_len, (b,), "new_len", dev),
                                _ints(block_table, (b, self.max_pages), "block_table", dev),
                                _ints(free_pages, (cap,), "free_pages", dev),
                                _ints(free_count, (1,), "free_count", dev), *self._outs)
        B.moe_kv_step(a, handle)
        return self


def _matrix(t, T, H, what, dev):
    if not (t.get_device() == dev and t.dtype is _BF16 and t.shape == (T, H)):
        raise ValueError(f"{what}: a bf16 tensor [{T}, {H}] on the current GPU is needed")
    st = t.stride()
    if st[1] != 1 and H > 1:
        raise ValueError(f"{what}: contiguous rows are needed")
    return t.data_ptr(), (st[0] if T > 1 else H)


def block_norm(x, residual, gate=None, w_post=None, w_pre=None, residual_scale=1.0, branch_scale=1.0, eps=1e-6,
               w_offset=0.0, residual_out=None, out=None, stream=None):
    """Norm after a block, gate, residual, norm before the next block, in one pass.

    ``r = residual_scale * residual + branch_scale * gate * rms(x) * (w_post +
    w_offset)``, ``out = rms(r) * (w_pre + w_offset)``; ``x`` bf16 ``[T, H]``
    or None (only the norm before), ``residual`` bf16 or fp32 ``[T, H]``,
    ``gate`` bf16 ``[T, H]`` or ``[H]``. Returns (r, out); out is None without
    ``w_pre``. ``residual_out`` may be ``residual`` itself.
    """
    (dev, handle), dtype = _where(stream), residual.dtype
    if not (residual.get_device() == dev and residual.dim() == 2 and (dtype is _BF16 or dtype is _F32)):
        raise ValueError("residual: a bf16 or fp32 tensor [T, H] on the current GPU is needed")
    T, H = shape = residual.shape
    rs = residual.stride()
    if rs[1] != 1 and H > 1:
        raise ValueError("residual: contiguous rows are needed")
    xp, xs = (0, 0) if x is None else _matrix(x, T, H, "x", dev)
    if gate is None:
        gp, gst = 0, 0
    elif gate.dim() == 1:
        gp, gst = _like(gate, (H,), _BF16, "gate", dev), 0
    else:
        gp, gst = _matrix(gate, T, H, "gate", dev)
    if residual_out is None:
        residual_out = _empty(shape, dtype, residual.device, stream)
        rp = residual_out.data_ptr()
    else:
        rp = _like(residual_out, shape, dtype, "residual_out", dev)
    if w_pre is None:
        out, op, wp = None, 0, 0
    else:
        wp = _like(w_pre, (H,), _BF16, "w_pre", dev)
        if out is None:
            out = _empty(shape, _BF16, residual.device, stream)
            op = out.data_ptr()
        else:
            op = _like(out, shape, _BF16, "out", dev)
    try:
        a = B.PACK_BLOCK_NORM.pack(T, H, xp, xs, gp, gst, residual.data_ptr(), rs[0] if T > 1 else H,
                                   1 if dtype is _F32 else 0,
                                   0 if w_post is None else _like(w_post, (H,), _BF16, "w_post", dev), wp,
                                   residual_scale, branch_scale, eps, w_offset, rp, op)
    except _UNPACKABLE as e:
        raise ValueError(f"scales, eps or w_offset: {e}") from None
    B.moe_block_norm(a, handle)
    return residual_out, out
