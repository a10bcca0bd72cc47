"""Host-side limits and checks of positions, block means, selection and sparse attention (include/moe_block.h, block.py)
at their corners: no GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

from test_block_host import BF, Fake, I32, U8
from test_oracle_block import L, _cache  # noqa: F401
from test_sparse_host import _index, _objects, _reaches_device, _select, bind, module, needs_no_gpu  # noqa: F401


# -------------------------------------------------- blocks of several pages

@needs_no_gpu
def test_blocks_of_several_pages_need_owners(L):  # noqa: F811
    B = bind()
    small = _cache(B, page_tokens=32)

    def both(**kw):
        index = _index(B, small, **kw)
        return (L.moe_kv4_index_update(ctypes.byref(index), 2, 3, 4, 256, 256, 256, None, None),
                L.moe_kv4_select(ctypes.byref(_select(B, index)), None))
    assert both() == both(owners=258) == (B.MOE_ERR_INVALID_ARG,) * 2
    assert all(_reaches_device(st, B) for st in both(owners=260) + both(block_tokens=32))


def test_owners_of_an_index(module):  # noqa: F811
    cache, _, index = _objects(module)                       # pages of 16, blocks of 32
    assert index.owners.tolist() == [-1] * 4 and index.desc.owners == index.owners.data_ptr()
    means = lambda *shape: Fake(0, torch.float16, *shape)  # noqa: E731
    kept = Fake(0, I32, 4)
    assert module.Kv4BlockIndex(cache, 64, means=means(4, 2, 64), owners=kept).owners is kept
    for bad in (Fake(0, I32, 5), Fake(0, torch.int64, 4), Fake(1, I32, 4)):
        with pytest.raises(ValueError):
            module.Kv4BlockIndex(cache, 64, means=means(4, 2, 64), owners=bad)
    large = module.Kv4Cache(4, 64, 2, 64, 1.0, 1.0, pool=Fake(0, U8, 4 * 64 * 2 * 72))
    plain = module.Kv4BlockIndex(large, 64, means=means(4, 2, 64))
    assert plain.owners is None and not plain.desc.owners
    with pytest.raises(ValueError):
        module.Kv4BlockIndex(large, 64, means=means(4, 2, 64), owners=kept)


# ------------------------------------------------------------ whole numbers

@pytest.mark.parametrize("whole", [np.int32, np.int64, np.uint8])
def test_whole_numbers_of_any_type(module, whole):  # noqa: F811
    """What counts as an index does as a size: lengths often come out of an array."""
    cache, _, index = _objects(module)
    F = lambda dtype, *shape: Fake(0, dtype, *shape)  # noqa: E731
    step = dict(cu_q=F(I32, 3), kv_len=F(I32, 2), block_table=F(I32, 2, 4))
    index.update(**step, max_q=whole(3))
    q, blocks = F(BF, 5, 4, 64), F(I32, 5, 2, 4)
    assert index.select(q, **step, max_q=whole(3), top=whole(4), sink=whole(1), local=whole(1), blocks=blocks) is blocks
    assert index.select(q, **step, max_q=3, top=whole(4)).shape == (5, 2, 4)
    cache.sparse_attention(q, **step, blocks=blocks, block_tokens=whole(32), max_q=whole(3), out=q)
    assert module.reached == ["moe_kv4_index_update", "moe_kv4_select", "moe_kv4_select", "moe_kv4_sparse_attention"]
    assert module.Rope(whole(64), device="cpu")._fields[0] == 64
    assert module.Kv4BlockIndex(cache, whole(32), means=F(torch.float16, 4, 2, 64)).desc.block_tokens == 32


def test_what_is_no_whole_number_is_a_value_error(module):  # noqa: F811
    cache, _, index = _objects(module)
    F = lambda dtype, *shape: Fake(0, dtype, *shape)  # noqa: E731
    step = dict(cu_q=F(I32, 3), kv_len=F(I32, 2), block_table=F(I32, 2, 4))
    q, means = F(BF, 5, 4, 64), F(torch.float16, 4, 2, 64)
    for i, f in enumerate((lambda x: index.update(**step, max_q=x), lambda x: index.select(q, **step, max_q=3, top=x),
                           lambda x: module.Rope(x, device="cpu"), lambda x: module.Kv4BlockIndex(cache, x, means=means))):
        for x in (32.0, np.float32(32), "32", None, 2 ** 40, -(2 ** 40)):
            with pytest.raises(ValueError):
                f(x)
                pytest.fail(f"{i} {x!r}")
    assert not module.reached
