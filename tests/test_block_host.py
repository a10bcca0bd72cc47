"""Host-side limits and checks of the block operators' entry points (include/moe_block.h, block.py): no GPU needed."""
import ctypes

import pytest

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
