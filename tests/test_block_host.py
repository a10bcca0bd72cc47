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
