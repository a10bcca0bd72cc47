"""Corners of the contracts of positions, block means, selection and sparse attention (include/moe_block.h) on the GPU.
Bars as in test_gpu_sparse.py."""
import numpy as np
import pytest
import torch

from test_gpu_block import Scene, built  # noqa: F401
from test_gpu_sparse import _attend, _check_sparse

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
