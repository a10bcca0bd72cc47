"""Corners of the block operators' contracts (include/moe_block.h) on the GPU."""
import numpy as np
import pytest
import torch

from test_gpu_block import Scene, built  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- bad queries

# Few rows in one range and cut across CTAs; many rows whole, of few rows (split over their tiles), and cut.
@pytest.mark.parametrize("qheads,heads,D,lens", [
    (8, 2, 64, [(300, 1), (90, 1)]), (8, 2, 128, [(90, 4), (300, 4)]), (8, 2, 128, [(3, 1), (20000, 1)]),
    (16, 1, 128, [(50, 1), (20000, 1)]), (16, 1, 64, [(9000, 1)]), (8, 2, 64, [(300, 40), (90, 40)]),
    (8, 2, 128, [(700, 300)]), (8, 2, 128, [(40, 9), (90, 9)]), (8, 2, 64, [(16000, 9)]), (8, 2, 128, [(16000, 70)])])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_query_gives_nan_rows(qheads, heads, D, lens, value):
    """A row with a NaN, or an infinity (inf * 0, inf - inf), is NaN in `out` and `lse`: zeros and -inf are what a row
    that sees nothing gives."""
    s = Scene(lens, qheads, heads, D, 32, seed=len(lens) + D)
    good, lse = s.run(want_lse=True)
    assert bool(torch.isfinite(good.float()).all()) and bool(torch.isfinite(lse).all())
    q = s.q.clone().cuda()
    row, head = s.total - 1, 3 % qheads        # the last request's last token
    q[row, head, 5] = value
    out, lse2 = s.run(q=q, want_lse=True)
    assert bool(torch.isnan(out[row, head]).all()) and bool(torch.isnan(lse2[row, head]))
    keep = torch.ones(s.total, qheads, dtype=torch.bool, device="cuda")
    keep[row, head] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse2[keep], lse[keep])
