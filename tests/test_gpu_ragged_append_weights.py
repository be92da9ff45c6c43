"""Norm weights of kvc_ragged_append that are zero or no numbers: a column takes its own weight, and one that is turned
its partner's, and no other."""
import math

import pytest
import torch

from test_gpu_ragged_append import BF16, F16, Case, K, reference  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,turned", [(64, 32), (80, 16), (128, 128), (256, 240), (128, 0)])
@pytest.mark.parametrize("odd", [math.inf, -math.inf, math.nan, 0.0])
def test_weights(K, D, turned, inter, odd, dtype):  # noqa: F811
    c = Case(K, D + turned, 37, 4, 2, D, 16, dtype, turned, inter)
    at = [D - 1, turned // 2 + 1, turned // 4, min((turned + D) // 2, D - 1)]  # of columns that stay and of either half that is turned
    c.qw[at] = odd
    c.kw[at[:2]] = odd
    out, st = c.run()
    assert st == 0
    pos, slot = c.pos.long(), c.slot.long()
    where = (slot // c.page, slice(None), slot % c.page)
    for what, got, x, w in (("queries", out.cpu(), c.q, c.qw), ("keys", c.gkp.cpu()[where], c.k, c.kw)):
        want, bound = reference(x, w, c.eps, c.rope, pos, inter)
        numbers = want.isfinite()
        # (an infinity times a cosine, and the sum of two, as the definition has it)
        assert torch.equal(got.isnan(), want.isnan()), what
        assert torch.equal(got[~numbers & ~want.isnan()].double(), want[~numbers & ~want.isnan()]), what
        assert ((got.double() - want).abs() <= bound)[numbers].all(), what
