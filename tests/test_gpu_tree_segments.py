"""kvc_gqa_tree where a CTA goes through many rows of the batch, of one to a few key tiles each: what the
two halves of a row hand each other at its end stays apart from the next row's first tile.  The output is
within the bound of the 64-bit form, and the same bits in every run."""
import pytest
import torch

from test_gpu_tree import BF16, F16, Case, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


@pytest.mark.parametrize("B,H,G,D,C,N,page,window,dtype", [
    (90, 8, 1, 128, 120, 3, 0, 0, BF16),      # a tile a row, five rows a CTA
    (60, 8, 16, 64, 192, 20, 64, 0, F16),     # three row tiles of a tile or two
    (40, 8, 4, 128, 700, 33, 0, 100, BF16),   # one to three tiles under a window
    (50, 8, 2, 256, 320, 9, 64, 0, BF16),
])
def test_many_rows_of_few_tiles(K, B, H, G, D, C, N, page, window, dtype):
    g = gen(B + D)
    past = [int(torch.randint(0, C - N + 1, (), generator=g)) for _ in range(B)]
    c = Case(K, g, B, H, G, D, C, N, past, page, dtype)
    c.append()
    ws = K.tree_workspace(c.gpu["q"], c.gpu["k"])
    want = c.attend(window, rows=[0, H - 1], workspace=ws)
    out = torch.empty_like(want)
    for _ in range(50):
        out.fill_(7.0)
        K.kvc_gqa_tree(out, c.gpu["q"], c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, block_table=c.gpu_table,
                       local_window_size=window, rope=c.gpu_rope, workspace=ws)
        assert torch.equal(out, want)
