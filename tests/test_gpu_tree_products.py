"""kvc_gqa_tree over rows of many key tiles at every head_dim, rotated (two parts of the query) and not: the scores of a
tile are written where the products of the tile before last read their weights.  Within the bound of the 64-bit form, and
the same bits in every run, alone and beside another stream's call."""
import pytest
import torch

from test_gpu_tree import BF16, F16, Case, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("D,dtype,page", [(64, BF16, 0), (64, F16, 64), (128, BF16, 192), (128, F16, 0), (256, BF16, 0), (256, F16, 64)])
def test_long_rows(K, D, dtype, page, rope):
    N, C = 24, 9600
    c = Case(K, gen(D), 3, 4, 4, D, C, N, [C - N, 5000, 2111], page, dtype, rope=rope)
    c.append()
    ws = [K.tree_workspace(c.gpu["q"], c.gpu["k"]) for _ in range(2)]
    want = c.attend(rows=[0, 3], workspace=ws[0])
    outs = [torch.empty_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(30):
        for out, w, s in zip(outs, ws, streams):
            s.wait_stream(torch.cuda.current_stream())
            K.kvc_gqa_tree(out, c.gpu["q"], c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, block_table=c.gpu_table,
                           rope=c.gpu_rope, workspace=w, stream=s)
            if i % 2:
                s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
