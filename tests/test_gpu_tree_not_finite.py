"""kvc_gqa_tree where single values of V are NaN or infinite: that column is NaN for the nodes that see the
row, wherever in a key tile and in whichever tile it lies and however small its weight; every other value keeps
its bits."""
import pytest
import torch

from test_gpu_tree import BF16, F16, Case, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def attend(K, c, window, ws):
    out = torch.full_like(c.gpu["q"], 7.0)
    K.kvc_gqa_tree(out, c.gpu["q"], c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, block_table=c.gpu_table,
                   local_window_size=window, rope=c.gpu_rope, workspace=ws, status=c.st)
    return out.cpu()


def seen(c, b, row, window):
    """the nodes of batch row b that see cache row `row`"""
    P, out = c.past[b], []
    for i, line in enumerate(c.lines[b]):
        if not line:
            continue
        at = P + len(line) - 1
        pos = row if row < P else P + len(c.lines[b][row - P]) - 1
        if (row < P or row - P in line) and (window <= 0 or at - pos < window):
            out.append(i)
    return out


TREE = [-1, 0, 0, 1, -2, 2, 3, 3, 6, 7, 8, 4, 10, -1]


@pytest.mark.parametrize("window", [0, 130])
@pytest.mark.parametrize("dtype,D,G,page", [(BF16, 128, 4, 0), (F16, 64, 12, 64), (BF16, 64, 1, 0), (F16, 128, 16, 192), (BF16, 256, 3, 64),
                                            (F16, 256, 2, 0)])
def test_one_column(K, dtype, D, G, page, window):
    N, C = len(TREE), 1152
    past = [C - N, 520, 131, 250]
    c = Case(K, gen(D + G), 4, 2, G, D, C, N, past, page, dtype, trees=[TREE] * 4)
    c.append()
    ws = K.tree_workspace(c.gpu["q"], c.gpu["k"])
    want = attend(K, c, window, ws)
    assert torch.isfinite(want).all()
    g = gen(5)
    kept = c.gpu["v"].clone()
    # rows below P by this much, or (negative) drafts; in every case another column of another head
    spots = [1, 2, 5, 62, 64, 100, 125, 126, 127, 128, 130, 131, 200, 249, 250, 500, 900, -1, -4, -6, -9, -13]
    for value in (float("nan"), float("inf"), -float("inf")):
        for spot in spots:
            col, head = int(torch.randint(0, D, (), generator=g)), int(torch.randint(0, 2, (), generator=g))
            expect = want.clone()
            c.gpu["v"].copy_(kept)
            for b, P in enumerate(past):
                row = P - spot
                if row < 0:
                    continue
                x, y = c.at(b, [row])
                c.gpu["v"][x.cuda(), head, y.cuda(), col] = value
                for i in seen(c, b, row, window):
                    expect[b, head * G:(head + 1) * G, i, col] = float("nan")
            got = attend(K, c, window, ws)
            assert torch.equal(torch.isnan(got), torch.isnan(expect)), (value, spot, col, head)
            assert torch.equal(got.nan_to_num(9.0), expect.nan_to_num(9.0)), (value, spot, col, head)
    assert c.st.item() == 0


@pytest.mark.parametrize("dtype,D,page", [(BF16, 128, 0), (F16, 64, 64), (BF16, 256, 0)])
def test_many_at_once(K, dtype, D, page):
    """a tenth of the rows with a few such values each, of all three kinds, among them rows that nobody sees"""
    N, C, G = len(TREE), 640, 4
    past = [C - N, 300]
    c = Case(K, gen(D), 2, 2, G, D, C, N, past, page, dtype, trees=[TREE] * 2)
    c.append()
    ws = K.tree_workspace(c.gpu["q"], c.gpu["k"])
    for window in (0, 40):
        want = attend(K, c, window, ws)
        expect, g, kept = want.clone(), gen(window), c.gpu["v"].clone()
        for b, P in enumerate(past):
            for row in range(C):
                if float(torch.rand((), generator=g)) < 0.1 and (row >= P - 12 or window):
                    x, y = c.at(b, [row])
                    head, cols = row % 2, torch.randint(0, D, (3,), generator=g)
                    kinds = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=dtype).cuda()
                    c.gpu["v"][x.cuda(), head, y.cuda()] = c.gpu["v"][x.cuda(), head, y.cuda()].index_copy(1, cols.cuda(), kinds[None])
                    if row < P + N:
                        for i in seen(c, b, row, window):
                            expect[b, head * G:(head + 1) * G, i, cols] = float("nan")
        got = attend(K, c, window, ws)
        c.gpu["v"].copy_(kept)
        assert torch.equal(torch.isnan(got), torch.isnan(expect)) and torch.isnan(expect).any()
        assert torch.equal(got.nan_to_num(9.0), expect.nan_to_num(9.0))


@pytest.mark.parametrize("C,N,heads", [(4000, 8, 1), (300, 8, 8)])
def test_a_weight_too_small_for_a_number(K, C, N, heads):
    """the row's key scores far below the others': its weight is zero in 32 bits, in the tile or in the join of parts"""
    D, G = 128, 2
    c = Case(K, gen(3), 1, heads, G, D, C, N, [C - N], 0, BF16, rope=False)
    c.append()
    ws = K.tree_workspace(c.gpu["q"], c.gpu["k"])
    # all queries and keys along one line, one row against it
    c.gpu["q"].fill_(4.0)
    c.gpu["k"].fill_(4.0)
    far = C - N - 40
    c.gpu["k"][0, :, :far + 1] = -4.0
    want = attend(K, c, 0, ws)
    c.gpu["v"][0, 0, far, 17] = float("inf")
    c.gpu["v"][0, 0, 5, 99] = float("nan")
    got = attend(K, c, 0, ws)
    for i, line in enumerate(c.lines[0]):
        if line:
            want[0, :G, i, 17] = want[0, :G, i, 99] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))
