"""kvc_gqa_decode_sparse where single values of V are NaN or infinite: that column is NaN for the queries of its
head when the page is read, however small the row's weight; every other value keeps its bits."""
import pytest
import torch

from test_gpu_sparse import BF16, F16, all_bounds, gen, lengths, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


@pytest.mark.parametrize("dtype,D,G,page,n", [(BF16, 64, 4, 64, 6), (F16, 64, 16, 64, 20), (BF16, 128, 2, 128, 3), (F16, 128, 12, 64, 6),
                                              (BF16, 256, 8, 64, 9), (F16, 256, 1, 192, 2)])
def test_one_column(K, dtype, D, G, page, n):
    B, H, m = 2, 2, 20
    totals = [m * page, 5 * page + 9]
    g = gen(D + G)
    table, k, v = make(g, B, H, D, page, m, dtype)
    q = torch.randn((B, H * G, 1, D), generator=g).to(dtype)
    d = [x.cuda() for x in (q, k, v, *all_bounds(k), table)]
    L = lengths(K, totals, 1, m * page)
    selected = torch.zeros((B, H, n), dtype=torch.int32, device="cuda")
    ws = K.sparse_workspace(d[0], d[1], selected)

    def attend():
        return K.kvc_gqa_decode_sparse(torch.full_like(d[0], 7.0), *d, L, selected, 0, 1, workspace=ws).cpu()

    want = attend()
    chosen = selected.tolist()
    assert torch.isfinite(want).all()
    kept = d[2].clone()
    for value in (float("nan"), float("inf"), -float("inf")):
        for row in (0, 1, 7, 8, 15, 16, 40, 63, page - 1):
            d[2].copy_(kept)
            expect = want.clone()
            for b, T in enumerate(totals):
                for h in range(H):
                    taken = [j for j in chosen[b][h] if j >= 0]
                    j, col = taken[row % len(taken)], int(torch.randint(0, D, (), generator=g))
                    d[2][table[b, j].item(), h, row, col] = value
                    if j * page + row < T:
                        expect[b, h * G:(h + 1) * G, 0, col] = float("nan")
                    # a page that is not read
                    other = next((p for p in range(m) if p not in taken), None)
                    if other is not None:
                        d[2][table[b, other].item(), h, row] = value
            got = attend()
            assert torch.equal(torch.isnan(got), torch.isnan(expect)), (value, row)
            assert torch.equal(got.nan_to_num(9.0), expect.nan_to_num(9.0)), (value, row)


@pytest.mark.parametrize("B", [1, 40])
def test_a_weight_too_small_for_a_number(K, B):
    """in the tile, among a block's warps, and in the join of parts"""
    H, G, D, page, m = 1, 2, 64, 64, 16
    g = gen(2)
    table, k, v = make(g, B, H, D, page, m, BF16)
    k.fill_(4.0)
    for b in range(B):
        k[table[b, :5].long()] = -4.0
        v[table[b, 0], 0, 0, 3] = float("inf")
        v[table[b, 4], 0, 63, 50] = float("nan")
    d = [x.cuda() for x in (torch.full((B, G, 1, D), 6.0, dtype=BF16), k, v, *all_bounds(k), table)]
    selected = torch.zeros((B, H, m), dtype=torch.int32, device="cuda")
    out = K.kvc_gqa_decode_sparse(torch.zeros_like(d[0]), *d, lengths(K, [m * page] * B, 1, m * page), selected)
    nan = torch.isnan(out).cpu()
    expect = torch.zeros_like(nan)
    expect[..., 3] = expect[..., 50] = True
    assert torch.equal(nan, expect) and torch.isfinite(out[~nan.cuda()]).all()
