"""kvc_gqa_decode_sparse with a scale of its own, of either sign: the pages taken are those of the header's score (of
-q for a negative scale, whose weights grow with -q . k), bit for bit, and the attention over them is within the
bound of the 64-bit form."""
import pytest
import torch

import _ops_reference as R
from test_gpu_sparse import BF16, F16, all_bounds, choose, gen, lengths, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


@pytest.mark.parametrize("scale", [0.3, -0.3, -0.02, 0.0])
@pytest.mark.parametrize("dtype,D,G,page,rope", [(BF16, 64, 4, 64, True), (F16, 128, 9, 64, False), (BF16, 256, 1, 128, True), (F16, 64, 8, 64, True)])
def test_pages_and_output(K, dtype, D, G, page, rope, scale):
    B, H, m, n, sink, recent = 3, 2, 60, 7, 1, 2
    totals = [m * page, 31 * page + 5, 4 * page]
    g = gen(D + G)
    table, k, v = make(g, B, H, D, page, m, dtype)
    q = torch.randn((B, H * G, 1, D), generator=g).to(dtype)
    bounds, bscale = all_bounds(k)
    tables = R.rope_tables(m * page, D) if rope else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    selected = torch.full((B, H, n), -7, dtype=torch.int32, device="cuda")
    d = [x.cuda() for x in (q, k, v, bounds, bscale, table)]
    out = K.kvc_gqa_decode_sparse(torch.full_like(d[0], 7.0), *d, lengths(K, totals, 1, m * page), selected, sink, recent, scale=scale,
                                  rope=tables and [x.cuda() for x in tables], status=st)
    assert st.item() == 0
    step = R.half_step(dtype)  # (query and weights are sums of two numbers of the type)
    for b, T in enumerate(totals):
        pages = -(-T // page)
        for h in range(H):
            heads, at = slice(h * G, (h + 1) * G), torch.tensor([T - 1])
            q32 = R.rotate32(q[b, heads], at, tables)[:, 0]
            phys = table[b, :pages].long()
            mine = choose(-q32 if scale < 0 else q32, bounds[phys, h], bscale[phys, h], pages, n, sink, recent)
            assert selected[b, h].tolist() == mine + [-1] * (n - len(mine)), f"row {b} head {h}"
            rows = torch.cat([torch.arange(j * page, min(T, (j + 1) * page)) for j in mine])
            kk, vv = (x[table[b, rows // page].long(), h, rows % page].double() for x in (k, v))
            want, bound = R.attention(R.rotate64(q[b, heads], at, tables)[:, 0], kk, vv, torch.ones((G, len(rows)), dtype=torch.bool),
                                      scale or D ** -0.5, step ** 2 if rope else 0.0, step ** 2, dtype,
                                      half_weights=torch.ones(len(rows)) if dtype == F16 else None)
            R.assert_within(out[b, heads, 0], want, bound, f"row {b} head {h}")


def test_the_page_that_holds_the_weight_is_taken(K):
    """one page along the query, one against it: each is taken under its sign of the scale"""
    D, G, page, m = 64, 2, 64, 40
    g = gen(1)
    table, k, v = make(g, 1, 1, D, page, m, BF16)
    q = torch.randn((1, 1, 1, D), generator=g).to(BF16).expand(1, G, 1, D).contiguous()
    k[table[0, 11], 0], k[table[0, 23], 0] = 3 * q[0, 0, 0], -3 * q[0, 0, 0]
    bounds, bscale = all_bounds(k)
    d = [x.cuda() for x in (q, k, v, bounds, bscale, table)]
    for scale, page_in, page_out in ((0.2, 11, 23), (-0.2, 23, 11)):
        selected = torch.zeros((1, 1, 4), dtype=torch.int32, device="cuda")
        K.kvc_gqa_decode_sparse(torch.zeros_like(d[0]), *d, lengths(K, [m * page], 1, m * page), selected, 0, 1, scale=scale)
        got = selected[0, 0].tolist()
        assert page_in in got and page_out not in got, scale
