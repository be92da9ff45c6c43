"""Caches and pools whose elements and bytes do not fit 32-bit offsets: the last heads and pages give what
a cache of their own gives."""
import pytest
import torch

import _ops_reference as R

pytestmark = pytest.mark.gpu

BF16, INT8 = torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def near(a, b, dtype=BF16):
    """two roundings of sums that differ by their order and, below the rounding, by the parts they are made of"""
    a, b = a.double(), b.double()
    assert (a - b).abs().max() <= 4 * R.half_step(dtype) * b.abs().max() and b.abs().max() > 0


def test_quantised_cache(K):
    H, C, D, S = 5, 1 << 23, 128, 3  # 5.4 GB of codes
    kq, vq = (torch.zeros((1, H, C, D), dtype=INT8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((1, H, C), device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    new_k, new_v = (torch.randn((1, H, S, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    for total in (C, 5 * C // 8 + 1):
        L = K.kvc_seq_lengths(torch.tensor([total - 1], dtype=torch.int32, device="cuda"), S, C, K.KVC_CONTIGUOUS)
        K.kvc_quant_append(kq, vq, ks, vs, new_k, new_v, L, K.KVC_CONTIGUOUS)
        for new, codes, scale in ((new_k, kq, ks), (new_v, vq, vs)):
            back = codes[0, :, total - S:total].float() * scale[0, :, total - S:total, None]
            assert (back - new[0].float()).abs().max() <= 0.51 * new.abs().max() / 127
            assert not codes[0, :, total - S - 1].any()
        # the three rows alone are seen: a window of three
        q = torch.randn((1, 2 * H, 1, D), generator=g, device="cuda").to(BF16)
        L1 = K.kvc_seq_lengths(torch.tensor([total - 1], dtype=torch.int32, device="cuda"), 1, C, K.KVC_CONTIGUOUS)
        out = K.kvc_gqa_decode_quant(torch.zeros_like(q), q, kq, vq, ks, vs, L1, K.KVC_CONTIGUOUS, local_window_size=S)
        small = [x[:, :, total - S:total].contiguous() for x in (kq, vq, ks, vs)]
        L3 = K.kvc_seq_lengths(torch.tensor([S - 1], dtype=torch.int32, device="cuda"), 1, S, K.KVC_CONTIGUOUS)
        near(out, K.kvc_gqa_decode_quant(torch.zeros_like(q), q, *small, L3, K.KVC_CONTIGUOUS))
        for x in (kq, vq, ks, vs):
            x[:, :, total - S:total] = 0
    # all of it, a ring's end in between: every value the same, so that the mean is that value
    kq[0, H - 1].fill_(3)
    vq[0, H - 1].fill_(5)
    ks.fill_(0.01)
    vs.fill_(0.25)
    L = K.kvc_seq_lengths(torch.tensor([C + 12345], dtype=torch.int32, device="cuda"), 1, C, K.KVC_RING, C)
    out = K.kvc_gqa_decode_quant(torch.zeros_like(q), q, kq, vq, ks, vs, L, K.KVC_RING)
    assert (out[0, -2:] == 1.25).all() and not out[0, :-2].any()
    rows = [torch.empty((1, H, 64, D), dtype=BF16, device="cuda") for _ in range(2)]
    small = K.kvc_seq_lengths(torch.tensor([63], dtype=torch.int32, device="cuda"), 1, C, K.KVC_CONTIGUOUS)
    K.kvc_dequant_rows(*rows, kq, vq, ks, vs, small, K.KVC_CONTIGUOUS)
    assert (rows[1][0, H - 1] == 1.25).all() and not rows[1][0, :H - 1].any()


@pytest.mark.parametrize("paged", [False, True])
def test_tree(K, paged):
    H, C, D, N, G, page = 3, 1 << 23, 128, 4, 2, 64  # 3.2e9 elements, 6.4 GB each of K and V
    k, v = (torch.zeros((C // page, H, page, D) if paged else (1, H, C, D), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.arange(C // page, dtype=torch.int32, device="cuda").flip(0)[None].contiguous() if paged else None
    g = torch.Generator(device="cuda").manual_seed(2)
    new_k, new_v = (torch.randn((1, H, N, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((1, H * G, N, D), generator=g, device="cuda").to(BF16)
    mask, depth = K.kvc_tree_mask(torch.tensor([[-1, 0, 0, 1]], dtype=torch.int32, device="cuda"))
    tiny = [torch.zeros((1, H, N, D), dtype=BF16, device="cuda") for _ in range(2)]
    L0 = K.kvc_seq_lengths(torch.tensor([N - 1], dtype=torch.int32, device="cuda"), N, N, K.KVC_CONTIGUOUS)
    K.kvc_tree_append(*tiny, new_k, new_v, depth, L0)
    want = K.kvc_gqa_tree(torch.zeros_like(q), q, *tiny, mask, depth, L0, local_window_size=N)
    for past in (C - N, 100):  # the last rows, and (paged) the last pages of the pool
        L = K.kvc_seq_lengths(torch.tensor([past + N - 1], dtype=torch.int32, device="cuda"), N, C, K.KVC_CONTIGUOUS)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        K.kvc_tree_append(k, v, new_k, new_v, depth, L, block_table=table, status=st)
        # depths are at most 2: a window of 1 at depth 0 is the node alone, so the rows before do not count
        out = K.kvc_gqa_tree(torch.zeros_like(q), q, k, v, mask, depth, L, block_table=table, local_window_size=1, status=st)
        alone = K.kvc_gqa_tree(torch.zeros_like(q), q, *tiny, mask, depth, L0, local_window_size=1)
        assert st.item() == 0
        near(out, alone)
        # node 3 (below 1 and 0) to the front
        path = torch.tensor([[0, 1, 3]], dtype=torch.int32, device="cuda")
        three, total = torch.tensor([3], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        K.kvc_tree_commit(k, v, path, three, L, total, N, block_table=table, status=st)
        assert total.item() == past + 2 and st.item() == 0
        at = past + 2
        row = v[table[0, at // page].item(), :, at % page] if paged else v[0, :, at]
        assert torch.equal(row, new_v[0, :, 3])
    assert want.isfinite().all()


def test_selected_pages(K):
    H, page, D, n = 2, 64, 128, 1 << 18  # 4.3e9 elements, 8.6 GB each of K and V
    k, v = (torch.zeros((n, H, page, D), dtype=BF16, device="cuda") for _ in range(2))
    bounds = torch.zeros((n, H, 2, D), dtype=INT8, device="cuda")
    bscale = torch.zeros((n, H), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    pages = 9
    table = torch.tensor([[n - 1 - 7 * i for i in range(pages)]], dtype=torch.int32, device="cuda")
    some = [torch.randn((pages, H, page, D), generator=g, device="cuda").to(BF16) for _ in range(2)]
    k[table[0].long()], v[table[0].long()] = some
    L = K.kvc_seq_lengths(torch.tensor([pages * page - 1], dtype=torch.int32, device="cuda"), pages * page, pages * page,
                          K.KVC_CONTIGUOUS)
    K.kvc_page_bounds(bounds, bscale, k, table, L, pages * page)
    own = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    sb, ss = torch.zeros((pages, H, 2, D), dtype=INT8, device="cuda"), torch.zeros((pages, H), device="cuda")
    K.kvc_page_bounds(sb, ss, some[0], own, L, pages * page)
    assert torch.equal(bounds[table[0].long()], sb) and torch.equal(bscale[table[0].long()], ss)
    q = torch.randn((1, 4 * H, 1, D), generator=g, device="cuda").to(BF16)
    L1 = K.kvc_seq_lengths(torch.tensor([pages * page - 1], dtype=torch.int32, device="cuda"), 1, pages * page, K.KVC_CONTIGUOUS)
    sel = [torch.zeros((1, H, 5), dtype=torch.int32, device="cuda") for _ in range(2)]
    a = K.kvc_gqa_decode_sparse(torch.zeros_like(q), q, k, v, bounds, bscale, table, L1, sel[0])
    b = K.kvc_gqa_decode_sparse(torch.zeros_like(q), q, *some, sb, ss, own, L1, sel[1])
    assert torch.equal(sel[0], sel[1]) and torch.equal(a, b)
