"""Trees over caches and pools whose elements do not fit 32-bit offsets, where the output hangs on the keys: a window
that takes in a few rows of zeros before the drafts, compared with a small cache that holds the same rows, and the keys
as they were appended and kept, bit for bit, in every head."""
import pytest
import torch

import _ops_reference as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


@pytest.mark.parametrize("paged", [False, True])
def test_tree(K, paged):
    H, C, D, N, G, page = 3, 1 << 23, 128, 4, 2, 64  # 3.2e9 elements, 6.4 GB each of K and V
    k, v = (torch.zeros((C // page, H, page, D) if paged else (1, H, C, D), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.arange(C // page, dtype=torch.int32, device="cuda").flip(0)[None].contiguous() if paged else None
    g = torch.Generator(device="cuda").manual_seed(4)
    new_k, new_v = (torch.randn((1, H, N, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((1, H * G, N, D), generator=g, device="cuda").to(BF16)
    mask, depth = K.kvc_tree_mask(torch.tensor([[-1, 0, 0, 1]], dtype=torch.int32, device="cuda"))

    def rows(x, at):
        return x[table[0, at // page].item(), :, at % page] if paged else x[0, :, at]

    small = [torch.zeros((1, H, 2 * N, D), dtype=BF16, device="cuda") for _ in range(2)]
    L0 = K.kvc_seq_lengths(torch.tensor([2 * N - 1], dtype=torch.int32, device="cuda"), N, 2 * N, K.KVC_CONTIGUOUS)
    K.kvc_tree_append(*small, new_k, new_v, depth, L0)
    want = K.kvc_gqa_tree(torch.zeros_like(q), q, *small, mask, depth, L0, local_window_size=N).double()
    # the nodes' own rows alone, with equal weights: what it would be if the keys were read as zeros
    plain = K.kvc_gqa_tree(torch.zeros_like(q), q, torch.zeros_like(small[0]), small[1], mask, depth, L0, local_window_size=N)
    assert (want - plain.double()).abs().amax((2, 3)).min() > 0.1  # (in every head)
    for past in (C - N, 5 * C // 8 + 3, 100):  # the last rows, and (paged) the last pages of the pool
        L = K.kvc_seq_lengths(torch.tensor([past + N - 1], dtype=torch.int32, device="cuda"), N, C, K.KVC_CONTIGUOUS)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        K.kvc_tree_append(k, v, new_k, new_v, depth, L, block_table=table, status=st)
        for i in range(N):
            assert torch.equal(rows(k, past + i), new_k[0, :, i]) and torch.equal(rows(v, past + i), new_v[0, :, i])
        out = K.kvc_gqa_tree(torch.zeros_like(q), q, k, v, mask, depth, L, block_table=table, local_window_size=N, status=st)
        # two roundings of sums that differ by their order and, below the rounding, by the parts they are made of
        assert (out.double() - want).abs().max() <= 4 * R.half_step(BF16) * want.abs().max()
        path = torch.tensor([[0, 1, 3]], dtype=torch.int32, device="cuda")
        three, total = torch.tensor([3], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        K.kvc_tree_commit(k, v, path, three, L, total, N, block_table=table, status=st)
        assert total.item() == past + 2 and st.item() == 0
        for at, i in ((past, 0), (past + 1, 1), (past + 2, 3)):
            assert torch.equal(rows(k, at), new_k[0, :, i]) and torch.equal(rows(v, at), new_v[0, :, i])
        for i in range(N):
            rows(k, past + i).zero_()
            rows(v, past + i).zero_()
