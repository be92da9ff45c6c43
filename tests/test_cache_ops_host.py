"""What the bindings of the quantised cache, the drafted trees and the selected pages refuse of the arguments whose
shapes the library cannot see, and what they do with some that may be left out (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import build
    build.build()
    from persistent_kv_cache_gb300 import kvc
    return kvc


def calls(K):
    """each call that takes a rope argument, with everything else in order"""
    B, H, C, D, N, page = 2, 2, 64, 64, 5, 64
    z, bf, i32 = torch.zeros, torch.bfloat16, torch.int32
    kq, s = z((B, H, C, D), dtype=torch.int8), z((B, H, C))
    k, new = z((B, H, C, D), dtype=bf), z((B, H, N, D), dtype=bf)
    q1, qn = z((B, 2 * H, 1, D), dtype=bf), z((B, 2 * H, N, D), dtype=bf)
    depth, mask = z((B, N), dtype=i32), z((B, N, 1), dtype=i32)
    table, sel = z((B, 1), dtype=i32), z((B, H, 2), dtype=i32)
    bounds, bscale = z((B, H, 2, D), dtype=torch.int8), z((B, H))
    return D, {
        "kvc_quant_append": lambda rope: K.kvc_quant_append(kq, kq, s, s, new, new, None, 0, rope=rope),
        "kvc_gqa_decode_quant": lambda rope: K.kvc_gqa_decode_quant(q1, q1, kq, kq, s, s, None, 0, rope=rope, workspace=None),
        "kvc_gqa_decode_sparse": lambda rope: K.kvc_gqa_decode_sparse(q1, q1, k, k, bounds, bscale, table, None, sel, rope=rope,
                                                                      workspace=None),
        "kvc_tree_append": lambda rope: K.kvc_tree_append(k, k, new, new, depth, None, rope=rope),
        "kvc_gqa_tree": lambda rope: K.kvc_gqa_tree(qn, qn, k, k, mask, depth, None, rope=rope, workspace=None),
    }


@pytest.mark.parametrize("name", ["kvc_quant_append", "kvc_gqa_decode_quant", "kvc_gqa_decode_sparse", "kvc_tree_append", "kvc_gqa_tree"])
def test_rope_tables_of_another_shape(K, name):
    D, made = calls(K)
    call, z = made[name], torch.zeros
    for cos, sin in ((z(9, D // 4), z(9, D // 4)), (z(9, D), z(9, D)), (z(9, D // 2 - 8), z(9, D // 2 - 8)), (z(9, D // 2), z(8, D // 2)),
                     (z(9, 1, D // 2), z(9, 1, D // 2)), (z(9 * D // 2), z(9 * D // 2)), (z(9, D // 2).double(), z(9, D // 2).double()),
                     (z(9, D // 2), z(9, D // 2).half())):
        with pytest.raises(ValueError, match="rope"):
            call((cos, sin))
    # tables as they should be get as far as the check of the device
    with pytest.raises(ValueError, match="CUDA"):
        call((z(9, D // 2), z(9, D // 2)))


def test_tree_mask_fills_the_buffer_that_it_is_given(K, monkeypatch):
    """mask without depth, depth without mask, both, neither: what is given is what is written and returned"""
    parents = torch.full((3, 40), -1, dtype=torch.int32)
    written = []

    class Library:
        def kvc_tree_mask(self, parents, batch, nodes, mask, depth, status, stream):
            written.append((batch, nodes, mask, depth))
            return 0

    monkeypatch.setattr(K, "library", Library)
    monkeypatch.setattr(K, "_addresses", lambda *tensors: [t if t is None else t.data_ptr() for t in tensors])
    monkeypatch.setattr(K, "_stream", lambda stream: 0)
    for has_mask in (False, True):
        for has_depth in (False, True):
            mask, depth = K.tree_buffers(parents)
            got = K.kvc_tree_mask(parents, mask if has_mask else None, depth if has_depth else None)
            assert got[0].shape == (3, 40, 2) and got[1].shape == (3, 40) and all(t.dtype == torch.int32 for t in got)
            assert (got[0] is mask) == has_mask and (got[1] is depth) == has_depth
            assert written.pop() == (3, 40, got[0].data_ptr(), got[1].data_ptr())
    with pytest.raises(ValueError, match="depth"):
        K.kvc_tree_mask(parents, mask, depth[:, :39])
    with pytest.raises(ValueError, match="mask"):
        K.kvc_tree_mask(parents, mask[..., :1], None)


def test_lengths_of_another_device_or_batch(K, monkeypatch):
    """every call that reads lengths refuses those that are not on the current device, before anything is launched"""
    B, H, C, D, N = 2, 2, 64, 64, 5
    z, bf, i32 = torch.zeros, torch.bfloat16, torch.int32
    kq, s, k, new = z((B, H, C, D), dtype=torch.int8), z((B, H, C)), z((B, H, C, D), dtype=bf), z((B, H, N, D), dtype=bf)
    q1, qn = z((B, 2 * H, 1, D), dtype=bf), z((B, 2 * H, N, D), dtype=bf)
    depth, mask, count = z((B, N), dtype=i32), z((B, N, 1), dtype=i32), z(B, dtype=i32)
    table, sel, bounds, bscale = z((B, 1), dtype=i32), z((B, H, 2), dtype=i32), z((B, H, 2, D), dtype=torch.int8), z((B, H))

    class Library:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(f"{name} was called")

    monkeypatch.setattr(K, "library", Library)
    monkeypatch.setattr(K, "_addresses", lambda *tensors: [0] * len(tensors))
    monkeypatch.setattr(K, "_get_device", lambda: 0)
    for L, what in ((K.Lengths(B, "cpu"), "current device, cuda:0, got cpu"), (K.Lengths(B + 1, "cpu"), "made for 3 batch rows")):
        for call in (lambda: K.kvc_quant_append(kq, kq, s, s, new, new, L, 0), lambda: K.kvc_dequant_rows(k, k, kq, kq, s, s, L, 0),
                     lambda: K.kvc_gqa_decode_quant(q1, q1, kq, kq, s, s, L, 0, workspace=None),
                     lambda: K.kvc_page_bounds(bounds, bscale, k, table, L, 1),
                     lambda: K.kvc_gqa_decode_sparse(q1, q1, k, k, bounds, bscale, table, L, sel, workspace=None),
                     lambda: K.kvc_tree_append(k, k, new, new, depth, L), lambda: K.kvc_gqa_tree(qn, qn, k, k, mask, depth, L, workspace=None),
                     lambda: K.kvc_tree_commit(k, k, depth, count, L, count, N)):
            with pytest.raises(ValueError, match=what):
                call()
