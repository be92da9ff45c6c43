"""Calls of several host threads whose kernels are one, with different amounts of shared memory: no call lowers what
another is about to launch with."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def window(K, C):
    """a step of a ring of C slots"""
    g = torch.Generator(device="cuda").manual_seed(C)
    B, H, G, D = 2, 2, 4, 64
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)  # noqa: E731
    q, k, v, nk, nv = rand(B, H * G, 1, D), rand(B, H, C, D), rand(B, H, C, D), rand(B, H, 1, D), rand(B, H, 1, D)
    last = torch.tensor([C // 2, 3 * C], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)

    def call():
        K.kvc_window_decode_step(out, q, k, v, nk, nv, last, C, windowed=K.KVC_RING)
        return out
    return call


def select(K, most):
    """the choice among a few pages, in a table with room for `most`"""
    g = torch.Generator(device="cuda").manual_seed(most)
    B, H, G, D, page, pool = 1, 2, 4, 64, 64, 12
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)  # noqa: E731
    q, k, v = rand(B, H * G, 1, D), rand(pool, H, page, D), rand(pool, H, page, D)
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    table[0, :pool] = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    bounds, scale = torch.zeros((pool, H, 2, D), dtype=torch.int8, device="cuda"), torch.zeros((pool, H), device="cuda")
    L = K.Lengths(B, "cuda")
    L.buf.copy_(torch.tensor([[699], [700], [699], [700], [0]]))
    K.kvc_page_bounds(bounds, scale, k, table, L, 1)
    out, taken = torch.empty_like(q), torch.empty((B, H, 5), dtype=torch.int32, device="cuda")
    ws = K.sparse_workspace(q, k, taken)

    def call():
        K.kvc_gqa_decode_sparse(out, q, k, v, bounds, scale, table, L, taken, workspace=ws)
        return out
    return call


@pytest.mark.parametrize("make,sizes", [(window, (512, 64, 448)), (select, (49152, 8600, 30000))])
def test_threads(K, make, sizes):
    calls = [make(K, n) for n in sizes]
    torch.cuda.synchronize()
    want = [call().clone() for call in calls]
    torch.cuda.synchronize()
    failed = []

    def many(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(500):
                    got = calls[i]()
                torch.cuda.current_stream().synchronize()
                assert torch.equal(got, want[i])
        except Exception as e:  # (told by the test's own thread)
            failed.append((sizes[i], e))
    threads = [threading.Thread(target=many, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
