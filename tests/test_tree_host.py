"""What the tree calls refuse on the host, before any launch (no GPU needed: the pointers are never
followed), and what the binding refuses."""
import pytest
import torch

F = 1 << 30


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import build
    build.build()
    from persistent_kv_cache_gb300 import kvc
    return kvc


def call(K, fn, args, **change):
    return getattr(K.library(), fn)(*dict(args, **change).values())


def rows(K):
    return dict(table=None, m=0, n=0, page=0, len=K.KvcLengths(F, F, F, F, F))


BOTH = ((dict(dtype=5), 3), (dict(dtype=0), 5), (dict(D=32), 5), (dict(N=257), 5), (dict(N=0), 2), (dict(B=-1), 2), (dict(H=0), 2),
        (dict(C=0), 6), (dict(C=1 << 31), 6), (dict(B=60000, H=100, C=1 << 12), 6), (dict(table=F, page=32, m=4, n=9), 2),
        (dict(table=F, page=64, m=0, n=9), 2), (dict(table=F, page=64, m=4, n=0), 2), (dict(table=F, page=64, m=1 << 26, n=9), 6),
        (dict(table=F, page=64, m=4, n=1 << 30), 6), (dict(k=None), 1), (dict(v=None), 1), (dict(len=None), 1), (dict(k=F + 8), 4),
        (dict(v=F + 64), 2))


def check(K, fn, a, more):
    assert call(K, fn, a, B=0) == 0
    for change, code in BOTH + more:
        change = dict(change)
        if "len" in change:
            change["len"] = K.KvcLengths()
        assert call(K, fn, a, **change) == code, (fn, change)


def test_append(K):
    a = dict(k=F, v=2 * F, nk=3 * F, nv=4 * F, depth=5 * F, **rows(K), B=2, H=2, N=8, C=64, D=64, dtype=1, cos=None, sin=None, rmax=0,
             st=None, stream=None)
    check(K, "kvc_tree_append", a, ((dict(depth=None), 1), (dict(nk=None), 1), (dict(cos=F), 1), (dict(cos=F, sin=F), 2),
                                    (dict(nv=4 * F + 2), 4)))


def test_attention(K):
    need = K.library().kvc_gqa_tree_workspace_size(2, 8, 2, 8, 64)
    assert need > 0 and K.library().kvc_gqa_tree_workspace_size(2, 8, 3, 8, 64) == 0
    a = dict(out=6 * F, q=7 * F, k=F, v=2 * F, mask=5 * F, depth=5 * F, **rows(K), B=2, Hq=8, H=2, N=8, C=64, D=64, dtype=1, window=0,
             scale=0.0, cos=None, sin=None, rmax=0, ws=8 * F, wsb=need, st=None, stream=None)
    check(K, "kvc_gqa_tree", a, ((dict(Hq=7), 2), (dict(Hq=0), 2), (dict(Hq=34), 5), (dict(mask=None), 1), (dict(depth=None), 1),
                                 (dict(out=None), 1), (dict(q=7 * F + 2), 4), (dict(ws=None), 8), (dict(wsb=need - 1), 8),
                                 (dict(ws=8 * F + 16), 4), (dict(sin=F), 1)))


def test_commit(K):
    a = dict(k=F, v=2 * F, path=3 * F, acc=4 * F, plen=4, **rows(K), seqlens=5 * F, B=2, H=2, N=8, C=64, D=64, dtype=1, st=None,
             stream=None)
    check(K, "kvc_tree_commit", a, ((dict(plen=0), 2), (dict(path=None), 1), (dict(acc=None), 1), (dict(seqlens=None), 1)))


def test_mask(K):
    f = K.library().kvc_tree_mask
    assert f(F, 0, 4, F, F, None, None) == 0
    assert f(F, -1, 4, F, F, None, None) == 2 and f(F, 1, 0, F, F, None, None) == 2 and f(F, 1, 257, F, F, None, None) == 5
    assert f(None, 1, 4, F, F, None, None) == 1 and f(F, 1, 4, None, F, None, None) == 1 and f(F, 1, 4, F, None, None, None) == 1


def test_binding_refuses(K):
    k = torch.zeros((2, 2, 64, 64), dtype=torch.bfloat16)
    n = torch.zeros((2, 2, 5, 64), dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 5, 64), dtype=torch.bfloat16)
    d, w = torch.zeros((2, 5), dtype=torch.int32), torch.zeros((2, 5, 1), dtype=torch.int32)
    t = torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="parents"):
        K.kvc_tree_mask(d.long(), w, d)
    for args, name in (((k, k[:1], n, n, d, None), "v_cache"), ((k, k, n.half(), n, d, None), "new_k"), ((k, k, n, n[:, :, :4], d, None), "new_v"),
                       ((k, k, n, n, d[:, :4], None), "depth"), ((k[:1], k[:1], n, n, d, None), "k_cache"),
                       ((k, k, n, n, d, None, t.long()), "block_table")):
        with pytest.raises(ValueError, match=name):
            K.kvc_tree_append(*args)
    for args, name in (((q.half(), q, k, k, w, d, None), "out"), ((q, q.half(), k, k, w, d, None), "q"), ((q, q, k, k, w[..., :0], d, None), "mask")):
        with pytest.raises(ValueError, match=name):
            K.kvc_gqa_tree(*args, workspace=None)
    with pytest.raises(ValueError, match="accepted"):
        K.kvc_tree_commit(k, k, d, d, None, d[:, 0], 5)
