"""What the page-selection calls refuse on the host, before any launch (no GPU needed: the pointers
are never followed), and what the binding refuses."""
import pytest
import torch

F = 1 << 26


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import build
    build.build()
    from persistent_kv_cache_gb300 import kvc
    return kvc


def call(K, fn, args, **change):
    return getattr(K.library(), fn)(*dict(args, **change).values())


def test_bounds(K):
    f, L = "kvc_page_bounds", K.KvcLengths(F, F, F, F, F)
    a = dict(bounds=F, scale=2 * F, k=3 * F, table=4 * F, m=8, n=32, page=64, len=L, B=2, H=2, S=5, D=64, dtype=1, st=None,
             stream=None)
    assert call(K, f, a, B=0) == 0
    for change, code in ((dict(dtype=4), 3), (dict(dtype=0), 5), (dict(D=32), 5), (dict(B=-1), 2), (dict(S=0), 2), (dict(m=0), 2),
                         (dict(n=0), 2), (dict(page=0), 2), (dict(m=1 << 26, page=64), 6), (dict(bounds=None), 1),
                         (dict(table=None), 1), (dict(len=K.KvcLengths()), 1), (dict(k=3 * F + 2), 4), (dict(scale=F), 2),
                         (dict(bounds=3 * F), 2)):
        assert call(K, f, a, **change) == code, change


def test_decode(K):
    f, L, lib = "kvc_gqa_decode_sparse", K.KvcLengths(F, F, F, F, F), K.library()
    need = lib.kvc_gqa_decode_sparse_workspace_size(2, 8, 2, 64, 4, 64, 1)
    # page ids and counts in 256-byte units; a CTA for each of four rows' four units, two slots each
    assert need == 256 + 256 + 2 * (4 * 4) * 4 * (64 + 2) * 4
    assert lib.kvc_gqa_decode_sparse_workspace_size(2, 8, 2, 64, 4, 96, 1) == 0
    assert lib.kvc_gqa_decode_sparse_workspace_size(2, 8, 3, 64, 4, 64, 1) == 0
    assert lib.kvc_gqa_decode_sparse_workspace_size(2, 8, 2, 63, 4, 64, 1) == 0
    a = dict(out=F, q=2 * F, k=3 * F, v=4 * F, bounds=5 * F, scale=6 * F, table=7 * F, m=8, n=32, page=64, len=L, B=2, Hq=8, H=2,
             D=64, dtype=1, n_select=4, sink=1, recent=1, selected=8 * F, scale_=0.0, cos=None, sin=None, rmax=0, ws=9 * F,
             wsb=need, st=None, stream=None)
    assert call(K, f, a, B=0) == 0
    for change, code in ((dict(dtype=4), 3), (dict(dtype=0), 5), (dict(D=96), 5), (dict(Hq=7), 2), (dict(Hq=34), 5),
                         (dict(page=32), 2), (dict(page=96), 2), (dict(n_select=0), 2), (dict(sink=-1), 2), (dict(recent=0), 2),
                         (dict(sink=4), 2), (dict(recent=2 ** 31 - 1), 2), (dict(m=0), 2), (dict(m=49153), 6),
                         (dict(B=40000), 2), (dict(n=1 << 30), 6), (dict(selected=None), 1), (dict(bounds=None), 1),
                         (dict(ws=None), 8), (dict(wsb=need - 1), 8), (dict(ws=9 * F + 16), 4), (dict(q=2 * F + 8), 4),
                         (dict(cos=F), 1), (dict(cos=F, sin=F), 2), (dict(len=K.KvcLengths()), 1)):
        assert call(K, f, a, **change) == code, change


def test_binding_refuses(K):
    k, q = torch.zeros((4, 2, 64, 64), dtype=torch.bfloat16), torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    b, s = torch.zeros((4, 2, 2, 64), dtype=torch.int8), torch.zeros((4, 2))
    t, sel = torch.zeros((1, 4), dtype=torch.int32), torch.zeros((1, 2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="bounds"):
        K.kvc_page_bounds(b[:3], s, k, t, None, 1)
    with pytest.raises(ValueError, match="block_table"):
        K.kvc_page_bounds(b, s, k, t.long(), None, 1)
    for change, name in ((dict(q=q.half()), "q"), (dict(v=k[:3]), "v_pool"), (dict(sel=sel.long()), "selected"),
                         (dict(t=t.expand(2, 4)), "block_table"), (dict(s=s.half()), "bound_scale")):
        a = dict(q=q, k=k, v=k, b=b, s=s, t=t, L=None, sel=sel)
        a.update(change)
        with pytest.raises(ValueError, match=name):
            K.kvc_gqa_decode_sparse(q, *a.values(), workspace=None)
