"""What the quantised cache's calls refuse on the host, before any launch (no GPU needed: the
pointers are never followed), and what the binding refuses."""
import pytest
import torch

F = 1 << 24


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import build
    build.build()
    from persistent_kv_cache_gb300 import kvc
    return kvc


def call(K, fn, args, **change):
    a = dict(args, **change)
    return getattr(K.library(), fn)(*a.values())


@pytest.fixture
def L(K):
    return K.KvcLengths(F, F, F, F, F)


def append_args(L):
    return dict(kq=F, vq=2 * F, ks=3 * F, vs=4 * F, nk=5 * F, nv=6 * F, len=L, B=2, H=2, S=3, C=64, D=64, dtype=1,
                fmt=0, windowed=0, cos=None, sin=None, rmax=0, st=None, stream=None)


def test_append(K, L):
    f, a = "kvc_quant_append", append_args(L)
    assert call(K, f, a, B=0) == 0
    for change, code in ((dict(dtype=3), 3), (dict(fmt=2), 3), (dict(fmt=-1), 3), (dict(B=-1), 2), (dict(H=0), 2),
                         (dict(S=0), 2), (dict(windowed=1), 5), (dict(windowed=2), 5), (dict(D=72), 5), (dict(D=272), 5),
                         (dict(C=0), 6), (dict(C=1 << 31), 6), (dict(cos=F), 1), (dict(cos=F, sin=F), 2), (dict(kq=None), 1),
                         (dict(vs=None), 1), (dict(nv=None), 1), (dict(len=K.KvcLengths()), 1), (dict(ks=3 * F + 4), 4),
                         (dict(nk=5 * F + 2), 4), (dict(vq=F + 1024), 2), (dict(ks=F), 2), (dict(vs=3 * F + 16), 2),
                         (dict(cos=F + 4, sin=F, rmax=9), 4)):
        assert call(K, f, a, **change) == code, change


def test_dequant(K, L):
    f = "kvc_dequant_rows"
    a = dict(ko=5 * F, vo=6 * F, kq=F, vq=2 * F, ks=3 * F, vs=4 * F, len=L, B=2, H=2, C=64, R=64, D=64, dtype=1, fmt=0,
             windowed=0, st=None, stream=None)
    assert call(K, f, a, B=0) == 0
    for change, code in ((dict(dtype=9), 3), (dict(fmt=2), 3), (dict(B=70000, H=1), 2), (dict(windowed=2), 5), (dict(D=8), 5),
                         (dict(R=0), 6), (dict(C=0), 6), (dict(ko=None), 1), (dict(ks=None), 1), (dict(vo=6 * F + 8), 4),
                         (dict(vo=5 * F + 16), 2), (dict(ko=F), 2), (dict(vo=4 * F), 2)):
        assert call(K, f, a, **change) == code, change


def test_decode(K, L):
    f = "kvc_gqa_decode_quant"
    need = K.library().kvc_gqa_decode_quant_workspace_size(2, 8, 2, 64 * 9, 64)
    assert need == 2 * (2 * 2 * 5) * 4 * 66 * 4  # a CTA for each of 20 units of 128 keys, two slots each
    assert K.library().kvc_gqa_decode_quant_workspace_size(2, 8, 2, 64, 64) == 0
    assert K.library().kvc_gqa_decode_quant_workspace_size(2, 8, 3, 640, 64) == 0
    a = dict(out=5 * F, q=6 * F, kq=F, vq=2 * F, ks=3 * F, vs=4 * F, len=L, B=2, Hq=8, H=2, C=64 * 9, D=64, dtype=1, fmt=0,
             windowed=0, window=0, scale=0.0, cos=None, sin=None, rmax=0, ws=7 * F, wsb=need, st=None, stream=None)
    assert call(K, f, a, B=0) == 0
    for change, code in ((dict(dtype=0), 5), (dict(dtype=7), 3), (dict(fmt=5), 3), (dict(Hq=7), 2), (dict(Hq=34), 5),
                         (dict(D=96), 5), (dict(windowed=1), 5), (dict(windowed=2), 5), (dict(C=0), 6), (dict(ws=None), 8),
                         (dict(wsb=need - 1), 8), (dict(ws=7 * F + 16), 4), (dict(out=None), 1), (dict(q=6 * F + 2), 4),
                         (dict(sin=F), 1), (dict(vq=None), 1), (dict(vs=3 * F), 2)):
        assert call(K, f, a, **change) == code, change


def test_binding_refuses(K):
    z = torch.zeros
    kq, s = z((1, 1, 4, 16), dtype=torch.int8), z((1, 1, 4))
    n = z((1, 1, 2, 16))
    with pytest.raises(ValueError, match="quantised cache"):
        K.kvc_quant_append(kq.view(torch.uint8), kq, s, s, n, n, None, 0)
    with pytest.raises(ValueError, match="vq"):
        K.kvc_quant_append(kq, kq.view(torch.float8_e4m3fn), s, s, n, n, None, 0)
    with pytest.raises(ValueError, match="k_scale"):
        K.kvc_quant_append(kq, kq, s[..., :3], s, n, n, None, 0)
    with pytest.raises(ValueError, match="new_v"):
        K.kvc_quant_append(kq, kq, s, s, n, n[:, :, :1], None, 0)
    with pytest.raises(ValueError, match="CUDA"):
        K.kvc_quant_append(kq, kq, s, s, n, n, None, 0)
    with pytest.raises(ValueError, match="v_out"):
        K.kvc_dequant_rows(n, n.half(), kq, kq, s, s, None, 0)
    with pytest.raises(ValueError, match="q: "):
        K.kvc_gqa_decode_quant(n, n, kq, kq, s, s, None, 0, workspace=None)
