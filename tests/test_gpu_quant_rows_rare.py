"""kvc_quant_append of rows whose largest value lies below 2^-100 or above 2^100, down to subnormals and up to the
largest float32: codes and scales are those of the header's divisions, bit for bit.  (A scale may be subnormal, whose
quotient then rounds past the largest code, or zero, which is a row of zeros.)"""
import pytest
import torch

import _ops_reference as R
from test_gpu_quant_cache import BF16, E4M3, F32, INT8, gen, lengths, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def rows(g, n, D, dtype):
    """[n, D], each row's largest value 2^e times something in [1, 2), e spread over the whole range and dense at the
    borders"""
    edges = [-149, -148, -145, -143, -142, -141, -140, -135, -133, -130, -127, -126, -125, -119, -118, -117, -102, -101, -100, -99, 98, 99,
             100, 101, 118, 120, 125, 126, 127]
    e = torch.cat([torch.tensor(edges * 3), torch.randint(-149, 128, (n - 3 * len(edges),), generator=g)]).double()
    x = torch.rand((n, D), generator=g, dtype=torch.float64) * 2 - 1
    top = 1 + torch.rand(n, generator=g, dtype=torch.float64) * (1 - 2.0 ** -7)
    x[:, D // 3] = torch.where(torch.rand(n, generator=g) < 0.5, 1.0, -1.0).double()
    x = x * (top * 2.0 ** e)[:, None]
    most = torch.finfo(dtype).max
    x[len(edges)] = x[len(edges)].sign() * most  # every value the largest there is
    return x.clamp(-most, most).to(dtype)


@pytest.mark.parametrize("code_type", [INT8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
def test_largest_and_smallest_rows(K, code_type, dtype, D):
    B, H, S = 1, 2, 400
    g = gen(D)
    new = [torch.stack([rows(g, S, D, dtype) for _ in range(H)])[None] for _ in range(2)]
    kq, vq = (torch.zeros((B, H, S, D), dtype=torch.int8).view(code_type).cuda() for _ in range(2))
    ks, vs = (torch.zeros((B, H, S), device="cuda") for _ in range(2))
    L = lengths(K, [S], S, S, K.KVC_CONTIGUOUS)
    K.kvc_quant_append(kq, vq, ks, vs, *[x.cuda() for x in new], L, K.KVC_CONTIGUOUS)
    for codes, scale, x in ((kq, ks, new[0]), (vq, vs, new[1])):
        want, s = R.quantise(x.float(), code_type)
        assert (s > 0).any() and (s == 0).any() and s.max() > 2.0 ** 117
        assert same(scale, s)
        assert same(codes, want)
    # and read back
    for out_type in (BF16, F32):
        out = [torch.zeros((B, H, S, D), dtype=out_type, device="cuda") for _ in range(2)]
        K.kvc_dequant_rows(*out, kq, vq, ks, vs, L, K.KVC_CONTIGUOUS)
        for got, codes, scale in ((out[0], kq, ks), (out[1], vq, vs)):
            assert same(got, (codes.float().cpu() * scale.cpu()[..., None]).to(out_type))
