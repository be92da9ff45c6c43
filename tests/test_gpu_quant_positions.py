"""kvc_gqa_decode_quant over a contiguous cache whose rows are not the positions: row r of L holds
position T - L + r, as in kvc_gqa_decode, for any T >= L and for T past the capacity (lengths of a
windowed, drifting or ring policy)."""
import math

import pytest
import torch

import _ops_reference as R

pytestmark = pytest.mark.gpu

INT8, E4M3 = torch.int8, torch.float8_e4m3fn
BF16, F16 = torch.bfloat16, torch.float16
B, H, C = 4, 2, 300


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def cache(seed, code_type, D):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = (torch.randn((B, H, C, D), generator=g) * (R.TOP[code_type] / 3.5)).clamp(-R.TOP[code_type], R.TOP[code_type])
        out.append((x.round().to(INT8) if code_type == INT8 else x.to(E4M3),
                    torch.exp(0.5 * torch.randn((B, H, C), generator=g)) * (3.5 / R.TOP[code_type])))
    return g, out


def held(K, totals, rows):
    """lengths of a one-token step: T tokens, L rows"""
    L = K.Lengths(len(totals), "cuda")
    for i, row in enumerate(zip(*[(t - 1, t, n - 1, n, 0) for t, n in zip(totals, rows)])):
        L.buf[i] = torch.tensor(row, dtype=torch.int32, device="cuda")
    return L


@pytest.mark.parametrize("code_type,dtype,D,G", [(INT8, BF16, 64, 4), (E4M3, F16, 128, 7), (INT8, F16, 256, 2), (E4M3, BF16, 128, 16)])
@pytest.mark.parametrize("window", [0, 1, 70, 1000])
def test_rows_are_counted_from_the_rows_held(K, code_type, dtype, D, G, window):
    g, ((kq, ks), (vq, vs)) = cache(D + G, code_type, D)
    q = (2 * torch.randn((B, H * G, 1, D), generator=g)).to(dtype)
    totals, rows = [299, 2 * C + 5, C + 1, 20000], [131, C, 1, 257]  # L < T <= C; T past C, with and without a full cache
    d = [x.cuda() for x in (q, kq, vq, ks, vs)]

    def run(L, rope=None):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = K.kvc_gqa_decode_quant(torch.full_like(d[0], 7.0), *d, L, K.KVC_CONTIGUOUS, local_window_size=window, status=st,
                                     rope=rope and [x.cuda() for x in rope])
        assert st.item() == 0
        return out

    # unrotated, the same rows give the same bits whatever T is
    assert torch.equal(run(held(K, totals, rows)), run(held(K, rows, rows)))
    rope = R.rope_tables(max(totals), D)
    out = run(held(K, totals, rows), rope)
    for b, (T, L) in enumerate(zip(totals, rows)):
        n = min(L, window or L)
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            qq = R.rotate64(q[b, heads], torch.tensor([T - 1]), rope)[:, 0]
            k, v = (R.values(x[b, h, L - n:L], s[b, h, L - n:L]) for x, s in ((kq, ks), (vq, vs)))
            # query and weights as halves, and for fp16 as sums of two
            step = 2.0 ** -22 if dtype == F16 else 2.0 ** -11
            want, bound = R.attention(qq, k, v, torch.ones((G, n), dtype=torch.bool), 1 / math.sqrt(D), step, step, dtype,
                                      half_weights=vs[b, h, L - n:L])
            R.assert_within(out[b, heads, 0], want, bound, f"row {b} head {h}")


@pytest.mark.parametrize("policy", ["KVC_WINDOWED", "KVC_DRIFTING", "KVC_RING"])
def test_lengths_of_other_policies(K, policy):
    """what kvc_seq_lengths gives for them, far past the capacity"""
    D, G = 128, 4
    g, ((kq, ks), (vq, vs)) = cache(7, INT8, D)
    q = torch.randn((B, H * G, 1, D), generator=g).to(BF16).cuda()
    d = [x.cuda() for x in (kq, vq, ks, vs)]
    sk = torch.tensor([10 * C, C, 5 * C + 17, 40], dtype=torch.int32, device="cuda")
    L = K.kvc_seq_lengths(sk, 1, C, getattr(K, policy), 200 if policy == "KVC_DRIFTING" else C)
    rows = L.cache_total.tolist()
    assert max(rows) <= C < L.total_abs.max().item()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = K.kvc_gqa_decode_quant(torch.zeros_like(q), q, *d, L, K.KVC_CONTIGUOUS, status=st)
    assert st.item() == 0
    assert torch.equal(got, K.kvc_gqa_decode_quant(torch.zeros_like(q), q, *d, held(K, rows, rows), K.KVC_CONTIGUOUS))
    # and the 16-bit decode over the same rows read back: it rounds rows, query and weights to bf16
    back = [torch.zeros((B, H, C, D), dtype=BF16, device="cuda") for _ in range(2)]
    K.kvc_dequant_rows(*back, *d, L, K.KVC_CONTIGUOUS)
    other = K.kvc_gqa_decode(torch.zeros_like(q), q, *back, L).cpu()
    for b, n in enumerate(rows):
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            k, v = (R.values(x[b, h, :n], s[b, h, :n]) for x, s in ((kq, ks), (vq, vs)))
            want, bound = R.attention(q[b, heads, 0].double().cpu(), k, v, torch.ones((G, n), dtype=torch.bool), D ** -0.5,
                                      2 * 2.0 ** -8, 2 * 2.0 ** -8, BF16)
            R.assert_within(other[b, heads, 0], want, bound, f"row {b} head {h}")
