"""The quantised cache: rows quantised as they are written (kvc_quant_append), read back
(kvc_dequant_rows) and attended over (kvc_gqa_decode_quant), against the float64 forms of
_ops_reference.py.  Codes, scales and rows read back are equal bit for bit; the attention is
within the bound that attention() derives: query and weights are halves (2^-11), for fp16 sums of
two, the codes and scales are exact."""
import math

import pytest
import torch

import _ops_reference as R

pytestmark = pytest.mark.gpu

INT8, E4M3 = torch.int8, torch.float8_e4m3fn
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def gen(seed):
    return torch.Generator().manual_seed(seed)


def same(a, b):
    """equal bit for bit, NaN patterns aside"""
    a, b = a.detach().cpu(), b.detach().cpu()
    if a.dtype == E4M3:
        a, b = a.view(torch.uint8), b.view(torch.uint8)
    return torch.equal(torch.nan_to_num(a, nan=12345.0) if a.is_floating_point() else a,
                       torch.nan_to_num(b, nan=12345.0) if b.is_floating_point() else b)


def codes(g, shape, code_type, spread=0.5):
    x = (torch.randn(shape, generator=g) * (R.TOP[code_type] / 3.5)).clamp(-R.TOP[code_type], R.TOP[code_type])
    scale = torch.exp(spread * torch.randn(shape[:-1], generator=g)) * (3.5 / R.TOP[code_type])
    return (x.round().to(INT8) if code_type == INT8 else x.to(E4M3)), scale


def lengths(K, totals, S, C, policy, st=None):
    sk = torch.tensor([t - 1 for t in totals], dtype=torch.int32, device="cuda")
    return K.kvc_seq_lengths(sk, S, C, policy, C, status=st)


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 208, 256])
@pytest.mark.parametrize("code_type,dtype", [(INT8, BF16), (E4M3, F16), (INT8, F32), (E4M3, F32)])
@pytest.mark.parametrize("ring,S,C", [(False, 1, 9), (False, 37, 70), (True, 1, 8), (True, 13, 5)])
def test_append_and_read_back(K, D, code_type, dtype, ring, S, C):
    B, H, g = 4, 3, gen(D * 131 + S)
    policy = K.KVC_RING if ring else K.KVC_CONTIGUOUS
    totals = [S, S + 3, 5 * C + 2, 0] if ring else [S, S + 3, C, 0]  # the last is refused
    rope = R.rope_tables(6 * C + S, D)
    new_k, new_v = (torch.randn((B, H, S, D), generator=g).to(dtype) for _ in range(2))
    new_k[0, 0, 0] = 0                       # a row of zeros
    new_v[0, 1, 0, D - 1] = math.inf         # rows that are not finite
    new_v[1, 1, S - 1, 0] = math.nan
    new_v[1, 2, 0] *= 1e-4 if dtype == F16 else 1e-30
    kq, ks = codes(g, (B, H, C, D), code_type)
    vq, vs = codes(g, (B, H, C, D), code_type)
    d = [x.cuda() for x in (kq, vq, ks, vs, new_k, new_v)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lengths(K, totals, S, C, policy, st)
    K.kvc_quant_append(*d, L, policy, rope=[x.cuda() for x in rope], status=st)
    for b, T in enumerate(totals[:3]):
        pos = torch.arange(max(T - S, T - C if ring else 0), T)
        i = pos - (T - S)
        for q, s, new in ((kq, ks, R.rotate32(new_k[b], torch.arange(T - S, T), rope)), (vq, vs, new_v[b].float())):
            c, x = R.quantise(new[:, i], code_type)
            q.view(torch.uint8)[b][:, pos % C] = c.view(torch.uint8)
            s[b][:, pos % C] = x
    for got, want in zip(d[:4], (kq, vq, ks, vs)):
        assert same(got, want)
    assert st.item() == K.KVC_DEV_SEQLEN_RANGE
    # read back: oldest first, the rows behind them left alone
    rows = C + 2
    for out_type in (BF16, F16, F32):
        out = [torch.full((B, H, rows, D), 7.0, dtype=out_type, device="cuda") for _ in range(2)]
        K.kvc_dequant_rows(*out, *d[:4], L, policy, status=st)
        for got, q, s in ((out[0], kq, ks), (out[1], vq, vs)):
            want = torch.full((B, H, rows, D), 7.0, dtype=out_type)
            for b, T in enumerate(totals[:3]):
                n = min(T, C)
                at = torch.arange(T - n, T) % C
                want[b, :, :n] = (q[b].view(torch.uint8)[:, at].view(code_type).float() * s[b][:, at][..., None]).to(out_type)
            assert same(got, want)


def test_append_refuses_rows_it_must_not_write(K):
    B, H, S, C, D = 3, 2, 2, 16, 64
    rope = [x.cuda() for x in R.rope_tables(10, D)]
    g = gen(5)
    kq, ks = codes(g, (B, H, C, D), INT8)
    d = [x.cuda() for x in (kq, kq.clone(), ks, ks.clone())]
    new = [torch.randn((B, H, S, D), generator=g).cuda() for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lengths(K, [16, 11, 10], S, C, K.KVC_CONTIGUOUS)
    K.kvc_quant_append(*d, *new, L, K.KVC_CONTIGUOUS, rope=rope, status=st)
    assert st.item() == K.KVC_DEV_ROPE_RANGE
    assert torch.equal(d[0][:2].cpu(), kq[:2]) and not torch.equal(d[0][2].cpu(), kq[2])
    # lengths made for a larger cache
    small = [x[:, :, :8].contiguous() for x in (kq.cuda(), kq.cuda(), ks.cuda(), ks.cuda())]
    before = [x.clone() for x in small]
    st.zero_()
    K.kvc_quant_append(*small, *new, L, K.KVC_CONTIGUOUS, status=st)
    assert st.item() == K.KVC_DEV_CAPACITY and all(torch.equal(a, b) for a, b in zip(small, before))
    st.zero_()
    out = [torch.zeros((B, H, C, D), device="cuda") for _ in range(2)]
    K.kvc_dequant_rows(*out, *small, L, K.KVC_CONTIGUOUS, status=st)
    K.kvc_gqa_decode_quant(torch.zeros((B, H, 1, D), dtype=BF16, device="cuda"),
                           torch.zeros((B, H, 1, D), dtype=BF16, device="cuda"), *small, L, K.KVC_CONTIGUOUS, status=st)
    assert st.item() == K.KVC_DEV_CAPACITY and not out[0].any()


def decode_case(K, code_type, dtype, B, H, G, D, C, ring, window, totals, rope=True, scale=0.0, seed=0, edit=None):
    g = gen(seed + D + C)
    kq, ks = codes(g, (B, H, C, D), code_type, 1.0)
    vq, vs = codes(g, (B, H, C, D), code_type, 1.0)
    q = (2 * torch.randn((B, H * G, 1, D), generator=g)).to(dtype)
    if edit:
        edit(q, kq, vq, ks, vs)
    rope = R.rope_tables(max(max(totals), 1), D) if rope else None
    policy = K.KVC_RING if ring else K.KVC_CONTIGUOUS
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lengths(K, totals, 1, C, policy, st)
    out = torch.full_like(q, 7.0, device="cuda")
    d = [x.cuda() for x in (q, kq, vq, ks, vs)]
    K.kvc_gqa_decode_quant(out, *d, L, policy, local_window_size=window, scale=scale,
                           rope=rope and [x.cuda() for x in rope], status=st)
    factor = scale or 1 / math.sqrt(D)
    for b, T in enumerate(totals):
        if T < 1 or (not ring and T > C):
            assert (out[b] == 7).all()
            continue
        n = min(T, C, window if window > 0 else T)
        at = torch.arange(T - n, T) % C
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            qq = R.rotate64(q[b, heads], torch.tensor([T - 1]), rope)[:, 0]
            k, v = (R.values(x[b, h].view(torch.uint8)[at].view(code_type), s[b, h][at]) for x, s in ((kq, ks), (vq, vs)))
            # query and weights as halves, and for fp16 as sums of two
            step = 2.0 ** -22 if dtype == F16 else 2.0 ** -11
            want, bound = R.attention(qq, k, v, torch.ones((G, n), dtype=torch.bool), factor, step, step, dtype,
                                      half_weights=vs[b, h][at])
            R.assert_within(out[b, heads, 0], want, bound, f"row {b} head {h}")
    return out, st.item()


@pytest.mark.parametrize("code_type,dtype", [(INT8, BF16), (E4M3, F16)])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 16), (128, 4), (128, 7), (128, 9), (256, 2), (256, 16)])
@pytest.mark.parametrize("C,ring,window", [(1, False, 0), (64, True, 64), (65, False, 0), (257, False, 100), (300, True, 300),
                                           (1021, True, 1), (1021, False, 0)])
def test_decode(K, code_type, dtype, D, G, C, ring, window):
    totals = [1, C, 0, max(1, C - 1), max(1, C // 3)]
    if ring:
        totals[1], totals[3] = 3 * C + 7, 2 * C
    _, st = decode_case(K, code_type, dtype, 5, 2, G, D, C, ring, window, totals)
    assert st == K.KVC_DEV_SEQLEN_RANGE


@pytest.mark.parametrize("B,H", [(1, 1), (40, 8), (3, 5)])
def test_decode_shares(K, B, H):
    """One row over all CTAs; more rows than CTAs; shares that end inside rows of odd lengths."""
    totals = [4999] if B == 1 else [1 + (37 * b * b) % 700 for b in range(B)]
    _, st = decode_case(K, INT8, BF16, B, H, 4, 128, max(totals), False, 0, totals)
    assert st == 0


def test_decode_without_rope_and_with_a_scale(K):
    decode_case(K, E4M3, BF16, 2, 2, 3, 128, 200, False, 0, [200, 131], rope=False, scale=0.25)
    decode_case(K, INT8, F16, 2, 2, 3, 64, 200, False, 0, [200, 131], rope=False, scale=-0.1)


def test_scales_of_any_size(K):
    """A value row of tiny scale that takes all of the weight, rows of scale 0, queries far from 1."""
    def edit(q, kq, vq, ks, vs):
        vs[:, :, ::3] *= 1e-18
        vs[:, :, 1::7] = 0
        ks[:, :, 5::11] = 0
        q[0] *= 1e-3
        q[1] *= 50
    decode_case(K, INT8, BF16, 2, 2, 4, 128, 500, False, 0, [500, 77], edit=edit)

    def only_tiny(q, kq, vq, ks, vs):
        vs *= 1e-25
    decode_case(K, E4M3, BF16, 2, 2, 4, 64, 300, True, 0, [1000, 77], edit=only_tiny)

    def zero(q, kq, vq, ks, vs):
        vs.zero_()
        q[1].zero_()
    out, _ = decode_case(K, E4M3, BF16, 2, 2, 4, 64, 300, True, 0, [1000, 77], edit=zero)
    assert not out.any()


def test_what_no_row_sees_may_be_anything(K):
    """NaN scales and NaN codes behind the window, behind the last row and in other sequences."""
    def edit(q, kq, vq, ks, vs):
        for x in (ks, vs):
            x[0, :, 150:] = math.nan
            x[0, :, :50] = math.inf
        for x in (kq, vq):
            x.view(torch.uint8)[0, :, 150:] = 0x7f
            x.view(torch.uint8)[0, :, :50] = 0xff
    out, _ = decode_case(K, E4M3, BF16, 2, 2, 4, 128, 300, False, 100, [150, 300], edit=edit)
    assert torch.isfinite(out).all()


def test_a_nan_row_that_is_seen_gives_nan(K):
    def edit(q, kq, vq, ks, vs):
        ks[0, 0, 17] = math.nan
        vs[1, 1, 3] = math.nan
        kq[0, 0, 17] = 0
        vq[1, 1, 3] = 0
    out, _ = decode_case(K, INT8, BF16, 2, 2, 4, 128, 300, False, 0, [300, 64], edit=edit)
    nan = torch.isnan(out[:, :, 0].float()).all(-1).cpu()
    assert nan.tolist() == [[True] * 4 + [False] * 4, [False] * 4 + [True] * 4]


def test_rope_range_of_the_query(K):
    q = torch.ones((2, 4, 1, 64), dtype=BF16, device="cuda")
    kq, ks = codes(gen(1), (2, 2, 40, 64), INT8)
    d = [x.cuda() for x in (kq, kq.clone(), ks, ks.clone())]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lengths(K, [31, 30], 1, 40, K.KVC_CONTIGUOUS)
    out = torch.full_like(q, 7.0)
    K.kvc_gqa_decode_quant(out, q, *d, L, K.KVC_CONTIGUOUS, rope=[x.cuda() for x in R.rope_tables(30, 64)], status=st)
    assert st.item() == K.KVC_DEV_ROPE_RANGE
    assert (out[0] == 7).all() and torch.isfinite(out[1]).all() and not (out[1] == 7).all()


def test_prompt_then_steps_then_chunk(K):
    """As a server runs it: a prompt and 20 tokens written, each token attended over; then a chunk whose
    attention reads the rows back; all captured into a graph and replayed on another stream."""
    B, H, G, D, C, P = 3, 2, 4, 128, 160, 70
    g = gen(9)
    rope = [x.cuda() for x in R.rope_tables(C, D)]
    kq = torch.zeros((B, H, C, D), dtype=INT8, device="cuda")
    vq, ks, vs = torch.zeros_like(kq), torch.zeros((B, H, C), device="cuda"), torch.zeros((B, H, C), device="cuda")
    nk, nv = (torch.randn((B, H, C, D), generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn((B, H * G, C, D), generator=g).to(BF16).cuda()
    rows = [torch.zeros((B, H, C, D), dtype=BF16, device="cuda") for _ in range(2)]
    outs = []

    def step(a, b):
        S = b - a
        L = K.Lengths(B, "cuda")
        sk = torch.full((B,), b - 1, dtype=torch.int32, device="cuda")
        K.kvc_seq_lengths(sk, S, C, K.KVC_CONTIGUOUS, out=L)
        K.kvc_quant_append(kq, vq, ks, vs, nk[:, :, a:b].contiguous(), nv[:, :, a:b].contiguous(), L, K.KVC_CONTIGUOUS, rope=rope)
        out = torch.zeros((B, H * G, S, D), dtype=BF16, device="cuda")
        if S == 1:
            K.kvc_gqa_decode_quant(out, q[:, :, a:b].contiguous(), kq, vq, ks, vs, L, K.KVC_CONTIGUOUS, rope=rope)
        else:
            K.kvc_dequant_rows(*rows, kq, vq, ks, vs, L, K.KVC_CONTIGUOUS)
            K.kvc_gqa_prefill_chunk(out, q[:, :, a:b].contiguous(), *rows, L, rope=rope)
        return out

    cuts = [0, P] + list(range(P + 1, P + 21)) + [C]
    eager = [step(a, b).clone() for a, b in zip(cuts, cuts[1:])]
    kept = [x.clone() for x in (kq, vq, ks, vs)]
    for x in (kq, vq, ks, vs, *rows):
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [step(a, b) for a, b in zip(cuts, cuts[1:])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, (kq, vq, ks, vs)))
    assert all(torch.equal(a, b) for a, b in zip(eager, outs))
    # against float64 over the quantised rows
    b, h = 1, 1
    k, v = (R.values(x[b, h].cpu(), s[b, h].cpu()) for x, s in ((kq, ks), (vq, vs)))
    rope = [x.cpu() for x in rope]
    for a, e, out in zip(cuts, cuts[1:], outs):
        for i in range(a, e):
            qq = R.rotate64(q[b, h * G:(h + 1) * G, i:i + 1].cpu(), torch.tensor([i]), rope)[:, 0]
            # a chunk's attention rounds rows, query and weights to bf16 (2^-8 each)
            step_q, step_w = (2.0 ** -11, 2.0 ** -11) if e - a == 1 else (2 * 2.0 ** -8, 2 * 2.0 ** -8)
            want, bound = R.attention(qq, k[:i + 1], v[:i + 1], torch.ones((G, i + 1), dtype=torch.bool), D ** -0.5,
                                      step_q, step_w, BF16, half_weights=vs[b, h, :i + 1].cpu())
            R.assert_within(out[b, h * G:(h + 1) * G, i - a], want, bound, f"token {i}")


def test_two_streams_with_their_own_workspaces(K):
    B, H, G, D, C = 2, 4, 4, 128, 3000
    kq, ks = codes(gen(3), (B, H, C, D), INT8)
    vq, vs = codes(gen(4), (B, H, C, D), INT8)
    d = [x.cuda() for x in (kq, vq, ks, vs)]
    q = torch.randn((2, B, H * G, 1, D), generator=gen(5)).to(BF16).cuda()
    L = lengths(K, [C, 1234], 1, C, K.KVC_CONTIGUOUS)
    want = [K.kvc_gqa_decode_quant(torch.zeros_like(x), x, *d, L, K.KVC_CONTIGUOUS) for x in q]
    ws = [K.quant_decode_workspace(x, d[0]) for x in q]
    got = [torch.zeros_like(x) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, o, s in zip(q, ws, got, streams):
            K.kvc_gqa_decode_quant(o, x, *d, L, K.KVC_CONTIGUOUS, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def after_a_wait(K, call, spoil):
    """call(stream) behind a wait on a stream of its own, and at once `spoil` bytes written on the current one"""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    call(side)
    junk = [torch.full((spoil // 4,), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk


def test_a_workspace_made_for_another_stream_stays_its_own(K):
    B, H, G, D, C = 2, 4, 4, 128, 3000
    kq, ks = codes(gen(3), (B, H, C, D), INT8)
    vq, vs = codes(gen(4), (B, H, C, D), INT8)
    d = [x.cuda() for x in (kq, vq, ks, vs)]
    q = torch.randn((B, H * G, 1, D), generator=gen(5)).to(BF16).cuda()
    L = lengths(K, [C, 1234], 1, C, K.KVC_CONTIGUOUS)
    want = K.kvc_gqa_decode_quant(torch.zeros_like(q), q, *d, L, K.KVC_CONTIGUOUS)
    got = torch.zeros_like(q)
    size = K.quant_decode_workspace(q, d[0]).numel()
    torch.cuda.synchronize()
    after_a_wait(K, lambda s: K.kvc_gqa_decode_quant(got, q, *d, L, K.KVC_CONTIGUOUS, stream=s), size)
    assert torch.equal(want, got)
    # a tree's masks and the attention's workspace
    N = 9
    parents = torch.tensor([[i // 2 - 1 if i else -1 for i in range(N)]] * B, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((B, H, C, D), generator=gen(6 + i)).to(BF16).cuda() for i in range(2))
    x = torch.randn((B, H * G, N, D), generator=gen(8)).to(BF16).cuda()
    L = lengths(K, [C, 1234], N, C, K.KVC_CONTIGUOUS)
    mask, depth = K.kvc_tree_mask(parents)
    want = K.kvc_gqa_tree(torch.zeros_like(x), x, k, v, mask, depth, L)
    got = torch.zeros_like(x)
    size = K.tree_workspace(x, k).numel()
    torch.cuda.synchronize()
    after_a_wait(K, lambda s: K.kvc_gqa_tree(got, x, k, v, mask, depth, L, stream=s), size)
    assert torch.equal(want, got)
    made = []
    after_a_wait(K, lambda s: made.extend(K.kvc_tree_mask(parents, stream=s)), mask.numel() * 4)
    assert torch.equal(made[0], mask) and torch.equal(made[1], depth)
