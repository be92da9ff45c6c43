"""Plain float64 forms of the cache operators, row by row, for the tests: no
code of the library and none of its order of work.  Tensors are on the CPU."""
import math

import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def half_step(dtype):
    """largest relative rounding error of a value stored in dtype"""
    return torch.finfo(dtype).eps / 2


def rope_tables(max_pos, D, theta=10000.0):
    i = torch.arange(D // 2, dtype=torch.float64)
    at = torch.arange(max_pos, dtype=torch.float64)[:, None] * theta ** (-2.0 * i / D)
    return at.cos().float(), at.sin().float()


def rotate32(x, pos, rope):
    """rows x [..., S, D] at positions [S]: float32, each product and sum rounded (the
    definition of the rotation that is stored)"""
    if rope is None:
        return x.float()
    c, s = rope[0][pos], rope[1][pos]
    lo, hi = x.float().chunk(2, -1)
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def rotate64(x, pos, rope):
    if rope is None:
        return x.double()
    c, s = rope[0][pos].double(), rope[1][pos].double()
    lo, hi = x.double().chunk(2, -1)
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def quantise(x, code_type):
    """float32 rows [..., D] -> (codes, scales), as the header states it"""
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    scale = top / torch.full_like(top, TOP[code_type])
    zero = (scale == 0) | bad
    y = x / torch.where(zero, torch.ones_like(scale), scale)[..., None]
    y = torch.where(zero[..., None], torch.zeros_like(y), y)
    if code_type == torch.int8:
        code = y.round().clamp(-127, 127).to(torch.int8)
    else:
        code = y.clamp(-448, 448).to(code_type)
    return code, torch.where(bad, torch.full_like(scale, math.nan), scale)


def values(code, scale):
    return code.float().double() * scale.double()[..., None]


def softmax_rows(s, visible):
    """s [.., R] float64, visible [.., R] -> weights; zeros where nothing is visible"""
    s = torch.where(visible, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.where(visible, torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m)),
                    torch.zeros_like(s))
    t = p.sum(-1, keepdim=True)
    return p / torch.where(t == 0, torch.ones_like(t), t)


def attention(q, k, v, visible, scale, q_step, w_step, out_type, half_weights=None):
    """q [G, D], k, v [R, D] float64, visible [G, R] -> (out, bound): the attention and how far
    a kernel may be off that rounds the query and the keys by q_step, the weights by w_step and
    the result to out_type.

    A score is off by at most e = |scale| * sum_d |q_d k_d| * (q_step + D 2^-23) (the last: the
    float32 sum); a weight p by a factor within exp(+-2 e_max) (its numerator and the
    denominator); then w_step and the float32 exponential and sum (R + 64) 2^-22; so the result by
    that times sum p |v|, and its own half step.

    half_weights: where weights are held as halves, the factor f [R] that value row r's weight
    has taken up (its scale, or 1): the weight is p_r f_r over a reference that is at most the
    largest p f, and below 2^-14 a half's step is 2^-24 however small it is, so a value v_r / f_r
    is off by another 2^-25 max(p f).  (A column in which the heavy rows hold nothing shows it.)"""
    k, v = torch.where(visible.any(0)[:, None], k, torch.zeros_like(k)), torch.where(
        visible.any(0)[:, None], v, torch.zeros_like(v))
    D = q.shape[-1]
    p = softmax_rows(q @ k.T * scale, visible)
    out = p @ v
    e = abs(scale) * (q.abs() @ k.abs().T) * (q_step + D * 2.0 ** -23)
    e = torch.where(visible, e, torch.zeros_like(e)).amax(-1, keepdim=True) if k.shape[0] else 0.0
    rel = torch.expm1(2 * e) + w_step + (v.shape[0] + 64) * 2.0 ** -22
    bound = rel * (p @ v.abs())
    if half_weights is not None:
        f = half_weights.double()
        held = torch.where((f > 0)[:, None], v.abs() / f.clamp(min=1e-300)[:, None], torch.zeros_like(v))
        bound = bound + 2.0 ** -25 * (p * f).amax(-1, keepdim=True) * (visible.double() @ held)
    tiny = torch.finfo(out_type).smallest_normal * torch.finfo(out_type).eps
    return out, bound + (out.abs() + bound) * half_step(out_type) + tiny


def assert_within(got, want, bound, what=""):
    got = got.detach().double().cpu()
    off = (got - want).abs()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    over = off > bound
    assert not over.any(), (f"{what}: {int(over.sum())} values off, the worst by "
                            f"{float((off / bound).nan_to_num(0).max()):.2f} of the bound")
