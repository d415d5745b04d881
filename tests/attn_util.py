"""Attention in 64 bits with a bound on a correct kernel's error, element by
element, shared by the tests of the tile engine's operators.

For one query row with exact weights w_j (sum 1) and exact output o, a kernel
that rounds its weights to the input type for the product with V (unit roundoff
u = 2^-8 for bf16, 2^-11 for fp16), sums them before or after that rounding,
accumulates in fp32 and rounds the output once, has
    out = sum_j w_j (1 + x_j) (1 + d_j) v_j / sum_j w_j (1 + x_j) (1 + s_j d_j)
with |d_j| <= u and s_j = 1 where the sum takes the rounded weight, else 0
(parts of both kinds may be joined), so to first order
    out - o = sum_j w_j x_j (v_j - o) + sum_j w_j d_j (v_j - s_j o),
and it is off by at most
    x sum_j w_j |v_j - o|           what moves a weight before it is rounded
  + u sum_j w_j max(|v_j|, |v_j - o|)   the weights' rounding
  + u |o|                           the output's rounding
  + n 2^-23 sum_j w_j |v_j|         fp32 sums over n keys (both of them)
  + 2^-25 sum_j max(|v_j|, |v_j - o|)   fp16 only: weights below 2^-14 have an
                                    absolute error of at most 2^-25, next to a
                                    sum of at least 1 (the key whose score is
                                    the reference has the weight 1)
x collects what moves a weight before it is rounded: its score is an fp32 dot
product of `d` terms (d 2^-24 of the sum of their magnitudes) times the scale,
a few more fp32 roundings of the score itself, and the exponential (2^-21):
a score off by e changes a weight by a factor within exp(+-2 e) (the weight
and the sum).  1 % on top covers the products of these.
"""
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def attend(q, k, v, scale, visible=None):
    """One KV head's queries q [n, d] (any order of tokens and heads) over keys
    k, v [m, d]; visible [n, m] bool or None.  Inputs in the tested type;
    returns (out, bound), float64 [n, d].  Rows that see nothing are 0."""
    u = U[q.dtype]
    fp16 = q.dtype == torch.float16
    q, k, v = q.double(), k.double(), v.double()
    n_keys, d = k.shape
    s = q @ k.T * scale
    mag = q.abs() @ k.abs().T * abs(scale)      # what the dot product adds up
    if visible is not None:
        s = s.masked_fill(~visible, float("-inf"))
        mag = mag.masked_fill(~visible, 0.0)
    top = s.amax(-1, keepdim=True)
    some = torch.isfinite(top)
    e = torch.where(some, torch.exp(s - torch.where(some, top, 0.0)), 0.0)
    w = e / e.sum(-1, keepdim=True).clamp_min(1e-300)
    o = w @ v
    x = torch.expm1(2 * ((d + 8) * 2.0 ** -24 * mag.amax(-1, keepdim=True) + 2.0 ** -21))
    # the sums over keys per output element, a slice of rows at a time
    spread = torch.empty_like(o)
    most = torch.empty_like(o)
    flat = torch.zeros_like(o)
    step = max(1, (1 << 24) // max(1, n_keys * d))
    for i in range(0, o.shape[0], step):
        dist = (v[None] - o[i:i + step, None]).abs()
        spread[i:i + step] = torch.einsum("nm,nmd->nd", w[i:i + step], dist)
        dist = torch.maximum(dist, v.abs()[None])
        most[i:i + step] = torch.einsum("nm,nmd->nd", w[i:i + step], dist)
        if fp16:
            seen = (w[i:i + step] > 0) if visible is None else visible[i:i + step]
            flat[i:i + step] = torch.einsum("nm,nmd->nd", seen.double(), dist)
    bound = (x * spread + u * most + u * o.abs() + n_keys * 2.0 ** -23 * (w @ v.abs())
             + 2.0 ** -25 * flat)
    if fp16:  # outputs below 2^-14 round to multiples of 2^-24
        bound = bound + 2.0 ** -25
    return o, 1.01 * bound + 1e-30


def check(got, want, bound, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - want).abs() - bound
    if over.numel() and float(over.max()) > 0:
        i = int(over.flatten().argmax())
        at = [int(x) for x in torch.unravel_index(torch.tensor(i), over.shape)]
        raise AssertionError(f"{what}: {got.flatten()[i]:.6g} at {at}, want "
                             f"{want.flatten()[i]:.6g} within {bound.flatten()[i]:.3g}")
