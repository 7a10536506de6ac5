"""Latent attention in 64 bits, written out from the definitions, and the error bounds of the 16-bit kernels.

Bounds, element by element.  With u = eps / 2 of the 16-bit type (a rounding
to it is off by at most u relative):
  out   one rounding of the result, u |out|, and one of every softmax weight,
        u sum_j p_j |v_j|;
  S     float32 sums of n products: n 2^-23 sum |q_i k_i| scale (2^-23 and not
        2^-24: the tensor core may truncate).  An error e of a score changes
        its weight by a factor exp(e), of all scores a weight by at most 2 e,
        as do the exponential's 2^-22 and the sum's m 2^-24 for m keys.
"""
import math

import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attend(q, k, v, scale, sees):
    """q [n, d], k [m, d], v [m, e] float64; row i sees keys 0 .. sees[i] - 1.
    Returns out, lse, sum p |v| and the largest error of a row's scores."""
    n, m = q.shape[0], k.shape[0]
    hidden = torch.arange(m, device=q.device) >= sees[:, None]
    s = (q @ k.T * scale).masked_fill(hidden, -math.inf)
    size = (q.abs() @ k.abs().T * scale).masked_fill(hidden, 0.0)
    top = s.amax(1, keepdim=True) if m else torch.full((n, 1), -math.inf, dtype=q.dtype, device=q.device)
    p = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    p = p / total.masked_fill(total == 0, 1.0)
    worst = size.amax(1) if m else torch.zeros(n, dtype=q.dtype, device=q.device)
    return p @ v, lse, p @ v.abs(), q.shape[1] * 2.0 ** -23 * worst


def check(out, lse, ref, ref_lse, spread, e_score, dtype, keys, what=""):
    """Holds out and lse to the bounds above (e_score [rows], the others [rows, ...])."""
    u = half_step(dtype)
    e = (2 * e_score + 2.0 ** -21 + keys * 2.0 ** -24)[:, None]
    tol = u * ref.abs() + (u + e) * spread * (1 + u) + 1e-30
    if dtype == torch.float16:                  # results below the least normal number: half its step
        tol = tol + 2.0 ** -25
    err = (out.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).nan_to_num(1e9).max()):.2f} x its bound"
    empty = ref_lse == -math.inf
    assert torch.equal(empty, lse == -math.inf), f"{what}: lse of rows that see nothing"
    tol = e_score + keys * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * ref_lse.abs()
    assert bool(((lse.double() - ref_lse).abs() <= tol)[~empty].all()), f"{what}: lse"
    assert bool((out[empty] == 0).all()), f"{what}: rows that see nothing are not zero"


def rotate(x, cos, sin, interleaved):
    """R_p x for x [..., 64], cos and sin [..., 32], float64."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y = torch.empty_like(x)
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0::2], y[..., 1::2] = ra, rb
    else:
        y[..., :32], y[..., 32:] = ra, rb
    return y
