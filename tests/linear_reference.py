"""Linear attention with a decay for each head, and the norms and rotation before
it, in 64 bits (torch on the CPU), written from their formulas, with the bounds
the GPU tests hold the kernels to.

As in layer_reference: float64 in and out, gradients written out
(test_linear_reference checks them against automatic differentiation and against
differences), ``EPS`` = 2^-24 half a step of FP32 relative to the value.
"""
from __future__ import annotations

import torch

EPS = 2.0 ** -24


# ------------------------------------------------------------- norms and rotation


def _pairs(x, R, interleaved):
    r = x[..., :R]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :R // 2], r[..., R // 2:])


def _joined(a, b, x, R, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, x[..., R:]], -1)


def turn(x, positions, inv_freq, interleaved, back=False):
    """The first 2 len(inv_freq) channels of x [T, H, D], by the positions."""
    if inv_freq is None:
        return x
    R = 2 * len(inv_freq)
    angle = positions.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(angle), torch.sin(-angle if back else angle)
    a, b = _pairs(x, R, interleaved)
    return _joined(a * c - b * s, a * s + b * c, x, R, interleaved)


def _both(x, inv_freq, interleaved):
    """|a| + |b| at both channels of every pair, |x| behind them."""
    x = x.abs()
    if inv_freq is None:
        return x
    R = 2 * len(inv_freq)
    a, b = _pairs(x, R, interleaved)
    return _joined(a + b, a + b, x, R, interleaved)


def _normed(x, eps):
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r, r


def norm_rotate(x, weight, scale, eps, positions, inv_freq, interleaved):
    n = scale * _normed(x, eps)[0]
    return turn(n if weight is None else n * weight, positions, inv_freq, interleaved)


def norm_rotate_bound(x, weight, scale, eps, positions, inv_freq, interleaved):
    """The mean of D <= 256 squares: three roundings a term, at most 20 additions
    and eps: 24 EPS, half of that in its reciprocal root, 4 more for the root,
    3 for the factors: 20 EPS of n.  Cosine and sine are within 9 EPS: 2 units
    (4 EPS) of their function, pi EPS for the turn rounded to FP32, one for its
    FP64 (2^23 radians at 2^-52).  The two products and their sum: 3 more."""
    n = scale * _normed(x, eps)[0]
    return 32 * EPS * _both(n if weight is None else n * weight, inv_freq, interleaved)


def norm_rotate_backward(d, x, weight, scale, eps, positions, inv_freq, interleaved):
    """(dx, dweight) for the cotangent d."""
    m = scale * turn(d, positions, inv_freq, interleaved, back=True)
    xn, r = _normed(x, eps)
    wm = m if weight is None else m * weight
    return r * (wm - xn * (wm * xn).mean(-1, keepdim=True)), None if weight is None else (m * xn).sum((0, 1))


def norm_rotate_backward_bounds(d, x, weight, scale, eps, positions, inv_freq, interleaved, heads):
    """m is within 16 EPS of A = scale (|da| + |db|) as in the forward; x r within
    20 EPS of itself; the mean of their products (24 EPS) within 64 EPS of
    mean(A w |x r|); r and the last operations add 24: 40 EPS of A w and 110 of
    |x r| mean(A w |x r|), times r.  The weight's gradient: 38 EPS a term, and
    one for each addition on the way: a lane group's rows one after another (16
    groups at least, 768 workgroups at most, `heads` rows a token), then the
    groups, waves and workgroups."""
    T = x.shape[0]
    A = abs(scale) * _both(d, inv_freq, interleaved)
    xn, r = _normed(x, eps)
    Aw = A if weight is None else A * weight.abs()
    dx = r * (40 * EPS * Aw + 110 * EPS * xn.abs() * (Aw * xn.abs()).mean(-1, keepdim=True))
    tokens = 4 if T >= 4096 else 2 if T >= 2048 else 1
    tiles = -(-T // tokens)
    blocks = min(tiles, 768)
    adds = -(-tokens * heads // 16) * -(-tiles // blocks) + 6 + -(-blocks // 16) + 16
    return dx, (38 + adds) * EPS * (A * xn.abs()).sum((0, 1))


# ------------------------------------------------------------- single tokens


def of_heads(x, H):
    """[.., heads, W] as H heads: neighbours share one."""
    return x.repeat_interleave(H // x.shape[-2], -2)


def step(q, k, v, g, state):
    """o [.., V], the new state and the magnitude of its terms, for q, k [.., K], v
    [.., V], g [..] and state [.., K, V]."""
    e = torch.exp(g)[..., None, None]
    new = e * state + k[..., None] * v[..., None, :]
    size = (e * state).abs() + (k[..., None] * v[..., None, :]).abs()
    return (new * q[..., None]).sum(-2), new, size


def step_bounds(q, size):
    """The state: 4 EPS of the exponential, two products and a sum: 8 EPS of its
    terms.  o: those, a product, and at most 16 + 8 additions."""
    return 34 * EPS * (size * q.abs()[..., None]).sum(-2), 8 * EPS * size
