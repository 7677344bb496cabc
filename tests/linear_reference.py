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


# ------------------------------------------------------------- packed sequences


def forward(q, k, v, g, cu, h0=None):
    """o [T, H, V], final states and the same of all terms' magnitudes, token after
    token; q, k, v with their own heads, g [T, H]."""
    T, H = g.shape
    q, k, v = (of_heads(x, H) for x in (q, k, v))
    o = torch.zeros(T, H, v.shape[-1], dtype=torch.float64)
    size, final, fsize = torch.zeros_like(o), [], []
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        S = torch.zeros(H, q.shape[-1], v.shape[-1], dtype=torch.float64) if h0 is None else h0[n].clone()
        A = S.abs()
        for t in range(lo, hi):
            e = torch.exp(g[t])[:, None, None]
            S = e * S + k[t][..., None] * v[t][:, None, :]
            A = e * A + k[t].abs()[..., None] * v[t].abs()[:, None, :]
            o[t], size[t] = (S * q[t][..., None]).sum(-2), (A * q[t].abs()[..., None]).sum(-2)
        final.append(S)
        fsize.append(A)
    return dict(o=o, final_state=torch.stack(final)), dict(o=size, final_state=torch.stack(fsize))


def _rows_sum(x, heads):
    T, H, W = x.shape
    return x.view(T, heads, H // heads, W).sum(2)


def backward(q, k, v, g, cu, d_o, d_final=None, h0=None):
    """dict(dq, dk, dv, dg, dh0) and the magnitudes of their terms.  Those of dg are
    the largest of its sequence and head: the kernel adds up from the end what
    passes each chunk's border."""
    T, H = g.shape
    heads = [x.shape[1] for x in (q, k, v)]
    q, k, v = (of_heads(x, H) for x in (q, k, v))
    K, V = q.shape[-1], v.shape[-1]
    out = dict(dq=torch.zeros(T, H, K, dtype=torch.float64), dk=torch.zeros(T, H, K, dtype=torch.float64),
               dv=torch.zeros(T, H, V, dtype=torch.float64), dg=torch.zeros(T, H, dtype=torch.float64), dh0=[])
    size = {n: torch.zeros_like(t) for n, t in out.items() if n != "dh0"} | dict(dh0=[])
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        S = torch.zeros(H, K, V, dtype=torch.float64) if h0 is None else h0[n].clone()
        states, A = [S], [S.abs()]
        for t in range(lo, hi):
            e = torch.exp(g[t])[:, None, None]
            S = e * S + k[t][..., None] * v[t][:, None, :]
            states.append(S)
            A.append(e * A[-1] + k[t].abs()[..., None] * v[t].abs()[:, None, :])
            out["dq"][t], size["dq"][t] = (S * d_o[t][:, None, :]).sum(-1), (A[-1] * d_o[t].abs()[:, None, :]).sum(-1)
        L = torch.zeros(H, K, V, dtype=torch.float64) if d_final is None else d_final[n].clone()
        B = L.abs()
        for t in range(hi - 1, lo - 1, -1):
            L = L + q[t][..., None] * d_o[t][:, None, :]
            B = B + q[t].abs()[..., None] * d_o[t].abs()[:, None, :]
            out["dk"][t], size["dk"][t] = (L * v[t][:, None, :]).sum(-1), (B * v[t].abs()[:, None, :]).sum(-1)
            out["dv"][t], size["dv"][t] = (L * k[t][..., None]).sum(-2), (B * k[t].abs()[..., None]).sum(-2)
            e = torch.exp(g[t])[:, None, None]
            L, B = e * L, e * B
            out["dg"][t], size["dg"][t] = (L * states[t - lo]).sum((-1, -2)), (B * A[t - lo]).sum((-1, -2))
        size["dg"][lo:hi] = size["dg"][lo:hi].amax(0)
        out["dh0"].append(L)
        size["dh0"].append(B)
    for d in (out, size):
        d["dh0"] = torch.stack(d["dh0"])
        for m, h in zip(("dq", "dk", "dv"), heads):
            d[m] = _rows_sum(d[m], h)
    return out, size


# A sum of n terms in the matrix cores loses at most one EPS of its terms'
# magnitude for each of them.  The parts of a split factor count as terms; the
# rest of the last part is 2^-16 with two parts and EPS with three.
def state_factor(cu):
    """EPS of a state's terms, as a count: a chunk's decay (two), the weights' (an
    exponential of at most 2^-149: 110), 3 x 64 terms, for every chunk of the
    longest sequence and the piece borders among them (twice)."""
    chunks = max(-(-(b - a) // 64) for a, b in zip(cu, cu[1:]))
    return 110 + 2 * (chunks + 1) * (3 * 64 + 2)


def pass_factor(cu, width, fp32):
    """EPS of an output's terms: x . y (width terms), decay (110), P's parts by 64
    tokens, the state's by width, the rests, the state itself."""
    parts = 3 if fp32 else 2
    rest = 1 if fp32 else 2 ** 8
    return width + 110 + parts * (64 + width) + 2 * rest + state_factor(cu)


def forward_bounds(size, cu, K, o_fp32):
    return dict(o=EPS * pass_factor(cu, K, o_fp32) * size["o"],
                final_state=EPS * state_factor(cu) * size["final_state"])


def backward_bounds(size, cu, K, V, fp32, H):
    """dq and dk are passes over V, dv over K, H more for shared heads.  dg is a sum
    of 64 x 64 pairs and of rows of the passes' state part (three parts always),
    and its border terms run from a chunk to the next."""
    chunks = max(-(-(b - a) // 64) for a, b in zip(cu, cu[1:]))
    dg = (64 + chunks) * 8 + K + V + (2 + chunks) * pass_factor(cu, V, True)
    return dict(dq=EPS * (pass_factor(cu, V, fp32) + H) * size["dq"], dk=EPS * (pass_factor(cu, V, fp32) + H) * size["dk"],
                dv=EPS * (pass_factor(cu, K, fp32) + H) * size["dv"], dg=EPS * dg * size["dg"],
                dh0=EPS * state_factor(cu) * size["dh0"])
