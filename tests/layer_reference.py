"""The operators around the recurrence in 64 bits (torch on the CPU), written
from their formulas, with the bounds the GPU tests hold the kernels to.

Every function takes float64 tensors (the exact values of the kernels' inputs)
and returns float64 results.  Gradients are written out; test_layer_reference
checks them against automatic differentiation and against differences.

Bounds.  ``EPS`` = 2^-24 is half a step of FP32 relative to the value, and
``half_step`` that of an output's type.  A kernel's error is at most its
output's rounding plus a few EPS of the magnitudes that enter the result: each
function documents the count it allows.
"""
from __future__ import annotations

import torch

EPS = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_close(got, want, slack, name):
    """|got - want| <= half_step |want| + slack elementwise, and the same where
    the values are not finite; ``slack`` bounds the FP32 arithmetic.  The slack
    is rounded with the value, hence its factor 1 + 2 half steps; values below
    the type's normal range round to multiples of its smallest one."""
    got64, h = got.detach().cpu().double(), half_step(got.dtype)
    assert got64.shape == want.shape, (name, got64.shape, want.shape)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got64), torch.isnan(want)), f"{name}: NaN in other places"
    assert torch.equal(got64[~finite & ~torch.isnan(want)], want[~finite & ~torch.isnan(want)]), f"{name}: infinities"
    slack = torch.as_tensor(slack, dtype=torch.float64).expand_as(want)
    bound = h * want.abs() + slack * (1 + 2 * h) + torch.finfo(got.dtype).tiny
    off = (got64 - want).abs()
    bad = finite & (off > bound)
    if bad.any():
        i = int(torch.argmax(torch.where(finite, off / bound, torch.zeros_like(off))))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{float(got64.flatten()[i])!r}, want {float(want.flatten()[i])!r}, "
                             f"bound {float(bound.flatten()[i])!r}")


# ------------------------------------------------------------- input preparation


def softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))


def sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def prepare(q, k, gate, beta, a_log, dt_bias, q_scale, eps):
    z = gate if dt_bias is None else gate + dt_bias
    return dict(q=q_scale * q / torch.sqrt((q * q).sum(-1, keepdim=True) + eps),
                k=k / torch.sqrt((k * k).sum(-1, keepdim=True) + eps),
                g=-torch.exp(a_log)[:, None] * softplus(z), beta=sigmoid(beta))


def prepare_bounds(want, gate, a_log, dt_bias):
    """q, k: a sum of 128 squares in 8 + 4 additions, a product each, the added
    eps, the reciprocal root and its scale, the product with x: 16 + 4 EPS
    covers them.  g: 2 (1 + |a|) EPS of the rate's exponential; the softplus is
    at least its exponential part, whose argument carries the rounding of z and
    of the exponential's scaled argument, (2 + 2 |z|) EPS, and a few more: all
    relative to the result where z <= 0 and below them where z > 0, but for
    z's own rounding, |z| EPS of the softplus's argument (slope at most 1)."""
    z = gate if dt_bias is None else gate + dt_bias
    zr = gate.abs() if dt_bias is None else gate.abs() + dt_bias.abs()
    rate = torch.exp(a_log)[:, None]
    g = want["g"].abs() * (16 + 2 * a_log.abs()[:, None] + 4 * z.clamp(-200, 200).abs()) + rate * zr.clamp(max=1e30) * sigmoid(z)
    return dict(q=20 * EPS * want["q"].abs(), k=20 * EPS * want["k"].abs(), g=EPS * torch.nan_to_num(g, posinf=0.0),
                beta=16 * EPS * want["beta"] * (1 + 0))


def prepare_backward(q, k, gate, beta, a_log, dt_bias, q_scale, eps, dq, dk, dg, dbeta):
    z = gate if dt_bias is None else gate + dt_bias
    rq = 1 / torch.sqrt((q * q).sum(-1, keepdim=True) + eps)
    rk = 1 / torch.sqrt((k * k).sum(-1, keepdim=True) + eps)
    rate = -torch.exp(a_log)[:, None]
    dz = dg * rate * sigmoid(z)
    b = sigmoid(beta)
    return dict(dq_raw=q_scale * rq * (dq - q * rq * rq * (q * dq).sum(-1, keepdim=True)),
                dk_raw=rk * (dk - k * rk * rk * (k * dk).sum(-1, keepdim=True)),
                dgate_raw=dz, dbeta_raw=dbeta * b * (1 - b),
                da_log=(dg * rate * softplus(z)).sum((0, 2)), ddt_bias=None if dt_bias is None else dz.sum(0))


def prepare_backward_bounds(q, k, gate, beta, a_log, dt_bias, q_scale, eps, dq, dk, dg, dbeta):
    """Of each difference's two terms, 24 EPS (the sums' 13 additions twice, the
    products and roots); dgate and dbeta 16 EPS plus those of the exponentials'
    arguments; sums over n terms: their terms' errors and at most log2(n) + 80
    further additions (a group's walk of at most 64 rows, the partial sums')."""
    z = gate if dt_bias is None else gate + dt_bias
    zabs = (gate.abs() if dt_bias is None else gate.abs() + dt_bias.abs()) + 1
    rq = 1 / torch.sqrt((q * q).sum(-1, keepdim=True) + eps)
    rk = 1 / torch.sqrt((k * k).sum(-1, keepdim=True) + eps)
    rate = torch.exp(a_log)[:, None]
    arg = 24 + 2 * a_log.abs()[:, None] + 4 * zabs
    dz = (dg * rate * sigmoid(z)).abs() * arg
    soft = (dg * rate).abs() * (softplus(z) * arg)
    b = sigmoid(beta)
    return dict(dq_raw=40 * EPS * abs(q_scale) * rq * (dq.abs() + q.abs() * rq * rq * (q * dq).abs().sum(-1, keepdim=True)),
                dk_raw=40 * EPS * rk * (dk.abs() + k.abs() * rk * rk * (k * dk).abs().sum(-1, keepdim=True)),
                dgate_raw=EPS * dz,
                # 1 - b loses b's own rounding where b is near 1: 16 EPS of b itself
                dbeta_raw=16 * EPS * dbeta.abs() * b * (1 + beta.abs()),
                da_log=EPS * (soft + 96 * (dg * rate).abs() * softplus(z)).sum((0, 2)),
                ddt_bias=EPS * (dz + 96 * (dg * rate * sigmoid(z)).abs()).sum(0))


# ------------------------------------------------------------- output norm


def activation(z, kind):
    """act(z) and its slope."""
    if kind == "none":
        return torch.ones(()), torch.zeros(())
    s = sigmoid(z)
    return (s, s * (1 - s)) if kind == "sigmoid" else (z * s, s + z * s * (1 - s))


def output_norm(o, weight, gate, kind, res_scale, residual, eps):
    a, _ = activation(gate, kind) if gate is not None else (1.0, 0.0)
    y = a * weight * o / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    y = y if res_scale is None else res_scale * y
    return y if residual is None else residual + y


def output_norm_bound(o, weight, gate, kind, res_scale, residual, eps):
    """The sum of squares of V channels adds at most 32 terms a lane and 8 over
    the lanes; half of their relative error reaches the root.  With the
    products, the gate's exponential (its argument's rounding, |z|) and the
    added residual: (48 + 2 |z|) EPS of the scaled norm and one of the sum."""
    part = output_norm(o, weight, gate, kind, res_scale, None, eps).abs()
    z = 0 if gate is None else gate.abs()
    total = part if residual is None else part + residual.abs()
    return EPS * (part * (48 + 2 * z) + total)


def output_norm_backward(dy, o, weight, gate, kind, res_scale, eps):
    r = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    n = o * r
    a, slope = activation(gate, kind) if gate is not None else (1.0, 0.0)
    s = 1.0 if res_scale is None else res_scale
    dn = dy * s * a * weight
    return dict(d_o=r * (dn - n * (dn * n).mean(-1, keepdim=True)),
                d_gate=None if gate is None else dy * s * weight * n * slope,
                d_weight=(dy * s * a * n).sum((0, 1)), d_res_scale=None if res_scale is None else (dy * a * weight * n).sum(0))


def output_norm_backward_bounds(dy, o, weight, gate, kind, res_scale, eps):
    """As the forward's and the input preparation's: (64 + 2 |z|) EPS of each
    term, sums of rows with at most 160 more additions each (a group's walk of
    at most 64 rows, 16 groups, the partial sums)."""
    r = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    n = (o * r).abs()
    if gate is None:
        a, slope, z = torch.ones(()), torch.zeros(()), torch.zeros(())
    else:
        sg = sigmoid(gate)
        # 1 - sigmoid loses the sigmoid's own rounding: its magnitude is 1 there
        a, slope, z = activation(gate, kind)[0].abs(), sg * (1 + gate.abs()), gate.abs()
    s = torch.ones(()) if res_scale is None else res_scale.abs()
    dn = (dy.abs() * s * a * weight.abs())
    c = 64 + 2 * z
    rows = (dy.abs() * a * n) * (c + 160)
    return dict(d_o=EPS * r * (dn * c + n * (dn * n * c).mean(-1, keepdim=True) + 64 * (dn + n * (dn * n).mean(-1, keepdim=True))),
                d_gate=EPS * dy.abs() * s * weight.abs() * n * slope * c,
                d_weight=EPS * (rows * s).sum((0, 1)), d_res_scale=EPS * (rows * weight.abs()).sum(0))


# ------------------------------------------------------------- per-channel scan


def scan(x, g, cu, h0, tied):
    """h and the final states; one token after another."""
    a = torch.exp(g)
    u = -torch.expm1(g) * x if tied else x
    h, final = torch.empty_like(u), []
    for n in range(len(cu) - 1):
        now = torch.zeros_like(u[0]) if h0 is None else h0[n]
        for t in range(cu[n], cu[n + 1]):
            now = a[t] * now + u[t]
            h[t] = now
        final.append(now)
    return h, torch.stack(final)


def scan_bound(x, g, cu, h0, tied):
    """Error bounds of h and the final states.  h_t is a sum of inputs times
    products of decays.  However the products are grouped, a factor a_t brings
    its own error and one product's and one addition's rounding, on each of at
    most two levels of partial results: (16 + 4 |g_t|) EPS of what it multiplies.
    So with M_t the sum of the magnitudes, W_t = a_t (W_{t-1} + c_t M_{t-1}) +
    16 |u_t| bounds the error in EPS."""
    g = g.clamp(min=-1e4)
    a = torch.exp(g)
    u = (-torch.expm1(g) * x if tied else x).abs()
    c = 16 + 4 * g.abs()
    W, final = torch.empty_like(u), []
    for n in range(len(cu) - 1):
        m = torch.zeros_like(u[0]) if h0 is None else h0[n].abs()
        w = torch.zeros_like(m)
        for t in range(cu[n], cu[n + 1]):
            w = a[t] * (w + c[t] * m) + 16 * u[t]
            m = a[t] * m + u[t]
            W[t] = w
        final.append(w)
    return EPS * W, EPS * torch.stack(final)


def _cotangents(g, cu, dh, d_final):
    """l_t and the decay that each of its steps takes, by walking back."""
    a = torch.exp(g)
    lam = torch.empty_like(dh)
    for n in range(len(cu) - 1):
        carry = torch.zeros_like(dh[0]) if d_final is None else d_final[n]
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            lam[t] = dh[t] + carry
            carry = a[t] * lam[t]
    return a, lam


def _before(h, cu, h0):
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    for n, t in enumerate(cu[:-1]):
        prev[t] = 0 if h0 is None else h0[n]
    return prev


def scan_backward(x, g, h, cu, h0, tied, dh, d_final):
    a, lam = _cotangents(g, cu, dh, d_final)
    prev = _before(h, cu, h0)
    return dict(dx=-torch.expm1(g) * lam if tied else lam, dg=a * lam * (prev - x if tied else prev),
                dh0=torch.stack([a[t] * lam[t] for t in cu[:-1]]))


def scan_backward_bounds(x, g, h, cu, h0, tied, dh, d_final):
    """The forward's bound from the other end for l, then a product or two."""
    g = g.clamp(min=-1e4)
    a = torch.exp(g)
    back = [cu[-1] - t for t in reversed(cu)]
    after = torch.zeros_like(g)
    after[:-1] = g[1:]
    W, M = torch.empty_like(dh), torch.empty_like(dh)
    for n in range(len(cu) - 1):
        m = torch.zeros_like(dh[0]) if d_final is None else d_final[n].abs()
        w = torch.zeros_like(m)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            m = m + dh[t].abs()
            w = w + 16 * m
            W[t], M[t] = w, m
            w = a[t] * (w + (16 + 4 * g[t].abs()) * m)
            m = a[t] * m
    prev = _before(h, cu, h0).abs() + (x.abs() if tied else 0)
    c = 16 + 4 * g.abs()
    share = -torch.expm1(g) if tied else torch.ones_like(g)
    return dict(dx=EPS * share * (W + c * M), dg=EPS * a * prev * (W + c * M),
                dh0=EPS * torch.stack([a[t] * (W[t] + c[t] * M[t]) for t in cu[:-1]]))


def scan_step(x, g, state, slots, h, tied):
    """In row order; returns the outputs and the pool after them."""
    h, pool = h.clone(), state.clone()
    for b in range(x.shape[0]):
        n = b if slots is None else int(slots[b])
        if 0 <= n < pool.shape[0]:
            pool[n] = torch.exp(g[b]) * pool[n] + (-torch.expm1(g[b]) if tied else 1) * x[b]
            h[b] = pool[n]
    return h, pool


# ------------------------------------------------------------- KDA, single tokens


def step(q, k, v, g, beta, state, slots, o, floor=None):
    """In row order; returns o, the pool and bounds of both.  With S' = Diag(e^g) S
    the error of S is at most (12 + 2 |g|) EPS of its own magnitude a token; u
    adds (8 + 128 / 8) EPS of beta (|v| + |S'|^T |k|), and the sums over 128
    channels (16 additions in a thread, 3 across) carry 24 EPS of their
    magnitudes and the errors of what they add."""
    o, pool = o.clone(), state.clone()
    eo, ep = torch.zeros_like(o), torch.zeros_like(state)
    for b in range(q.shape[0]):
        n = b if slots is None else int(slots[b])
        if not 0 <= n < pool.shape[0]:
            continue
        gb = g[b] if floor is None else torch.clamp(g[b], min=floor)
        decay = torch.exp(gb)[:, :, None]
        S = decay * pool[n]
        E = decay * ep[n] + S.abs() * ((12 + 2 * gb.clamp(min=-1e4).abs())[:, :, None]) * EPS
        kc = k[b][:, :, None]
        u = beta[b][:, None] * (v[b] - (S * kc).sum(1))
        eu = beta[b][:, None] * (24 * EPS * (v[b].abs() + (S * kc).abs().sum(1)) + (E * kc.abs()).sum(1))
        pool[n] = S + kc * u[:, None, :]
        ep[n] = E + kc.abs() * eu[:, None, :] + 4 * EPS * (S.abs() + (kc * u[:, None, :]).abs())
        qk = (q[b] * k[b]).sum(-1)
        o[b] = (S * q[b][:, :, None]).sum(1) + qk[:, None] * u
        qa = q[b].abs()[:, :, None]
        eo[b] = (E * qa).sum(1) + 24 * EPS * (S.abs() * qa).sum(1) + qk.abs()[:, None] * eu + 32 * EPS * (
            (q[b] * k[b]).abs().sum(-1)[:, None] * u.abs())
    return o, pool, eo, ep
