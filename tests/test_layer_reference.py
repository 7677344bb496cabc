"""The 64-bit reference of the operators around the recurrence: its gradients
against automatic differentiation and against central differences, its single
tokens against the sequence forms (CPU)."""
import pytest
import torch

from oracle import kda_oracle as ko
import layer_reference as lr


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _check_gradients(f, inputs, cotangents, grads, step=1e-5):
    """``grads`` (by input name) against autograd of sum <f, cotangent> and, in a
    random direction, against a central difference (error O(step^2))."""
    leaves = {n: t.clone().requires_grad_() for n, t in inputs.items()}

    def loss(xs):
        return sum((y * cotangents[n]).sum() for n, y in f(**xs).items())

    loss(leaves).backward()
    for n, want in grads.items():
        torch.testing.assert_close(want, leaves[n].grad, rtol=1e-10, atol=1e-10, msg=n)
        move = _randn(*inputs[n].shape, seed=99)
        up = loss({**inputs, n: inputs[n] + step * move})
        down = loss({**inputs, n: inputs[n] - step * move})
        torch.testing.assert_close((want * move).sum(), (up - down) / (2 * step), rtol=1e-6, atol=1e-6, msg=n)


@pytest.mark.parametrize("bias", [True, False])
def test_prepare_gradients(bias):
    T, H, K = 3, 2, 8
    x = dict(q=_randn(T, H, K, seed=1), k=_randn(T, H, K, seed=2), gate=_randn(T, H, K, seed=3),
             beta=_randn(T, H, seed=4), a_log=_randn(H, seed=5))
    if bias:
        x["dt_bias"] = _randn(H, K, seed=6)
    d = dict(q=_randn(T, H, K, seed=7), k=_randn(T, H, K, seed=8), g=_randn(T, H, K, seed=9), beta=_randn(T, H, seed=10))
    b = x.get("dt_bias")
    got = lr.prepare_backward(x["q"], x["k"], x["gate"], x["beta"], x["a_log"], b, 0.7, 1e-3, d["q"], d["k"], d["g"],
                              d["beta"])
    names = dict(dq_raw="q", dk_raw="k", dgate_raw="gate", dbeta_raw="beta", da_log="a_log", ddt_bias="dt_bias")
    _check_gradients(lambda dt_bias=None, **a: lr.prepare(**a, dt_bias=dt_bias, q_scale=0.7, eps=1e-3), x, d,
                     {names[n]: t for n, t in got.items() if t is not None})


@pytest.mark.parametrize("kind", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("scaled", [True, False])
def test_output_norm_gradients(kind, scaled):
    T, H, V = 3, 2, 5
    x = dict(o=_randn(T, H, V, seed=1), weight=_randn(V, seed=2))
    if kind != "none":
        x["gate"] = _randn(T, H, V, seed=3)
    if scaled:
        x["res_scale"] = _randn(H, V, seed=4)
    dy = _randn(T, H, V, seed=5)
    got = lr.output_norm_backward(dy, x["o"], x["weight"], x.get("gate"), kind, x.get("res_scale"), 1e-3)

    def f(gate=None, res_scale=None, **a):
        return dict(y=lr.output_norm(gate=gate, kind=kind, res_scale=res_scale, residual=_randn(T, H, V, seed=6),
                                     eps=1e-3, **a))

    _check_gradients(f, x, dict(y=dy), {n[2:]: t for n, t in got.items() if t is not None})


@pytest.mark.parametrize("tied", [True, False])
def test_scan_gradients(tied):
    cu, D = [0, 1, 6, 9], 3
    x = dict(x=_randn(9, D, seed=1), g=-_randn(9, D, seed=2).abs(), h0=_randn(3, D, seed=3))
    d = dict(h=_randn(9, D, seed=4), final=_randn(3, D, seed=5))
    h, _ = lr.scan(x["x"], x["g"], cu, x["h0"], tied)
    got = lr.scan_backward(x["x"], x["g"], h, cu, x["h0"], tied, d["h"], d["final"])

    def f(x, g, h0):
        a = torch.exp(g)
        u = -torch.expm1(g) * x if tied else x
        rows, final = [], []
        for n in range(3):
            now = h0[n]
            for t in range(cu[n], cu[n + 1]):
                now = a[t] * now + u[t]
                rows.append(now)
            final.append(now)
        return dict(h=torch.stack(rows), final=torch.stack(final))

    _check_gradients(f, x, d, {n[1:]: t for n, t in got.items()})


def test_scan_step_is_the_scan():
    x, g, h0 = _randn(5, 4, seed=1), -_randn(5, 4, seed=2).abs(), _randn(1, 4, seed=3)
    h, final = lr.scan(x, g, [0, 5], h0, True)
    got, pool = lr.scan_step(x, g, torch.cat([h0 * 2, h0]), torch.full((5,), 1), torch.zeros(5, 4).double(), True)
    torch.testing.assert_close(got, h)
    torch.testing.assert_close(pool, torch.cat([h0 * 2, final]))


def test_step_is_the_recurrence():
    T, H, K = 6, 2, 8
    q, k, v = (_randn(T, H, K, seed=s) for s in (1, 2, 3))
    g, beta, h0 = -_randn(T, H, K, seed=4).abs(), torch.sigmoid(_randn(T, H, seed=5)), _randn(1, H, K, K, seed=6)
    o, final = ko.recurrence(q.numpy(), k.numpy(), v.numpy(), g.numpy(), beta.numpy(), [0, T],
                             h0=h0.numpy())
    got, pool, _, _ = lr.step(q, k, v, g, beta, h0, torch.zeros(T), torch.zeros(T, H, K).double())
    torch.testing.assert_close(got, torch.from_numpy(o))
    torch.testing.assert_close(pool, torch.from_numpy(final))
