"""The 64-bit reference of linear attention and of the norms and rotation before
it: gradients against automatic differentiation and against differences, the
forms against each other (CPU only)."""
import math

import pytest
import torch

import linear_reference as ref

F64 = torch.float64


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


@pytest.mark.parametrize("D,R,interleaved,weighted", [(8, 8, False, True), (10, 6, True, True), (6, 0, False, False),
                                                      (12, 4, False, False), (4, 2, True, True)])
def test_rotation(D, R, interleaved, weighted):
    T, H = 5, 3
    x, d = _randn(T, H, D, seed=1).requires_grad_(), _randn(T, H, D, seed=2)
    w = (1 + 0.3 * _randn(D, seed=3)).requires_grad_() if weighted else None
    pos, inv = torch.tensor([0, 3, -7, 1000, 12]), torch.rand(R // 2, dtype=F64) if R else None
    args = (0.7, 1e-3, pos, inv, interleaved)
    y = ref.norm_rotate(x, w, *args)
    y.backward(d)
    dx, dw = ref.norm_rotate_backward(d, x.detach(), None if w is None else w.detach(), *args)
    assert torch.allclose(dx, x.grad, rtol=1e-12, atol=1e-13)
    if weighted:
        assert torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-13)
    # central differences along one direction
    u, h = _randn(T, H, D, seed=4), 1e-5
    f = lambda s: float((ref.norm_rotate(x.detach() + s * u, None if w is None else w.detach(), *args) * d).sum())  # noqa: E731
    assert math.isclose((f(h) - f(-h)) / (2 * h), float((dx * u).sum()), rel_tol=1e-7, abs_tol=1e-8)
    # a rotation keeps each pair's length, and turns back
    t = ref.turn(d, pos, inv, interleaved)
    assert torch.allclose((t * t).sum(-1), (d * d).sum(-1), rtol=1e-12)
    assert torch.allclose(ref.turn(t, pos, inv, interleaved, back=True), d, rtol=1e-12, atol=1e-13)
    assert torch.equal(t[..., R:], d[..., R:])


def test_rotation_by_hand():
    """One pair of each layout by ninety degrees."""
    x = torch.arange(1.0, 5.0, dtype=F64).view(1, 1, 4)
    pos, inv = torch.tensor([1]), torch.tensor([math.pi / 2, 0.0], dtype=F64)
    assert torch.allclose(ref.turn(x, pos, inv, False), torch.tensor([[[-3.0, 2.0, 1.0, 4.0]]], dtype=F64))
    assert torch.allclose(ref.turn(x, pos, inv, True), torch.tensor([[[-2.0, 1.0, 3.0, 4.0]]], dtype=F64))


def test_only_relative_positions_count():
    q, k = _randn(1, 1, 8, seed=1), _randn(1, 1, 8, seed=2)
    inv = torch.rand(4, dtype=F64)
    dots = [float((ref.turn(q, torch.tensor([p + 5]), inv, False) * ref.turn(k, torch.tensor([p]), inv, False)).sum())
            for p in (0, 17, -400)]
    assert max(dots) - min(dots) < 1e-12


def test_step_is_the_recurrence():
    q, k, v = _randn(2, 3, seed=1), _randn(2, 3, seed=2), _randn(2, 4, seed=3)
    g, S = torch.tensor([-0.5, -math.inf], dtype=F64), _randn(2, 3, 4, seed=4)
    o, new, size = ref.step(q, k, v, g, S)
    for h in range(2):
        want = math.exp(g[h]) * S[h] + torch.outer(k[h], v[h])
        assert torch.allclose(new[h], want) and torch.allclose(o[h], want.T @ q[h])
        assert (size[h] >= want.abs() - 1e-12).all()


def test_heads_are_shared_by_neighbours():
    x = _randn(5, 2, 3, seed=1)
    y = ref.of_heads(x, 6)
    assert y.shape == (5, 6, 3)
    for h in range(6):
        assert torch.equal(y[:, h], x[:, h // 3])


def _packed(cu, H, Hq, Hk, Hv, K, V, init, seed):
    T, N = cu[-1], len(cu) - 1
    x = dict(q=_randn(T, Hq, K, seed=seed), k=_randn(T, Hk, K, seed=seed + 1), v=_randn(T, Hv, V, seed=seed + 2),
             g=-torch.rand(T, H, generator=torch.Generator().manual_seed(seed + 3), dtype=F64))
    if init:
        x["h0"] = _randn(N, H, K, V, seed=seed + 4)
    return x, _randn(T, H, V, seed=seed + 5), _randn(N, H, K, V, seed=seed + 6)


def test_forward_is_attention_with_decay():
    """Over all pairs of a sequence's tokens, and the bound's magnitudes."""
    cu = [0, 1, 6, 17]
    x, _, _ = _packed(cu, 4, 2, 1, 4, 3, 5, False, 7)
    out, size = ref.forward(**x, cu=cu)
    q, k, v = (ref.of_heads(x[n], 4) for n in "qkv")
    for lo, hi in zip(cu, cu[1:]):
        G = torch.cumsum(x["g"][lo:hi], 0)
        D = torch.exp(G[:, None] - G[None]) * torch.ones(hi - lo, hi - lo, dtype=F64).tril()[..., None]
        o = torch.einsum("ihk,jhk,ijh,jhv->ihv", q[lo:hi], k[lo:hi], D, v[lo:hi])
        assert torch.allclose(out["o"][lo:hi], o, rtol=1e-11, atol=1e-12)
    assert (size["o"] >= out["o"].abs() - 1e-12).all()


@pytest.mark.parametrize("Hq,Hk,Hv,init", [(4, 4, 4, True), (2, 2, 4, True), (4, 1, 2, False)])
def test_backward(Hq, Hk, Hv, init):
    """Against automatic differentiation of the forward pass and differences."""
    cu = [0, 3, 4, 13]
    x, d_o, d_final = _packed(cu, 4, Hq, Hk, Hv, 3, 5, init, 11)
    leaves = {n: t.clone().requires_grad_() for n, t in x.items()}
    loss = _loss(leaves, cu, d_o, d_final)
    loss.backward()
    out, size = ref.backward(**x, cu=cu, d_o=d_o, d_final=d_final)
    for n, t in leaves.items():
        name = "dh0" if n == "h0" else "d" + n
        assert torch.allclose(out[name], t.grad, rtol=1e-10, atol=1e-11), name
        assert (size[name] >= out[name].abs() - 1e-12).all()
        u, h = _randn(*t.shape, seed=99), 1e-5
        with torch.no_grad():
            f = [float(_loss({**x, n: x[n] + s * u}, cu, d_o, d_final)) for s in (h, -h)]
        assert math.isclose((f[0] - f[1]) / (2 * h), float((out[name] * u).sum()), rel_tol=1e-6, abs_tol=1e-6)


def _loss(x, cu, d_o, d_final):
    """sum d_o o + sum d_final S_T, by stacking (in place writes cannot be differentiated)."""
    H = x["g"].shape[1]
    q, k, v = (ref.of_heads(x[n], H) for n in "qkv")
    loss = 0.0
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        S = x["h0"][n] if "h0" in x else torch.zeros(H, q.shape[-1], v.shape[-1], dtype=F64)
        for t in range(lo, hi):
            S = torch.exp(x["g"][t])[:, None, None] * S + k[t][..., None] * v[t][:, None, :]
            loss = loss + ((S * q[t][..., None]).sum(-2) * d_o[t]).sum()
        loss = loss + (S * d_final[n]).sum()
    return loss


def test_steps_are_the_forward_pass():
    cu = [0, 5]
    x, _, _ = _packed(cu, 2, 2, 2, 2, 3, 4, True, 3)
    out, _ = ref.forward(**x, cu=cu)
    S = x["h0"][0]
    for t in range(5):
        o, S, _ = ref.step(x["q"][t], x["k"][t], x["v"][t], x["g"][t], S)
        assert torch.allclose(o, out["o"][t])
    assert torch.allclose(S, out["final_state"][0])
