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
