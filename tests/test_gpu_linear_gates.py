"""The gradient of linear attention's gates where neighbouring chunks are of very
different size: behind a gate that forgets all or nearly all, and between tokens
that are many times larger.  Against the 64-bit reference, part by part, so that
the large part's roundings cannot hide the small part's."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer
import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32

# As over whole outputs (test_gpu_linear): roundings are independent, so that they
# stay near the largest single one, 2^-24 of a value, times a root of their number,
# 16; what passes by a chunk is at most four steps from a product of both states,
# each with the roundings of two sums of that kind and of one magnitude: 4 times that.
PART = 64 * ref.EPS


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _inputs(T, H, K, V, seed):
    return (_randn(T, H, K, seed=seed, dtype=BF, scale=K ** -0.5), _randn(T, H, K, seed=seed + 1, dtype=BF),
            _randn(T, H, V, seed=seed + 2, dtype=BF), _randn(T, H, V, seed=seed + 3, dtype=BF))


def _dg(plan, q, k, v, g, d_o):
    return layer.linear_backward(plan, *(t.to(DEV) for t in (q, k, v, g, d_o)))["dg"].cpu().double()


def _reference(q, k, v, g, cu, d_o):
    return ref.backward(*(t.double() for t in (q, k, v, g)), cu, d_o.double())[0]["dg"]


def _off(got, want):
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("K,V", [(128, 128), (64, 64), (24, 128)])
@pytest.mark.parametrize("gate", [float("-inf"), -100.0, -30.0, -12.0])
def test_small_gradients_before_a_gate(K, V, gate):
    """One fragment of 13 chunks, a gate in its seventh, and outputs that count 2^-13
    as much before it."""
    T, H, at = 13 * 64 - 3, 2, 6 * 64 + 10
    q, k, v, d_o = _inputs(T, H, K, V, seed=K)
    g = torch.full((T, H), -0.01)
    g[:, 1] = -0.002
    g[at] = gate
    d_o[:at] *= 2.0 ** -13
    got, want = _dg(kda.Plan([0, T], 1), q, k, v, g, d_o), _reference(q, k, v, g, [0, T], d_o)
    for h in range(H):
        for part in (slice(1, at), slice(at + 1, T)):
            assert _off(got[part, h], want[part, h]) <= PART, (h, part)
    if gate <= -100.0:
        assert (got[at] == 0).all()
    else:   # what that gate scales: below e^gate times the sizes of both states
        state = torch.zeros(H, K, V, dtype=torch.float64)
        for t in range(at):
            state = torch.exp(g[t].double())[:, None, None] * state + (k[t].double()[..., None] * v[t].double()[:, None, :])
        cotangent = torch.zeros_like(state)
        for t in range(T - 1, at - 1, -1):
            cotangent = cotangent + q[t].double()[..., None] * d_o[t].double()[:, None, :]
            cotangent = cotangent * (torch.exp(g[t].double())[:, None, None] if t > at else 1.0)
        most = torch.exp(torch.tensor(gate).double()) * state.flatten(1).norm(dim=1) * cotangent.flatten(1).norm(dim=1)
        assert ((got[at] - want[at]).abs() <= most).all()


@pytest.mark.parametrize("K,V,plan", [(64, 64, 1), (128, 32, 1), (64, 64, 3)])
def test_quiet_tokens_between_loud_ones(K, V, plan):
    """Values and cotangents 2^-17 as large in the middle of 41 chunks, with decays that
    forget the loud ones within some chunks, or not."""
    T, H, lo, hi = 40 * 64 + 17, 3, 700, 1900
    q, k, v, d_o = _inputs(T, H, K, V, seed=K + V + plan)
    g = -torch.tensor([0.1, 0.02, 0.001]).expand(T, H).contiguous()
    for t in (v, d_o):
        t[lo:hi] *= 2.0 ** -17
    got, want = _dg(kda.Plan([0, T], plan), q, k, v, g, d_o), _reference(q, k, v, g, [0, T], d_o)
    for h in range(H):
        for part in (slice(1, lo), slice(lo + 300, hi - 300), slice(hi, T)):
            assert _off(got[part, h], want[part, h]) <= PART, (h, part)


def test_what_is_not_finite_does_not_reach_back():
    """A key that is not finite counts in no gate at or before its token, a query in
    none behind it, also within one fragment."""
    T, H, at = 12 * 64, 2, 5 * 64 + 7
    q, k, v, d_o = _inputs(T, H, 64, 64, seed=9)
    g, plan = torch.full((T, H), -0.01), kda.Plan([0, T], 1)
    base = _dg(plan, q, k, v, g, d_o)
    for tensor, kept in ((k, slice(0, 5 * 64)), (q, slice(6 * 64, T))):
        keep = tensor[at, 1].clone()
        tensor[at, 1] = float("nan")
        got = _dg(plan, q, k, v, g, d_o)
        tensor[at, 1] = keep
        assert torch.equal(got[:, 0], base[:, 0])
        assert got[kept, 1].isfinite().all() and _off(got[kept, 1], base[kept, 1]) <= PART
