"""The gradient of one gate for a head (g [H]), which is a sum over all tokens, and
sequences of more than 64 chunks in one piece: held over whole outputs, where the
elementwise bounds add up every rounding's largest value and leave room for more
than the gradient itself."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer
import layer_reference as lr
import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# As over whole outputs (test_gpu_linear): independent roundings, 2^-24 of a value times
# a root of their number, 16; in the gates' gradient 4 times that, as what passes by a
# chunk is up to four steps from a product of both states (test_gpu_linear_gates).  Its
# sum over the tokens: what a chunk's 64 tokens have in common, the states' roundings
# and what passes by them, is off for all of them together, which is a root of 64 more
# than a norm over the tokens has.
WHOLE, GATES, SUM = 16 * ref.EPS, 64 * ref.EPS, 128 * ref.EPS


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _rel(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


def _case(T, N, H, K, V, seed):
    return dict(q=_randn(T, H, K, seed=seed, dtype=BF, scale=K ** -0.5), k=_randn(T, H, K, seed=seed + 1, dtype=BF),
                v=_randn(T, H, V, seed=seed + 2, dtype=BF), d_o=_randn(T, H, V, seed=seed + 3, dtype=BF),
                d_final=_randn(N, H, K, V, seed=seed + 4), h0=_randn(N, H, K, V, seed=seed + 5))


def _backward(plan, x, g, **how):
    d = {n: t.to(DEV) for n, t in x.items()}
    return layer.linear_backward(plan, d["q"], d["k"], d["v"], g.to(DEV), d["d_o"], d_final=d["d_final"],
                                 initial_state=d["h0"], **how)


def _reference(cu, x, g):
    w = {n: t.double() for n, t in x.items()}
    out, size = ref.backward(w["q"], w["k"], w["v"], g.double().expand(cu[-1], -1), cu, w["d_o"], w["d_final"], w["h0"])
    return out, size


# cu_seqlens, plan (segments, piece tokens)
SHARED = [([0, 300], (1, 0)), ([0, 300], (3, 0)), ([0, 100, 101, 165, 500], (2, 0)), ([0, 700], (7, 32)),
          (list(range(0, 70 * 5, 5)) + [350], (1, 0)), ([0, 40, 900, 1125], (139, 0))]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
@pytest.mark.parametrize("cu,plan", SHARED)
def test_one_gate_a_head(cu, plan, K, V, dtype):
    """Rates of some tokens to some thousands."""
    T, H = cu[-1], 3
    x = _case(T, len(cu) - 1, H, K, V, seed=T + K)
    g = -torch.tensor([0.5, 0.03, 0.001]).to(dtype)
    plan = kda.Plan(cu, plan[0], piece_tokens=plan[1])
    got = _backward(plan, x, g)["dg"]
    out, size = _reference(cu, x, g)
    want = out["dg"].sum(0)
    assert got.shape == (H,) and got.dtype == dtype
    # the terms' magnitudes, of which the roundings are: the gradient is a good part of them
    terms = out["dg"].norm(dim=0)
    off = (got.cpu().double() - want).abs()
    print(f"{plan.F} fragments", (off / want.abs()).tolist())
    assert (off <= SUM * torch.maximum(want.abs(), terms) + lr.half_step(dtype) * want.abs()).all()
    assert (SUM * torch.maximum(want.abs(), terms) <= 1e-3 * want.abs()).all()   # nothing else would pass


def test_the_fragments_cases_differ():
    assert [kda.Plan(cu, p[0], piece_tokens=p[1]).F for cu, p in SHARED] == [1, 3, 5, 28, 70, 140]


@pytest.mark.parametrize("tail", [1, 7 * 64 + 5])
def test_more_than_64_chunks_in_one_piece(tail):
    """All gradients of a sequence of 64 chunks and some, behind a short one, uncut and in
    pieces of more and of less than 64 chunks."""
    cu, H, K, V = [0, 30, 30 + 64 * 64 + tail], 2, 16, 24
    T = cu[-1]
    x, g = _case(T, 2, H, K, V, seed=tail), -0.02 * torch.rand(T, H, generator=torch.Generator().manual_seed(1))
    want, _ = _reference(cu, x, g)
    for plan in (kda.Plan(cu, 1), kda.Plan(cu, 2, custom_bounds=[0, 20, T]), kda.Plan(cu, 5)):
        got = _backward(plan, x, g, grad_dtype=F32)
        off = {n: _rel(t, want[n]) for n, t in got.items()}
        print(plan.F, off)
        assert off.pop("dg") <= GATES and max(off.values()) <= WHOLE, off


def test_129_chunks_and_one_gate():
    """Three rounds of 64 chunks, a gate a head."""
    cu, H, K, V = [0, 128 * 64 + 3], 1, 8, 8
    x, g = _case(cu[-1], 1, H, K, V, seed=7), -torch.tensor([0.004])
    out, _ = _reference(cu, x, g)
    got = _backward(kda.Plan(cu, 1), x, g)["dg"].cpu().double()
    want = out["dg"].sum(0)
    assert ((got - want).abs() <= SUM * torch.maximum(want.abs(), out["dg"].norm(dim=0))).all()
