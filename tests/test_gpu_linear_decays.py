"""How exact linear attention's decays are in what is FP32: with inputs of single
channels every result is one product of a decay, so that nothing else can hide it."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer
import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
H = 48
# In EPS of the value.  A decay: 4, as exact_exp.  P or a state: its decay and a
# rounding, its three parts (1), a sum of three (3): 9; an output through the state
# has the decay behind the sum; the gates' sums add zeros.  12 leaves 2^-20 of those
# for the products of errors and the sums' order.
ONE = 12 * ref.EPS
# Parts below 2^-126, where BF16's normal numbers end, are 0 to the matrix cores.  Of a
# value x of 2^-115 the parts are at most 2^-115, 2^-9 2^-115 = 2^-124 and 2^-133: the
# third is always lost there, 2^-133 / 2^-116 = 128 EPS of x, the second where it
# happens to be small.  What is lost, with factors of 1 beside it, is below 2^-126 (1 +
# 2^-9) in all: nothing next to 12 EPS of results above 2^-100.
LOST = 1.01 * torch.finfo(F32).tiny


def _gates(T, seed):
    """Of about -80 in all: decays down to e^-83, far from FP32's least."""
    return -(80.0 / T) * (0.97 + 0.06 * torch.rand(T, H, generator=torch.Generator().manual_seed(seed)))


def _hot(T, width, tokens=None):
    """Channel 0 of every token, or of those named."""
    x = torch.zeros(T, H, width, dtype=BF)
    x[slice(None) if tokens is None else tokens, :, 0] = 1.0
    return x


def _state(K, V, seed):
    """One value a head, in the corner."""
    s = torch.zeros(1, H, K, V)
    s[0, :, 0, 0] = 1 + torch.rand(H, generator=torch.Generator().manual_seed(seed))
    return s


def _same(got, want, bound):
    for n, t in want.items():
        off = (got[n].cpu().double() - t).abs()
        worst = float((off / t.abs().clamp(min=1e-300)).max()) / ref.EPS
        assert (off <= bound * t.abs() + LOST).all() and (off[t == 0] == 0).all(), (n, f"{worst:.1f} EPS")


SIZES = [(8, 8), (128, 64), (128, 128)]


@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("through", ["tokens", "state"])
def test_outputs_and_states(K, V, through):
    T, g = 64, _gates(64, seed=K + V)
    k = _hot(T, K, [0] if through == "tokens" else [])
    h0 = None if through == "tokens" else _state(K, V, seed=1)
    q, v = _hot(T, K), _hot(T, V)
    got = layer.linear_forward(kda.Plan([0, T], 1), *(t.to(DEV) for t in (q, k, v, g)),
                               initial_state=None if h0 is None else h0.to(DEV), o_dtype=F32)
    want, _ = ref.forward(*(t.double() for t in (q, k, v, g)), [0, T], None if h0 is None else h0.double())
    _same(got, want, ONE)


@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("start,end", [("tokens", "tokens"), ("state", "tokens"), ("tokens", "state"), ("state", "state")])
def test_gradients(K, V, start, end):
    """From the first token's key or the initial state to the last token's cotangent or
    the final state's."""
    T, g = 64, _gates(64, seed=K + V + 1)
    q, v = _hot(T, K), _hot(T, V)
    k = _hot(T, K, [0] if start == "tokens" else [])
    d_o = _hot(T, V, [T - 1] if end == "tokens" else [])
    h0 = _state(K, V, seed=1) if start == "state" else torch.zeros(1, H, K, V)
    d_final = _state(K, V, seed=2) if end == "state" else torch.zeros(1, H, K, V)
    got = layer.linear_backward(kda.Plan([0, T], 1), *(t.to(DEV) for t in (q, k, v, g, d_o)), d_final=d_final.to(DEV),
                                initial_state=h0.to(DEV), grad_dtype=F32)
    want, _ = ref.backward(*(t.double() for t in (q, k, v, g)), [0, T], d_o.double(), d_final.double(), h0.double())
    _same(got, want, ONE)


@pytest.mark.parametrize("K,V", SIZES)
def test_pieces(K, V):
    """A state that passes by a piece: 5 for a chunk's decay of it and one for each
    rounding by the scan, twice, then as above: 24."""
    T, g = 192, _gates(192, seed=K + V + 2)
    q, k, v = _hot(T, K), _hot(T, K, []), _hot(T, V)
    h0, d_final, d_o = _state(K, V, seed=1), _state(K, V, seed=2), _hot(T, V, [])
    plan, x = kda.Plan([0, T], 3), [t.to(DEV) for t in (q, k, v, g)]
    got = layer.linear_forward(plan, *x, initial_state=h0.to(DEV), o_dtype=F32)
    want, _ = ref.forward(*(t.double() for t in (q, k, v, g)), [0, T], h0.double())
    _same(got, want, 24 * ref.EPS)
    got = layer.linear_backward(plan, *x, d_o.to(DEV), d_final=d_final.to(DEV), initial_state=h0.to(DEV), grad_dtype=F32)
    want, _ = ref.backward(*(t.double() for t in (q, k, v, g)), [0, T], d_o.double(), d_final.double(), h0.double())
    _same(got, want, 24 * ref.EPS)
