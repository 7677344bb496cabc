"""Single tokens of linear attention on the GPU against their 64-bit reference,
within the reference's bounds."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer
import layer_reference as lr
import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
NONE = -1


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _case(B, H, Hq, Hk, Hv, K, V, g_kind, num_slots, seed):
    x = dict(q=_randn(B, Hq, K, seed=seed, dtype=BF), k=_randn(B, Hk, K, seed=seed + 1, dtype=BF),
             v=_randn(B, Hv, V, seed=seed + 2, dtype=BF))
    g = -torch.nn.functional.softplus(_randn(H if g_kind == "head" else B * H, seed=seed + 3))
    g[0] = 0.0
    if len(g) > 2:
        g[1], g[2] = float("-inf"), -200.0
    g = g if g_kind == "head" else g.view(B, H).to(BF if g_kind == "bf16" else F32)
    return x, g, _randn(num_slots, H, K, V, seed=seed + 4)


def _reference(x, g, state, slots):
    """Row after row; o NaN where a row is unused, with the bounds of each row's own
    step from the kernel's previous state (rows of one slot add theirs up)."""
    B, H = len(slots), state.shape[1]
    pool = state.double().clone()
    q, k, v = (ref.of_heads(x[n].double(), H) for n in ("q", "k", "v"))
    g = g.double().expand(B, H)
    o = torch.full((B, H, state.shape[3]), float("nan"), dtype=torch.float64)
    slack_o, slack = torch.zeros_like(o), torch.zeros_like(pool)
    for b, s in enumerate(slots):
        if 0 <= s < len(pool):
            e = torch.exp(g[b])[:, None, None]
            o[b], pool[s], size = ref.step(q[b], k[b], v[b], g[b], pool[s])
            so, ss = ref.step_bounds(q[b], size)
            slack_o[b] = so + (e * slack[s] * q[b].abs()[..., None]).sum(-2)
            slack[s] = e * slack[s] + ss
    return o, pool, slack_o, slack


# B, H, Hq, Hk, Hv, K, V, g, o, slots
CASES = [
    (1, 1, 1, 1, 1, 128, 128, "fp32", BF, None),
    (3, 4, 4, 4, 4, 128, 128, "head", F32, [2, 0, 4]),
    (5, 6, 2, 2, 6, 64, 128, "fp32", BF, [4, NONE, 0, 7, 2]),
    (5, 6, 6, 3, 3, 128, 64, "bf16", F32, [1, 1, 0, 1, 99]),
    (2, 3, 3, 1, 3, 8, 8, "fp32", F32, None),
    (4, 2, 1, 1, 1, 40, 96, "head", BF, [3, 2, 1, 0]),
    (2, 2, 2, 2, 2, 120, 104, "fp32", F32, [0, 0]),
    (2, 2, 2, 2, 2, 96, 120, "bf16", BF, None),
    (1, 5, 1, 1, 5, 128, 8, "fp32", F32, [0]),
    (1, 5, 1, 1, 5, 8, 128, "fp32", BF, [0]),
    (70, 2, 2, 2, 2, 64, 64, "fp32", BF, [i * 7 % 80 for i in range(70)]),
]


@pytest.mark.parametrize("B,H,Hq,Hk,Hv,K,V,g_kind,o_dtype,slots", CASES)
def test_linear_step(B, H, Hq, Hk, Hv, K, V, g_kind, o_dtype, slots):
    n = B if slots is None else 5 if B < 70 else 80
    x, g, state = _case(B, H, Hq, Hk, Hv, K, V, g_kind, n, seed=K + V)
    dev = {m: t.to(DEV) for m, t in x.items()}
    where = None if slots is None else torch.tensor(slots, dtype=torch.int32, device=DEV)
    pool, mark = state.to(DEV), 3.5
    out = torch.full((B, H, V), mark, dtype=o_dtype, device=DEV)
    got = layer.linear_step(dev["q"], dev["k"], dev["v"], g.to(DEV), pool, where, o=out)
    assert got is out
    o, new, slack_o, slack = _reference(x, g, state, range(B) if slots is None else slots)
    unused = o.isnan().all(-1).all(-1)
    assert (out.cpu()[unused] == mark).all()
    lr.assert_close(out.cpu()[~unused], o[~unused], slack_o[~unused], "o")
    lr.assert_close(pool, new, slack, "state")
    # another pool to write: the old one, and slots that no row names, stay
    old, other = state.to(DEV), torch.full_like(pool, mark)
    again = layer.linear_step(dev["q"], dev["k"], dev["v"], g.to(DEV), old, where, state_out=other, o_dtype=o_dtype)
    assert torch.equal(old.cpu(), state) and torch.equal(again[~unused], out[~unused])
    named = torch.zeros(n, dtype=torch.bool)
    named[[s for s in (range(B) if slots is None else slots) if 0 <= s < n]] = True
    assert torch.equal(other[named], pool[named]) and (other[~named] == mark).all()


def test_not_finite():
    """A state or gate that is not finite stays in its own row and head."""
    x, g, state = _case(3, 2, 2, 2, 2, 64, 64, "fp32", 3, seed=3)
    dev = {m: t.to(DEV) for m, t in x.items()}
    base = layer.linear_step(dev["q"], dev["k"], dev["v"], g.to(DEV), state.to(DEV))
    state[1, 0, 3, 4], g[2, 1] = float("inf"), float("nan")
    pool = state.to(DEV)
    got = layer.linear_step(dev["q"], dev["k"], dev["v"], g.to(DEV), pool)
    assert not got[1, 0].isfinite().all() and got[2, 1].isnan().all()
    got[1, 0], got[2, 1] = base[1, 0], base[2, 1]
    assert torch.equal(got, base)


def test_captured_follows_slots():
    x, g, state = _case(6, 2, 1, 1, 2, 128, 64, "fp32", 9, seed=4)
    dev = {m: t.to(DEV) for m, t in x.items()}
    gd, slots = g.to(DEV), torch.arange(6, dtype=torch.int32, device=DEV)
    pool, pool2 = state.to(DEV), state.to(DEV)
    layer.linear_step(dev["q"], dev["k"], dev["v"], gd, pool.clone(), slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.linear_step(dev["q"], dev["k"], dev["v"], gd, pool, slots)
    for i in range(3):
        slots.copy_(torch.tensor([(3 * i + j) % 9 if j != i else -1 for j in range(6)], dtype=torch.int32))
        keep = got.clone()
        graph.replay()
        torch.cuda.synchronize()
        want = layer.linear_step(dev["q"], dev["k"], dev["v"], gd, pool2, slots)
        assert torch.equal(pool, pool2)
        want[i] = keep[i]   # the unused row: what the memory held, NaN or not, so bits are compared
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_refusals():
    x, g, state = _case(2, 4, 2, 2, 4, 64, 64, "fp32", 3, seed=4)
    q, k, v = (x[n].to(DEV) for n in ("q", "k", "v"))
    g, state = g.to(DEV), state.to(DEV)
    with pytest.raises(TypeError, match="q"):
        layer.linear_step(q.float(), k, v, g, state)
    with pytest.raises(ValueError, match="state"):
        layer.linear_step(q, k, v, g, state[:, :3].contiguous())
    with pytest.raises(ValueError, match="g"):
        layer.linear_step(q, k, v, g[:1], state)
    with pytest.raises(TypeError, match="g"):
        layer.linear_step(q, k, v, g.half(), state)
    with pytest.raises(ValueError, match="contiguous"):
        layer.linear_step(q, k, v.transpose(0, 1).contiguous().transpose(0, 1), g, state)
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):       # 4 states, 3 key heads
        layer.linear_step(q, torch.cat([k, k[:, :1]], 1), v, g, state)
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):       # fewer slots than rows
        layer.linear_step(q, k, v, g, state[:1])
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):       # overlapping pools
        both = torch.zeros(4, 4, 64, 64, device=DEV)
        layer.linear_step(q, k, v, g, both[:3], state_out=both[1:])
    with pytest.raises(kda.KdaError, match="UNSUPPORTED"):
        layer.linear_step(q[..., :12].contiguous(), k[..., :12].contiguous(), v, g, state[:, :, :12].contiguous())
