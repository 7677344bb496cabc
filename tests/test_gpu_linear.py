"""Linear attention with a decay for each head on the GPU against its 64-bit
reference, within the reference's bounds (linear_reference states the counts)."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer
import layer_reference as lr
import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _d(t):
    return None if t is None else t.to(DEV)


def _w(t):
    return None if t is None else t.double()


def _in_wider(parts):
    """The parts' rows side by side in one tensor, as slices of it."""
    T = parts[0].shape[0]
    wide = torch.cat([p.reshape(T, -1) for p in parts] + [torch.full((T, 8), 7.0, dtype=parts[0].dtype)], 1).to(DEV)
    out, at = [], 0
    for p in parts:
        n = p[0].numel()
        out.append(wide[:, at:at + n].view(p.shape))
        at += n
    return out


# cu_seqlens, plan (segments, bounds, piece tokens), H, Hq, Hk, Hv, K, V, g, fp32 outputs, initial states, slices
CASES = [
    ([0, 1], (1, None, 0), 1, 1, 1, 1, 128, 128, "fp32", False, False, False),
    ([0, 1], (1, None, 0), 2, 2, 2, 2, 64, 64, "head", True, True, False),
    ([0, 64], (1, None, 0), 2, 2, 2, 2, 128, 128, "fp32", True, True, False),
    ([0, 65], (1, None, 0), 3, 1, 1, 3, 128, 64, "fp32", False, False, True),
    ([0, 2, 3, 130], (1, None, 0), 2, 2, 2, 2, 64, 128, "bf16", True, True, True),
    ([0, 300], (5, None, 0), 2, 2, 2, 2, 128, 128, "fp32", True, True, False),
    ([0, 300], (5, None, 0), 2, 2, 2, 2, 128, 128, "fp32", False, True, False),
    ([0, 300], (7, [0, 1, 2, 64, 128, 200, 299, 300], 0), 2, 1, 2, 2, 64, 64, "fp32", True, False, False),
    ([0, 100, 101, 165, 500], (9, None, 0), 4, 2, 1, 4, 128, 96, "fp32", False, True, True),
    ([0, 100, 101, 165, 500], (2, None, 32), 4, 4, 2, 2, 40, 128, "head", True, True, False),
    ([0, 63, 127, 191, 256], (4, None, 0), 1, 1, 1, 1, 8, 8, "fp32", True, True, False),
    ([0, 127], (2, None, 0), 6, 6, 3, 3, 72, 8, "bf16", False, False, True),
    ([0, 127], (3, None, 0), 6, 3, 6, 2, 8, 72, "fp32", True, True, False),
    (list(range(0, 90, 3)) + [90], (11, None, 0), 2, 2, 2, 2, 64, 56, "fp32", True, True, False),
    ([0, 700], (1, None, 0), 2, 2, 2, 2, 112, 120, "fp32", True, False, False),
    ([0, 700], (6, None, 64), 2, 2, 2, 2, 128, 128, "head", True, True, False),
]


def _case(cu, H, Hq, Hk, Hv, K, V, g_kind, init, sliced, seed):
    T, N = cu[-1], len(cu) - 1
    x = [_randn(T, Hq, K, seed=seed, dtype=BF, scale=K ** -0.5), _randn(T, Hk, K, seed=seed + 1, dtype=BF),
         _randn(T, Hv, V, seed=seed + 2, dtype=BF)]
    rate = torch.tensor([1.0, 0.02, 0.2, 0.001, 3.0, 0.0])[:H]
    if g_kind == "head":
        g = -rate.clone()
    else:
        g = -torch.nn.functional.softplus(_randn(T, H, seed=seed + 3)) * rate
        g[::17, 0] = float("-inf")       # a head that is reset now and then
        g[::13, H - 1] = -60.0
        g = g.to(BF if g_kind == "bf16" else F32)
    h0 = _randn(N, H, K, V, seed=seed + 4) if init else None
    dev = _in_wider(x) if sliced else [_d(t) for t in x]
    return x, g, h0, dev


def _plan(cu, plan):
    segments, bounds, piece = plan
    return kda.Plan(cu, segments, custom_bounds=bounds, piece_tokens=piece)


@pytest.mark.parametrize("cu,plan,H,Hq,Hk,Hv,K,V,g_kind,fp32,init,sliced", CASES)
def test_linear_forward(cu, plan, H, Hq, Hk, Hv, K, V, g_kind, fp32, init, sliced):
    x, g, h0, dev = _case(cu, H, Hq, Hk, Hv, K, V, g_kind, init, sliced, seed=cu[-1] + K)
    got = layer.linear_forward(_plan(cu, plan), *dev, _d(g), initial_state=_d(h0), o_dtype=F32 if fp32 else BF)
    out, size = ref.forward(*(_w(t) for t in x), _w(g).expand(cu[-1], H), cu, _w(h0))
    bounds = ref.forward_bounds(size, cu, K, fp32)
    assert got["o"].dtype == (F32 if fp32 else BF)
    for n, t in out.items():
        lr.assert_close(got[n], t, bounds[n], n)


@pytest.mark.parametrize("cu,plan,H,Hq,Hk,Hv,K,V,g_kind,fp32,init,sliced", CASES)
def test_linear_backward(cu, plan, H, Hq, Hk, Hv, K, V, g_kind, fp32, init, sliced):
    T, N = cu[-1], len(cu) - 1
    x, g, h0, dev = _case(cu, H, Hq, Hk, Hv, K, V, g_kind, init, sliced, seed=cu[-1] + K)
    d_o, d_final = _randn(T, H, V, seed=50, dtype=BF), _randn(N, H, K, V, seed=51) if init else None
    got = layer.linear_backward(_plan(cu, plan), *dev, _d(g), _d(d_o), d_final=_d(d_final), initial_state=_d(h0),
                                grad_dtype=F32 if fp32 else BF)
    out, size = ref.backward(*(_w(t) for t in x), _w(g).expand(T, H), cu, _w(d_o), _w(d_final), _w(h0))
    bounds = ref.backward_bounds(size, cu, K, V, fp32, H)
    if g_kind == "head":
        out["dg"] = out["dg"].sum(0)
        bounds["dg"] = bounds["dg"].sum(0) + T * ref.EPS * size["dg"].sum(0)
    assert got["dg"].dtype == g.dtype and got["dq"].dtype == (F32 if fp32 else BF)
    assert (got["dh0"] is None) == (h0 is None)
    for n, t in got.items():
        if t is not None:
            lr.assert_close(t, out[n], bounds[n], n)


def _rel(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


def test_precision_over_whole_outputs():
    """What the elementwise bounds leave open, as they add up every rounding's
    largest value: roundings are independent, so that over a whole FP32 output
    they stay near the largest single one, 2^-24 of a value, times a root of
    their number (a few hundred): 2^-24 * 16 = 1e-6."""
    cu, H, K, V = [0, 40, 500], 3, 128, 128
    x, g, h0, dev = _case(cu, H, H, H, H, K, V, "fp32", True, False, seed=3)
    d_o, d_final = _randn(500, H, V, seed=50, dtype=BF), _randn(2, H, K, V, seed=51)
    plan = kda.Plan(cu, 3)
    args = [_w(t) for t in x]
    got = layer.linear_forward(plan, *dev, _d(g), initial_state=_d(h0), o_dtype=F32)
    out, _ = ref.forward(*args, _w(g), cu, _w(h0))
    back = layer.linear_backward(plan, *dev, _d(g), _d(d_o), d_final=_d(d_final), initial_state=_d(h0), grad_dtype=F32)
    grads, _ = ref.backward(*args, _w(g), cu, _w(d_o), _w(d_final), _w(h0))
    off = {n: _rel(t, out[n]) for n, t in got.items()} | {n: _rel(t, grads[n]) for n, t in back.items()}
    print(off)
    assert max(off.values()) < 1e-6, off


def test_gate_gradient_of_nothing_is_zero():
    """Single tokens from a zero state: their gate scales nothing; and where every
    gate forgets all (-inf, or far below FP32), nothing crosses it."""
    cu, H = [0, 1, 2, 3], 2
    x, g, _, dev = _case(cu, H, H, H, H, 64, 128, "fp32", False, False, seed=5)
    d_o, d_final = _randn(3, H, 128, seed=50, dtype=BF), _randn(3, H, 64, 128, seed=51)
    got = layer.linear_backward(kda.Plan(cu, 2), *dev, _d(g), _d(d_o), d_final=_d(d_final))
    assert (got["dg"] == 0).all()
    cu = [0, 65, 300]
    for gate in (float("-inf"), -200.0):
        x, g, h0, dev = _case(cu, H, H, H, H, 64, 128, "fp32", True, False, seed=6)
        g.fill_(gate)
        d_o, d_final = _randn(300, H, 128, seed=50, dtype=BF), _randn(2, H, 64, 128, seed=51)
        got = layer.linear_backward(kda.Plan(cu, 3), *dev, _d(g), _d(d_o), d_final=_d(d_final), initial_state=_d(h0))
        assert (got["dg"] == 0).all() and (got["dh0"] == 0).all()


def test_sequences_stay_apart():
    """What is not finite stays in its own sequence and head, and reaches no token
    of an earlier chunk."""
    cu, H = [0, 70, 71, 300, 400], 2
    x, g, h0, dev = _case(cu, H, H, H, H, 64, 64, "fp32", True, False, seed=4)
    d_o, d_final = _d(_randn(400, H, 64, seed=5, dtype=BF)), _d(_randn(4, H, 64, 64, seed=6))
    plan, g, h0 = kda.Plan(cu, 5), _d(g), _d(h0)

    def run():
        f = layer.linear_forward(plan, *dev, g, initial_state=h0)
        b = layer.linear_backward(plan, *dev, g, d_o, d_final=d_final, initial_state=h0)
        return {"o": f["o"], "dq": b["dq"], "dk": b["dk"], "dv": b["dv"], "dg": b["dg"][..., None],
                "final_state": f["final_state"], "dh0": b["dh0"]}

    base = run()
    for tensor, at in ((dev[0], (200, 1)), (dev[1], (200, 1)), (dev[2], (200, 1)), (g, (200, 1)), (d_o, (200, 1))):
        keep = tensor[at].clone()
        for bad in (float("nan"), float("inf")):
            tensor[at] = bad
            got = run()
            tensor[at] = keep
            for n, t in got.items():
                if n in ("final_state", "dh0"):
                    t[2, 1] = base[n][2, 1]
                else:
                    if n == "o":
                        assert torch.equal(t[71:135], base[n][71:135]), n
                    t[71:300, 1] = base[n][71:300, 1]
                assert torch.equal(t, base[n]), n


def test_step_goes_on_from_the_forward_pass():
    """A prompt's states are what a step takes: its next token is the forward
    pass's, within both bounds."""
    cu, H, Hq, K, V = [0, 90, 201], 4, 2, 128, 64
    x, g, h0, dev = _case(cu, H, Hq, Hq, H, K, V, "fp32", False, False, seed=8)
    q, k, v = dev
    g = _d(g)
    keep = torch.tensor([i for i in range(201) if i not in (89, 200)], device=DEV)
    short = layer.linear_forward(kda.Plan([0, 89, 199], 4), q[keep], k[keep], v[keep], g[keep])
    ends = torch.tensor([89, 200], device=DEV)
    pool = torch.zeros(5, H, K, V, device=DEV)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    pool[slots.long()] = short["final_state"]
    o = layer.linear_step(q[ends], k[ends], v[ends], g[ends], pool, slots, o_dtype=F32)
    out, size = ref.forward(*(_w(t) for t in x), g.cpu().double(), cu)
    bounds = ref.forward_bounds(size, cu, K, True)
    lr.assert_close(o, out["o"][[89, 200]], 2 * bounds["o"][[89, 200]], "o")
    lr.assert_close(pool[slots.long()], out["final_state"], 2 * bounds["final_state"], "state")


def test_plans_differ_by_rounding_only():
    """A sequence cut in another way, and any plan that the recurrence uses."""
    cu, H, K, V = [0, 600], 2, 128, 128
    x, g, h0, dev = _case(cu, H, H, H, H, K, V, "fp32", True, False, seed=9)
    out, size = ref.forward(*(_w(t) for t in x), _w(g), cu, _w(h0))
    bounds = ref.forward_bounds(size, cu, K, True)
    for plan in (kda.Plan(cu, 1), kda.Plan(cu, 600), kda.Plan(cu, 3, piece_tokens=32),
                 kda.Plan(cu, layer.linear_segments(cu, H))):
        got = layer.linear_forward(plan, *dev, _d(g), initial_state=_d(h0), o_dtype=F32)
        for n, t in out.items():
            lr.assert_close(got[n], t, bounds[n], n)


def test_given_buffers_streams_and_bits():
    cu, H = [0, 333, 1000], 2
    x, g, h0, dev = _case(cu, H, 1, 1, H, 128, 128, "head", True, True, seed=10)
    plan, g, h0, d_o = kda.Plan(cu, 7), _d(g), _d(h0), _d(_randn(1000, H, 128, seed=5, dtype=BF))
    want = layer.linear_forward(plan, *dev, g, initial_state=h0)
    back = layer.linear_backward(plan, *dev, g, d_o, initial_state=h0)
    out = {n: torch.empty_like(t) for n, t in want.items()}
    assert layer.linear_forward(plan, *dev, g, initial_state=h0, out=out) is out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer.linear_forward(plan, *dev, g, initial_state=h0, stream=side)
    again = layer.linear_backward(plan, *dev, g, d_o, initial_state=h0, stream=side)
    side.synchronize()
    for n, t in want.items():
        assert torch.equal(out[n], t) and torch.equal(got[n], t), n
    for n, t in back.items():
        assert torch.equal(again[n], t), n


def test_two_streams_at_once():
    """Each call has its own workspace: two that overlap in time change nothing."""
    cu, H = [0, 2000], 4
    plan, runs = kda.Plan(cu, 8), []
    for seed in (1, 2):
        x, g, h0, dev = _case(cu, H, H, H, H, 128, 128, "fp32", False, False, seed=seed)
        runs.append((dev, _d(g), _d(_randn(2000, H, 128, seed=seed + 20, dtype=BF))))
    want = [layer.linear_backward(plan, *dev, g, d_o) for dev, g, d_o in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for _ in range(3):
        for i, (dev, g, d_o) in enumerate(runs):
            got[i].append(layer.linear_backward(plan, *dev, g, d_o, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for n, t in want[i].items():
                assert t is None or torch.equal(r[n], t), n


def test_captured():
    """Both directions in a graph, replayed with other inputs and eager work between."""
    cu, H = [0, 100, 391], 2
    x, g, h0, dev = _case(cu, H, 1, 2, H, 64, 128, "fp32", True, False, seed=11)
    plan, g, h0, d_o = kda.Plan(cu, 3), _d(g), _d(h0), _d(_randn(391, H, 128, seed=5, dtype=BF))
    f = lambda: layer.linear_forward(plan, *dev, g, initial_state=h0)  # noqa: E731
    b = lambda: layer.linear_backward(plan, *dev, g, d_o, initial_state=h0)  # noqa: E731
    f(), b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, back = f(), b()
    for i in range(3):
        dev[2].copy_(_randn(391, H, 128, seed=60 + i, dtype=BF))
        g.mul_(0.9)
        graph.replay()
        torch.cuda.synchronize()
        want, wanted = f(), b()
        for a, c in ((got, want), (back, wanted)):
            for n in a:
                assert torch.equal(a[n], c[n]), (i, n)


def test_refusals():
    cu, H = [0, 10, 30], 4
    x, g, h0, (q, k, v) = _case(cu, H, 2, 2, H, 64, 64, "fp32", True, False, seed=12)
    plan, g, h0 = kda.Plan(cu, 2), _d(g), _d(h0)
    d_o = torch.zeros(30, H, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="plan"):
        layer.linear_forward(kda.Plan([0, 31], 1), q, k, v, g)
    with pytest.raises(TypeError, match="v"):
        layer.linear_forward(plan, q, k, v.float(), g)
    with pytest.raises(TypeError, match="g"):
        layer.linear_forward(plan, q, k, v, g.half())
    with pytest.raises(ValueError, match="k"):
        layer.linear_forward(plan, q, k[..., :32].contiguous(), v, g)
    with pytest.raises(ValueError, match="initial_state"):
        layer.linear_forward(plan, q, k, v, g, initial_state=h0[:1])
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        layer.linear_forward(plan, torch.cat([q, q[:, :1]], 1), k, v, g)
    with pytest.raises(kda.KdaError, match="UNSUPPORTED"):
        layer.linear_forward(plan, q, k, torch.zeros(30, H, 136, dtype=BF, device=DEV), g)
    wide = torch.zeros(30, 2 * 64 + 4, dtype=BF, device=DEV)
    with pytest.raises(kda.KdaError, match="MISALIGNED"):
        layer.linear_forward(plan, wide[:, :128].view(30, 2, 64), k, v, g)
    with pytest.raises(TypeError, match="d_o"):
        layer.linear_backward(plan, q, k, v, g, d_o.float())
    with pytest.raises(TypeError, match="grad_dtype"):
        layer.linear_backward(plan, q, k, v, g, d_o, grad_dtype=torch.float16)
    with pytest.raises(ValueError, match="d_final"):
        layer.linear_backward(plan, q, k, v, g, d_o, d_final=h0[:1])
