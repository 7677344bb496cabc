"""The operators around the recurrence at the edges of their domains, on the
GPU: gates that are not finite, rows of large values, saturated gates, and the
precision of their exponentials.  Each bound counts units of EPS = 2^-24, half
a step of FP32: an exponential is off by at most 4 (the hardware's 2^x is within
2, its correction adds a rounding), a reciprocal by 2, a product or sum by 1."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer
import layer_reference as lr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _uniform(lo, hi, *shape, seed):
    return lo + (hi - lo) * torch.rand(*shape, generator=torch.Generator().manual_seed(seed))


def _d(t):
    return None if t is None else t.to(DEV)


# ------------------------------------------------------------- gates that are not finite


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,dtype", [(72, F32), (13, BF), (2, F32), (1600, BF)])
def test_scan_keeps_sequences_apart_from_bad_gates(D, dtype, bad):
    """A gate that is not a number stays in its own sequence in both directions,
    at a sequence's first token, inside it and at its last; the others give the
    same bits as without it."""
    cu, T, N = [0, 100, 101, 400, 900, 905, 1300], 1300, 6
    x, dh = (_d(_randn(T, D, seed=s, dtype=dtype)) for s in (1, 2))
    g = _d((-0.01 * _randn(T, D, seed=3).abs()).to(dtype))
    h0, d_final = _d(_randn(N, D, seed=4)), _d(_randn(N, D, seed=5))
    plan = kda.Plan(cu, 1)

    def both(gates, h):
        f = layer.scan_forward(plan, x, gates, initial_state=h0, tied=True)
        b = layer.scan_backward(plan, x, gates, h if h is not None else f["h"], dh, d_final=d_final,
                                initial_state=h0, tied=True)
        return f, b

    f, b = both(g, None)
    for places in ((cu[1], cu[3]), (cu[3] + 250,), (cu[2] - 1, cu[4] - 1)):
        g2 = g.clone()
        g2[list(places)] = bad
        hit = {n for n in range(N) for t in places if cu[n] <= t < cu[n + 1]}
        f2, b2 = both(g2, f["h"])
        for n in sorted(set(range(N)) - hit):
            rows = slice(cu[n], cu[n + 1])
            assert torch.equal(f2["h"][rows], f["h"][rows]), (places, n)
            assert torch.equal(f2["final_state"][n], f["final_state"][n]), (places, n)
            assert all(torch.equal(b2[k][rows], b[k][rows]) for k in ("dx", "dg")), (places, n)
            assert torch.equal(b2["dh0"][n], b["dh0"][n]), (places, n)
        if bad != bad:
            assert all(f2["final_state"][n].isnan().all() and b2["dh0"][n].isnan().all() for n in hit)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_inputs_stay_as_they_were(dtype):
    """The scan's backward, called twice on one set of inputs, writes into none
    of them and gives the same bits; h, dh in FP32, as the recurrence keeps them."""
    cu, T, D, N = [0, 40, 300], 300, 70, 2
    x, g = _d(_randn(T, D, seed=1, dtype=dtype)), _d((-_randn(T, D, seed=2).abs()).to(dtype))
    h0, d_final, dh = _d(_randn(N, D, seed=3)), _d(_randn(N, D, seed=4)), _d(_randn(T, D, seed=5))
    plan = kda.Plan(cu, 1)
    h = layer.scan_forward(plan, x, g, initial_state=h0, h_dtype=F32)["h"]
    ins = [x, g, h, dh, d_final, h0]
    kept = [t.clone() for t in ins]
    runs = [layer.scan_backward(plan, x, g, h, dh, d_final=d_final, initial_state=h0) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(ins, kept))
    assert all(torch.equal(runs[0][n], runs[1][n]) for n in runs[0])
    args = (x.cpu().double(), g.cpu().double(), h.cpu().double(), cu, h0.cpu().double(), False, dh.cpu().double(),
            d_final.cpu().double())
    want, bounds = lr.scan_backward(*args), lr.scan_backward_bounds(*args)
    for n, t in runs[1].items():
        lr.assert_close(t, want[n], bounds[n], n)


# ------------------------------------------------------------- large values


@pytest.mark.parametrize("V", [128, 520, 1000, 2048, 8191, 8192])
@pytest.mark.parametrize("o_dtype", [F32, BF])
def test_output_norm_of_large_values(V, o_dtype):
    """Rows whose mean of squares is finite in FP32 (about 2.5e37) and whose sum
    of squares is not."""
    T, H = 3, 2
    x = dict(o=_randn(T, H, V, seed=V, dtype=o_dtype, scale=5e18), weight=1 + 0.5 * _randn(V, seed=1),
             gate=_randn(T, H, V, seed=2), res_scale=_randn(H, V, seed=3))
    residual, dy = _randn(T, H, V, seed=4), _randn(T, H, V, seed=5)
    dev, w = {n: _d(t) for n, t in x.items()}, {n: t.double() for n, t in x.items()}
    assert (w["o"] ** 2).mean(-1).max() < torch.finfo(F32).max
    got = layer.output_norm(**dev, activation="silu", residual=_d(residual))
    args = dict(**w, kind="silu", eps=1e-6)
    lr.assert_close(got, lr.output_norm(**args, residual=residual.double()),
                    lr.output_norm_bound(**args, residual=residual.double()), "y")
    grads = layer.output_norm_backward(_d(dy), **dev, activation="silu")
    want, bounds = lr.output_norm_backward(dy.double(), **args), lr.output_norm_backward_bounds(dy.double(), **args)
    for n, t in grads.items():
        lr.assert_close(t, want[n], bounds[n], n)


# ------------------------------------------------------------- saturated gates


def _both_signs(lo, hi, *shape, seed):
    z = _uniform(lo, hi, *shape, seed=seed)
    return torch.where(_randn(*shape, seed=seed + 1) < 0, -z, z)


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
def test_output_norm_backward_of_saturated_gates(kind):
    """The slope of a saturated gate keeps its relative precision: sigmoid(z)
    sigmoid(-z), not s (1 - s).  The norm's and the products' 64 EPS and 4 |z|
    of the exponential; silu's 1 + z sigmoid(-z) has no cancellation there."""
    T, H, V = 5, 2, 128
    z = _both_signs(8.0, 80.0, T, H, V, seed=1)
    o, dy, weight = _randn(T, H, V, seed=3), _randn(T, H, V, seed=4), 1 + 0.5 * _randn(V, seed=5)
    got = layer.output_norm_backward(_d(dy), _d(o), _d(weight), gate=_d(z), activation=kind)["d_gate"]
    zw, ow = z.double(), o.double()
    up, down = lr.sigmoid(zw), lr.sigmoid(-zw)
    slope = up * down if kind == "sigmoid" else up * (1 + zw * down)
    n = ow / torch.sqrt((ow * ow).mean(-1, keepdim=True) + 1e-6)
    want = dy.double() * weight.double() * n * slope
    lr.assert_close(got, want, lr.EPS * want.abs() * (64 + 4 * zw.abs()), "d_gate")


def test_prepare_backward_of_saturated_beta():
    """dbeta sigmoid(b) sigmoid(-b), 24 EPS and 4 |b| of the exponential."""
    T, H = 40, 8
    b, dbeta = _both_signs(8.0, 80.0, T, H, seed=1), _randn(T, H, seed=3)
    rows = _d(_randn(T, H, 128, seed=4))
    got = layer.prepare_inputs_backward(rows, rows, rows, _d(b), _d(torch.zeros(H)), None, rows, rows, rows, _d(dbeta))
    want = dbeta.double() * lr.sigmoid(b.double()) * lr.sigmoid(-b.double())
    lr.assert_close(got["dbeta_raw"], want, lr.EPS * want.abs() * (24 + 4 * b.double().abs()), "dbeta_raw")


# ------------------------------------------------------------- 1 - e^g on both sides of zero


@pytest.mark.parametrize("one_token", [False, True])
def test_tied_input_of_any_gate(one_token):
    """h = (1 - e^g) x from zero.  Near zero a series, 8 EPS of the value; else a
    difference, 4 EPS of e^g and |g| for its argument's rounding, and its own."""
    g = torch.cat([torch.linspace(-3, 3, 193), torch.tensor([0.0, -0.25, 0.25, 1e-6, -1e-6, 1e-30, -1e-30, 5.0])])
    x, D = torch.ones_like(g), g.numel()
    if one_token:
        got = layer.scan_step(_d(x[None]), _d(g[None]), torch.zeros(1, D, device=DEV), tied=True)
    else:
        got = layer.scan_forward(kda.Plan([0, 1], 1), _d(x[None]), _d(g[None]), tied=True)["h"]
    w = g.double()
    want = -torch.expm1(w)
    slack = torch.where(w.abs() < 0.25, 8 * want.abs(), 2 * want.abs() + torch.exp(w) * (4 + w.abs()))
    lr.assert_close(got[0], want, lr.EPS * slack, "h")


# ------------------------------------------------------------- precision of the exponentials


def test_prepare_backward_keeps_fp32_precision():
    """dgate = -dg e^a sigmoid(z): the rate 4 EPS, the sigmoid 10 (exponential 4,
    its weight in 1 + t 2, that sum 1, reciprocal 2, product 1), two products:
    16.  da: the softplus 16, rate and products 6, 128 terms in 8 + 4 additions
    and 2 of the partial sums: 36 of the terms' magnitudes."""
    T, H = 6, 5
    z, dg = _uniform(-80.0, 20.0, T, H, 128, seed=1), _randn(T, H, 128, seed=2)
    a_log = _uniform(-6.0, 6.0, H, seed=3)
    one = torch.ones(T, H, 128)
    got = layer.prepare_inputs_backward(_d(one), _d(one), _d(z), _d(torch.zeros(T, H)), _d(a_log), None, _d(one), _d(one),
                                        _d(dg), _d(torch.zeros(T, H)))
    rate, w = -torch.exp(a_log.double())[:, None], z.double()
    want = dg.double() * rate * lr.sigmoid(w)
    lr.assert_close(got["dgate_raw"], want, 16 * lr.EPS * want.abs(), "dgate_raw")
    terms = dg.double() * rate * lr.softplus(w)
    lr.assert_close(got["da_log"], terms.sum((0, 2)), 40 * lr.EPS * terms.abs().sum((0, 2)), "da_log")


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
def test_output_norm_keeps_fp32_precision(kind):
    """Rows of 8 channels, one lane's: 8 terms' additions and the mean's scaling
    give at most 10 EPS of the mean square, 5 of the root, 2 of the reciprocal
    root, 4 products, the gate's 10 and its product: 22."""
    T, H, V = 300, 2, 8
    z, o = _uniform(-80.0, 20.0, T, H, V, seed=1), _randn(T, H, V, seed=2)
    weight = 1 + 0.5 * _randn(V, seed=3)
    got = layer.output_norm(_d(o), _d(weight), gate=_d(z), activation=kind)
    args = dict(o=o.double(), weight=weight.double(), gate=z.double(), kind=kind, res_scale=None, residual=None, eps=1e-6)
    want = lr.output_norm(**args)
    lr.assert_close(got, want, 22 * lr.EPS * want.abs(), "y")


@pytest.mark.parametrize("D", [512, 3])
def test_decays_keep_fp32_precision(D):
    """One token from a state, no input: h = e^g h0, 4 EPS of the exponential, a
    product and a sum; the gradient dg = e^g dh h0 one product more."""
    N = 1024 if D == 3 else 64
    g, h0, dh = _uniform(-80.0, 0.0, N, D, seed=1), _randn(N, D, seed=2), _randn(N, D, seed=3)
    zero, plan = torch.zeros(N, D, device=DEV), kda.Plan(list(range(N + 1)), 1)
    a = torch.exp(g.double())
    want = a * h0.double()
    got = layer.scan_forward(plan, zero, _d(g), initial_state=_d(h0))
    for n in ("h", "final_state"):
        lr.assert_close(got[n], want, 6 * lr.EPS * want.abs(), n)
    pool = _d(h0).clone()
    lr.assert_close(layer.scan_step(zero, _d(g), pool), want, 6 * lr.EPS * want.abs(), "step h")
    lr.assert_close(pool, want, 6 * lr.EPS * want.abs(), "step state")
    back = layer.scan_backward(plan, None, _d(g), got["h"], _d(dh), initial_state=_d(h0))
    lr.assert_close(back["dg"], dh.double() * want, 8 * lr.EPS * (dh.double() * want).abs(), "dg")
    lr.assert_close(back["dh0"], dh.double() * a, 6 * lr.EPS * (dh.double() * a).abs(), "dh0")


def test_step_decay_keeps_fp32_precision():
    """kda_step with k = 0: S = Diag(e^g) S, 4 EPS and a product."""
    B, H = 6, 3
    g, state = _uniform(-80.0, 0.0, B, H, 128, seed=1).to(BF), _randn(B, H, 128, 128, seed=2)
    zero = torch.zeros(B, H, 128, dtype=BF, device=DEV)
    pool = _d(state).clone()
    layer.step(zero, zero, zero, _d(g), torch.zeros(B, H, dtype=BF, device=DEV), pool)
    want = torch.exp(g.double())[..., None] * state.double()
    lr.assert_close(pool, want, 6 * lr.EPS * want.abs(), "state")


# ------------------------------------------------------------- single tokens, slot by slot


@pytest.mark.parametrize("D,dtype,tied", [(8, BF, True), (13, F32, False), (300, F32, True)])
def test_scan_step_slot_by_slot(D, dtype, tied):
    """As many roundings as the element's own slot has tokens, of its own
    magnitudes: 24 EPS a token of |state| + sum |x|.  Unused rows count nowhere."""
    B, n = 300, 400
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32)
    slots[::17] = -1
    slots[5] = slots[B - 1]
    x, g = _randn(B, D, seed=1, dtype=dtype), (-_randn(B, D, seed=2).abs()).to(dtype)
    state, h0 = _randn(n, D, seed=3), torch.full((B, D), -7.0).to(dtype)
    pool = _d(state).clone()
    h = layer.scan_step(_d(x), _d(g), pool, _d(slots), h=_d(h0), tied=tied)
    want_h, want = lr.scan_step(x.double(), g.double(), state.double(), slots, h0.double(), tied)
    used = (slots >= 0) & (slots < n)
    tokens = torch.bincount(slots[used].long(), minlength=n).double()
    assert tokens.max() == 2
    mag = state.double().abs().index_add(0, slots[used].long(), x.double()[used].abs())
    slack = 24 * lr.EPS * tokens[:, None] * mag
    lr.assert_close(pool, want, slack, "state")
    row_slack = torch.zeros(B, D).double()
    row_slack[used] = slack[slots[used].long()]
    lr.assert_close(h, want_h, row_slack, "h")


# ------------------------------------------------------------- sequences and tiles


@pytest.mark.parametrize("D,dtype,h_dtype", [(70, F32, F32), (2, BF, F32), (1600, BF, BF)])
@pytest.mark.parametrize("cu,S", [
    ([0, 128], 1), ([0, 128, 256], 1), ([0, 127, 128, 129, 384], 1), ([0, 1, 256, 257], 2),   # at a tile's edge
    (list(range(0, 601)), 1), ([0, 5] + list(range(6, 700, 2)), 1),                          # more than 256 sequences
    ([0, 500, 3000], 300)])                                                                   # more than 256 segments
def test_scan_boundaries(cu, S, D, dtype, h_dtype):
    """Tokens that are whole tiles, sequences that begin where a tile does, and
    more fragments of the plan than a workgroup has threads."""
    T, N = cu[-1], len(cu) - 1
    at = slice(0, D) if D < 100 else torch.cat([torch.arange(0, 16), torch.arange(D - 16, D)])   # the channels looked at
    x, g = _randn(T, D, seed=1, dtype=dtype), (-0.05 * _randn(T, D, seed=2).abs()).to(dtype)
    h0, d_final, dh = _randn(N, D, seed=3), _randn(N, D, seed=4), _randn(T, D, seed=5, dtype=h_dtype)
    plan = kda.Plan(cu, S)
    got = layer.scan_forward(plan, _d(x), _d(g), initial_state=_d(h0), tied=True, h_dtype=h_dtype)
    w = [t[:, at].double() for t in (x, g)]
    want, final = lr.scan(*w, cu, h0[:, at].double(), True)
    eh, ef = lr.scan_bound(*w, cu, h0[:, at].double(), True)
    lr.assert_close(got["h"][:, at], want, eh, "h")
    lr.assert_close(got["final_state"][:, at], final, ef, "final_state")
    back = layer.scan_backward(plan, _d(x), _d(g), got["h"], _d(dh), d_final=_d(d_final), initial_state=_d(h0), tied=True)
    args = (*w, got["h"].cpu()[:, at].double(), cu, h0[:, at].double(), True, dh[:, at].double(), d_final[:, at].double())
    want, bounds = lr.scan_backward(*args), lr.scan_backward_bounds(*args)
    for n, t in back.items():
        lr.assert_close(t[:, at], want[n], bounds[n], n)
