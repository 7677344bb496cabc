"""The operators around the recurrence on the GPU against their 64-bit
reference, within the reference's bounds (layer_reference states the counts)."""
import itertools

import pytest
import torch

from gated_delta_rule_37_amd import kda, layer, synth
import layer_reference as lr

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
    """The parts' rows side by side in one tensor, as slices of it (16-byte
    aligned), on the device."""
    T = parts[0].shape[0]
    flat = [p.reshape(T, -1) for p in parts]
    pad = [torch.zeros(T, -f.shape[1] % 8, dtype=f.dtype) for f in flat]
    wide = torch.cat([x for pair in zip(flat, pad) for x in pair], 1).to(DEV)
    out, at = [], 0
    for p, f, z in zip(parts, flat, pad):
        out.append(wide[:, at:at + f.shape[1]].view(p.shape))
        at += f.shape[1] + z.shape[1]
    return out


# ------------------------------------------------------------- input preparation


def _prepare_inputs(T, H, dtype, bias, seed):
    raw = dict(q=_randn(T, H, 128, seed=seed, dtype=dtype), k=_randn(T, H, 128, seed=seed + 1, dtype=dtype, scale=30.0),
               gate=_randn(T, H, 128, seed=seed + 2, dtype=dtype, scale=4.0),
               beta=_randn(T, H, seed=seed + 3, dtype=dtype, scale=3.0))
    raw["q"][0, 0] = 0                      # a row of zeros
    raw["k"][-1, -1] = 1e-4                 # eps counts: the sum of squares is 1.28e-6
    raw["gate"][0, 0, :4] = torch.tensor([-60.0, 0.0, 60.0, 1e4])
    raw["beta"][0, 0] = -40.0
    return raw, _randn(H, seed=seed + 4), _randn(H, 128, seed=seed + 5) if bias else None


@pytest.mark.parametrize("T,H,dtype,bias,strided", [
    (1, 1, BF, True, False), (3, 5, BF, False, True), (37, 4, F32, True, True), (130, 16, BF, True, False),
    (1, 70, F32, False, False), (2500, 17, BF, True, True)])
def test_prepare_inputs(T, H, dtype, bias, strided):
    raw, a_log, dt_bias = _prepare_inputs(T, H, dtype, bias, seed=T + H)
    dev = _in_wider(list(raw.values())) if strided else [_d(t) for t in raw.values()]
    got = layer.prepare_inputs(*dev, _d(a_log), _d(dt_bias), q_scale=0.25, eps=1e-5)
    w = {n: t.double() for n, t in raw.items()}
    want = lr.prepare(**w, a_log=_w(a_log), dt_bias=_w(dt_bias), q_scale=0.25, eps=torch.tensor(1e-5, dtype=F32).double())
    bounds = lr.prepare_bounds(want, w["gate"], _w(a_log), _w(dt_bias))
    for n in ("q", "k", "g", "beta"):
        lr.assert_close(got[n], want[n], bounds[n], n)


@pytest.mark.parametrize("T,H,dtype,bias,strided", [
    (1, 1, BF, True, False), (3, 5, BF, False, True), (37, 4, F32, True, True), (130, 16, BF, True, False),
    (1, 70, F32, False, False), (2500, 17, BF, True, True)])
def test_prepare_inputs_backward(T, H, dtype, bias, strided):
    raw, a_log, dt_bias = _prepare_inputs(T, H, dtype, bias, seed=T + H)
    d = dict(dq=_randn(T, H, 128, seed=50), dk=_randn(T, H, 128, seed=51), dg=_randn(T, H, 128, seed=52),
             dbeta=_randn(T, H, seed=53))
    dev = _in_wider(list(raw.values())) if strided else [_d(t) for t in raw.values()]
    got = layer.prepare_inputs_backward(*dev, _d(a_log), _d(dt_bias), **{n: _d(t) for n, t in d.items()}, q_scale=0.25,
                                        eps=1e-5)
    args = dict(**{n: t.double() for n, t in raw.items()}, a_log=_w(a_log), dt_bias=_w(dt_bias), q_scale=0.25,
                eps=torch.tensor(1e-5, dtype=F32).double(), **{n: t.double() for n, t in d.items()})
    want, bounds = lr.prepare_backward(**args), lr.prepare_backward_bounds(**args)
    assert (got["ddt_bias"] is None) == (not bias)
    for n, t in got.items():
        if t is not None:
            lr.assert_close(t, want[n], bounds[n], n)


# ------------------------------------------------------------- output norm

NORM_SHAPES = [(1, 1, 128), (37, 5, 128), (9, 3, 40), (5, 2, 1), (4, 3, 7), (3, 1, 512), (3, 2, 513), (2, 1, 1000),
               (3, 1, 2048), (2, 1, 2049), (2, 1, 2056), (2, 1, 4104), (2, 1, 8192), (1, 1, 8191), (1300, 17, 128),
               (700, 1, 264), (5, 3, 129), (4, 1, 200), (900, 1, 256), (3, 1, 1024), (2, 1, 1025), (2, 1, 4096), (2, 1, 4097),
               (1100, 1, 777), (2, 2, 9)]


def _norm_case(T, H, V, o_dtype, dtype, kind, scaled, strided, seed):
    x = dict(o=_randn(T, H, V, seed=seed, dtype=o_dtype), weight=1 + 0.5 * _randn(V, seed=seed + 1),
             gate=None if kind == "none" else _randn(T, H, V, seed=seed + 2, dtype=dtype, scale=3.0),
             res_scale=_randn(H, V, seed=seed + 3) if scaled else None)
    x["o"][0, 0] = 0                         # a row of zeros
    if T * H > 1:
        x["o"][-1, -1] *= 1e-4               # eps counts
    dev = {n: _d(t) for n, t in x.items()}
    if strided and x["gate"] is not None:
        dev["gate"] = _in_wider([_randn(T, H, V, seed=1, dtype=dtype), x["gate"]])[1]
    return x, dev


def _norm_cases():
    kinds = itertools.cycle(["sigmoid", "silu", "none"])
    types = itertools.cycle([(F32, BF), (BF, BF), (F32, F32), (BF, F32)])
    for i, shape in enumerate(NORM_SHAPES):
        o, e = next(types)
        yield (*shape, o, e, next(kinds), i % 2 == 0, i % 3 == 1)
    for o, e in [(F32, BF), (BF, BF), (F32, F32), (BF, F32)]:
        for kind in ("sigmoid", "silu", "none"):
            yield (11, 3, 128, o, e, kind, kind != "none", o == BF)


@pytest.mark.parametrize("T,H,V,o_dtype,dtype,kind,scaled,strided", _norm_cases())
def test_output_norm(T, H, V, o_dtype, dtype, kind, scaled, strided):
    x, dev = _norm_case(T, H, V, o_dtype, dtype, kind, scaled, strided, seed=V)
    residual = _randn(T, H, V, seed=9, dtype=dtype) if scaled else None
    got = layer.output_norm(dev["o"], dev["weight"], gate=dev["gate"], activation=kind, res_scale=dev["res_scale"],
                            residual=_d(residual), eps=1e-5, dtype=dtype)
    args = dict(**{n: _w(t) for n, t in x.items()}, kind=kind, residual=_w(residual),
                eps=torch.tensor(1e-5, dtype=F32).double())
    lr.assert_close(got, lr.output_norm(**args), lr.output_norm_bound(**args), "y")
    if residual is not None:     # in place
        buf = _d(residual).clone()
        layer.output_norm(dev["o"], dev["weight"], gate=dev["gate"], activation=kind, res_scale=dev["res_scale"],
                          residual=buf, eps=1e-5, out=buf)
        assert torch.equal(buf, got)


@pytest.mark.parametrize("T,H,V,o_dtype,dtype,kind,scaled,strided", _norm_cases())
def test_output_norm_backward(T, H, V, o_dtype, dtype, kind, scaled, strided):
    x, dev = _norm_case(T, H, V, o_dtype, dtype, kind, scaled, strided, seed=V)
    dy = _randn(T, H, V, seed=8, dtype=dtype)
    args = dict(dy=dy.double(), **{n: _w(t) for n, t in x.items()}, kind=kind,
                eps=torch.tensor(1e-5, dtype=F32).double())
    want, bounds = lr.output_norm_backward(**args), lr.output_norm_backward_bounds(**args)
    for d_o_dtype in (F32, BF):
        got = layer.output_norm_backward(_d(dy), dev["o"], dev["weight"], gate=dev["gate"], activation=kind,
                                         res_scale=dev["res_scale"], eps=1e-5, d_o_dtype=d_o_dtype)
        assert got["d_o"].dtype == d_o_dtype
        for n, t in got.items():
            assert (t is None) == (want[n] is None), n
            if t is not None:
                lr.assert_close(t, want[n], bounds[n], n)


@pytest.mark.parametrize("V", [8, 128, 250, 512, 1000, 2048, 4104])
def test_output_norm_backward_infinite_scale(V):
    """An infinite residual scale reaches its own channel's sums alone, and as
    the formula has it: lanes without a row add nothing, not 0 inf."""
    T, H = 5, 3
    o, dy = _randn(T, H, V, seed=1).abs() + 0.5, _randn(T, H, V, seed=2).abs() + 0.5
    weight, s = torch.ones(V), torch.ones(H, V)
    s[0, 3] = float("inf")
    got = layer.output_norm_backward(_d(dy), _d(o), _d(weight), res_scale=_d(s), activation="none")
    d_weight, d_scale = got["d_weight"].cpu(), got["d_res_scale"].cpu()
    others = torch.arange(V) != 3
    assert d_weight[3] == float("inf")
    assert d_weight[others].isfinite().all() and d_scale.isfinite().all()
    assert got["d_o"].cpu()[:, 1:].isfinite().all()


# ------------------------------------------------------------- per-channel scan

# cu_seqlens, segments, channels, dtype, h's dtype, tied, initial states, strided
SCANS = [
    ([0, 1], 1, 1, F32, F32, False, False, False),
    ([0, 1], 1, 8, BF, BF, True, True, False),
    ([0, 2, 3, 64], 1, 24, BF, F32, True, True, True),
    ([0, 700], 1, 16, F32, F32, False, True, False),
    ([0, 700], 5, 16, F32, F32, True, True, False),
    ([0, 100, 101, 102, 900], 7, 40, BF, BF, False, True, True),
    ([0, 1, 2, 3, 4, 5], 3, 13, BF, F32, True, False, True),
    ([0, 511, 1030, 1543], 4, 9, F32, BF, True, True, False),
    ([0, 3000], 1, 3, F32, F32, False, False, True),
    ([0, 2999, 3001], 40, 264, BF, F32, False, True, False),
    (list(range(0, 600, 7)) + [600], 1, 72, BF, BF, True, True, False),
]


def _scan_case(cu, D, dtype, tied, init, strided, seed, slow=False):
    T, N = cu[-1], len(cu) - 1
    x = _randn(T, D, seed=seed, dtype=dtype)
    rate = 0.01 if slow else 1.0
    g = (-torch.nn.functional.softplus(_randn(T, D, seed=seed + 1)) * rate)
    # a channel that never forgets, one that is reset now and then, one whose decay underflows
    g[:, 0] = 0.0
    if D > 2:
        g[::5, 1] = float("-inf")
        g[:, 2] = -200.0
    g = g.to(dtype)
    h0 = _randn(N, D, seed=seed + 2) if init else None
    if strided:
        dev = _in_wider([x, g])
    else:
        dev = [_d(x), _d(g)]
    return x, g, h0, dev


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("cu,S,D,dtype,h_dtype,tied,init,strided", SCANS)
def test_scan_forward(cu, S, D, dtype, h_dtype, tied, init, strided, slow):
    x, g, h0, dev = _scan_case(cu, D, dtype, tied, init, strided, seed=D, slow=slow)
    got = layer.scan_forward(kda.Plan(cu, S), *dev, initial_state=_d(h0), tied=tied, h_dtype=h_dtype)
    h, final = lr.scan(x.double(), g.double(), cu, _w(h0), tied)
    eh, ef = lr.scan_bound(x.double(), g.double(), cu, _w(h0), tied)
    lr.assert_close(got["h"], h, eh, "h")
    lr.assert_close(got["final_state"], final, ef, "final_state")


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("cu,S,D,dtype,h_dtype,tied,init,strided", SCANS)
def test_scan_backward(cu, S, D, dtype, h_dtype, tied, init, strided, slow):
    x, g, h0, dev = _scan_case(cu, D, dtype, tied, init, strided, seed=D, slow=slow)
    T, N = cu[-1], len(cu) - 1
    h = lr.scan(x.double(), g.double(), cu, _w(h0), tied)[0].to(h_dtype)
    dh = _randn(T, D, seed=60, dtype=h_dtype)
    d_final = _randn(N, D, seed=61) if init else None
    got = layer.scan_backward(kda.Plan(cu, S), *dev, _d(h), _d(dh), d_final=_d(d_final), initial_state=_d(h0),
                              tied=tied, want_dh0=True)
    args = (x.double(), g.double(), h.double(), cu, _w(h0), tied, dh.double(), _w(d_final))
    want, bounds = lr.scan_backward(*args), lr.scan_backward_bounds(*args)
    for n, t in got.items():
        lr.assert_close(t, want[n], bounds[n], n)
    without = layer.scan_backward(kda.Plan(cu, S), dev[0] if tied else None, dev[1], _d(h), _d(dh),
                                  d_final=_d(d_final), initial_state=_d(h0), tied=tied, want_dh0=False)
    assert without["dh0"] is None
    assert torch.equal(without["dx"], got["dx"]) and torch.equal(without["dg"], got["dg"])


def test_scan_of_pieces_and_repeats():
    """A plan with pieces works too, and every run gives the same bits."""
    cu, D = [0, 300, 1000], 24
    x, g, h0, dev = _scan_case(cu, D, BF, True, True, False, seed=3, slow=True)
    plan = kda.Plan(cu, 2, None, 64)
    assert plan.F > 2
    h, final = lr.scan(x.double(), g.double(), cu, _w(h0), True)
    eh, ef = lr.scan_bound(x.double(), g.double(), cu, _w(h0), True)
    runs = [layer.scan_forward(plan, *dev, initial_state=_d(h0), tied=True) for _ in range(3)]
    lr.assert_close(runs[0]["h"], h, eh, "h")
    lr.assert_close(runs[0]["final_state"], final, ef, "final_state")
    for r in runs[1:]:
        assert torch.equal(r["h"], runs[0]["h"]) and torch.equal(r["final_state"], runs[0]["final_state"])


def test_scan_repeats_of_many_tiles():
    """The same bits on every run, however the tiles' workgroups race."""
    cu, D = [0, 9000, 20011], 200
    x, g, h0, dev = _scan_case(cu, D, BF, False, True, False, seed=13, slow=True)
    plan, dh = kda.Plan(cu, 1), _d(_randn(cu[-1], D, seed=14))
    f = [layer.scan_forward(plan, *dev, initial_state=_d(h0), h_dtype=F32) for _ in range(6)]
    b = [layer.scan_backward(plan, *dev, f[0]["h"], dh, initial_state=_d(h0)) for _ in range(6)]
    for runs in (f, b):
        for r in runs[1:]:
            assert all(torch.equal(r[n], runs[0][n]) for n in r)


@pytest.mark.parametrize("D,dtype", [(72, F32), (13, BF)])
def test_scan_keeps_sequences_apart(D, dtype):
    """An infinity or NaN in one sequence does not reach the others, wherever
    the boundaries lie, in either direction."""
    cu = [0, 100, 101, 400, 900, 905, 1300]
    x, g, h0, dev = _scan_case(cu, D, dtype, True, True, False, seed=9, slow=True)
    g[:, 1:3] = g[:, 3:5]                    # finite everywhere
    dev[1] = _d(g)
    plan = kda.Plan(cu, 3)
    dh, d_final = _d(_randn(1300, D, seed=70, dtype=dtype)), _d(_randn(6, D, seed=71))
    ref = layer.scan_forward(plan, *dev, initial_state=_d(h0), tied=True)
    back = layer.scan_backward(plan, *dev, ref["h"], dh, d_final=d_final, initial_state=_d(h0), tied=True)
    for bad in (float("nan"), float("inf")):
        x2, dh2 = dev[0].clone(), dh.clone()
        for n in (1, 3):
            x2[cu[n + 1] - 1], dh2[cu[n]] = bad, bad
        got = layer.scan_forward(plan, x2, dev[1], initial_state=_d(h0), tied=True)
        grads = layer.scan_backward(plan, dev[0], dev[1], ref["h"], dh2, d_final=d_final, initial_state=_d(h0), tied=True)
        for n in (0, 2, 4, 5):
            rows = slice(cu[n], cu[n + 1])
            assert torch.equal(got["h"][rows], ref["h"][rows]) and torch.equal(got["final_state"][n], ref["final_state"][n])
            assert all(torch.equal(grads[k][rows], back[k][rows]) for k in ("dx", "dg"))
            assert torch.equal(grads["dh0"][n], back["dh0"][n])
        assert not torch.isfinite(got["final_state"][[1, 3]]).any()
        assert not torch.isfinite(grads["dh0"][[1, 3]]).any()


# ------------------------------------------------------------- single tokens

SLOTS = [
    (1, 1, None), (3, 5, None), (4, 4, [2, 0, 3, 1]), (5, 6, [5, -1, 0, 6, 2]),
    (6, 3, [1, 1, 2, 1, -7, 2]),                       # several tokens of one sequence
    (300, 400, "many"), (9, 2, [0, 0, 0, 0, 0, 0, 0, 0, 0]), (2, 3, [7, -1]),
]


def _slots(B, n, slots):
    if slots == "many":
        perm = torch.randperm(n, generator=torch.Generator().manual_seed(B))[:B]
        perm[::17] = -1
        perm[5] = perm[B - 1]                          # far apart rows of one slot
        return perm.to(torch.int32)
    return None if slots is None else torch.tensor(slots, dtype=torch.int32)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,n,slots", SLOTS)
@pytest.mark.parametrize("D,dtype,tied", [(8, BF, True), (13, F32, False), (2056, BF, False), (300, F32, True)])
def test_scan_step(B, n, slots, D, dtype, tied, in_place):
    slots = _slots(B, n, slots)
    x, g = _randn(B, D, seed=1, dtype=dtype), (-_randn(B, D, seed=2).abs()).to(dtype)
    g[0, 0] = float("-inf")
    state, h0 = _randn(n, D, seed=3), torch.full((B, D), -7.0).to(dtype)
    pool, h = _d(state).clone(), _d(h0).clone()
    out = pool if in_place else torch.full((n, D), -9.0, device=DEV)
    got = layer.scan_step(_d(x), _d(g), pool, _d(slots), state_out=None if in_place else out, h=h, tied=tied)
    assert got is h
    want_h, want = lr.scan_step(x.double(), g.double(), state.double(), slots, h0.double(), tied)
    used = {b if slots is None else int(slots[b]) for b in range(B)} & set(range(n))
    if not in_place:
        assert torch.equal(pool, _d(state))
        for i in set(range(n)) - used:
            want[i] = -9.0
    # up to B tokens of one slot, each with a decay, its product and an addition
    tokens = 1 if slots is None else int(torch.bincount(slots.clamp(min=0).long()).max())
    mag = state.abs().amax().double() + tokens * x.double().abs().amax()
    lr.assert_close(h, want_h, 24 * tokens * lr.EPS * mag, "h")
    lr.assert_close(out, want, 24 * tokens * lr.EPS * mag, "state")
    for i in set(range(n)) - used:
        assert torch.equal(out[i].cpu(), state[i] if in_place else torch.full((D,), -9.0))


def _step_inputs(B, H, seed, slow=False):
    x = synth.make_inputs(B, H, 128, 128, seed=seed, gate_scale=0.05 if slow else 1.0)
    return {n: x[n] for n in ("q", "k", "v", "g", "beta")}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,n,slots", [s for s in SLOTS if s[0] < 300] + [(40, 41, "many")])
@pytest.mark.parametrize("H,o_dtype,floor,heads", [(1, F32, None, None), (3, BF, -1.5, (1, 2))])
def test_step(B, n, slots, H, o_dtype, floor, heads, in_place):
    slots = _slots(B, n, slots)
    x = _step_inputs(B, H, seed=B, slow=True)
    x["g"][0, 0, 0] = float("-inf")
    state, o0 = _randn(n, H, 128, 128, seed=4), torch.full((B, H, 128), -7.0).to(o_dtype)
    pool, o = _d(state).clone(), _d(o0).clone()
    out = pool if in_place else torch.full((n, H, 128, 128), -9.0, device=DEV)
    got = layer.step(*(_d(t) for t in x.values()), pool, _d(slots), state_out=None if in_place else out, o=o,
                     gate_lower_bound=floor, heads=heads)
    assert got is o
    want_o, want, eo, ep = lr.step(*(t.double() for t in x.values()), state.double(), slots, o0.double(), floor=floor)
    run = slice(None) if heads is None else slice(heads[0], heads[0] + heads[1])
    lr.assert_close(o[:, run], want_o[:, run], eo[:, run], "o")
    used = sorted({b if slots is None else int(slots[b]) for b in range(B)} & set(range(n)))
    rest = sorted(set(range(n)) - set(used))
    lr.assert_close(out[used][:, run], want[used][:, run], ep[used][:, run], "state")
    untouched = state if in_place else torch.full_like(state, -9.0)
    assert torch.equal(out[rest].cpu(), untouched[rest])
    if heads is not None:
        assert torch.equal(out[:, :1].cpu(), untouched[:, :1])
        assert torch.equal(o[:, :1].cpu(), o0[:, :1])


def test_steps_continue_a_forward():
    """Tokens one by one from kda.forward's final states give what the forward
    gives over all of them (within its own stated tolerance)."""
    H, cu = 2, [0, 50, 90]
    x = {n: t.to(DEV) for n, t in synth.make_inputs(90, H, 128, 128, seed=5, cu_seqlens=cu, gate_scale=0.05).items()
         if n != "cu_seqlens"}
    whole = kda.forward(kda.Plan(cu, 1), *(x[n] for n in ("q", "k", "v", "g", "beta")))
    keep = [t for n in range(2) for t in range(cu[n], cu[n + 1] - 10)]
    first = {n: t[keep].contiguous() for n, t in x.items()}
    state = kda.forward(kda.Plan([0, 40, 70], 1), *(first[n] for n in ("q", "k", "v", "g", "beta")))["final_state"]
    slots = torch.tensor([1, 0], dtype=torch.int32, device=DEV)      # row 0 is sequence 1
    for i in range(10):
        at = [cu[2] - 10 + i, cu[1] - 10 + i]
        o = layer.step(*(x[n][at].contiguous() for n in ("q", "k", "v", "g", "beta")), state, slots)
        assert (o - whole["o"][at]).abs().max() <= 2e-3
    for n in range(2):
        ref = whole["final_state"][n]
        assert (state[n] - ref).abs().max() <= 1e-4 * ref.abs().max()


# ------------------------------------------------------------- beyond 32 bits


def test_step_in_a_long_pool():
    """A pool of more than 2^31 elements: the last slots' addresses need 64 bits."""
    H, n = 32, 4200                          # 2.2e9 elements, 8.8 GB
    state = torch.empty(n, H, 128, 128, device=DEV)
    slots = torch.tensor([n - 1, 0, n - 2, n], dtype=torch.int32)
    x = _step_inputs(4, H, seed=3, slow=True)
    init = _randn(3, H, 128, 128, seed=4)
    for i, at in enumerate((n - 1, 0, n - 2)):
        state[at] = _d(init[i])
    o = layer.step(*(_d(t) for t in x.values()), state, _d(slots))
    want_o, want, eo, ep = lr.step(*(t.double() for t in x.values()), init.double(), torch.tensor([0, 1, 2, 3]),
                                   torch.zeros(4, H, 128).double())
    lr.assert_close(o[:3], want_o[:3], eo[:3], "o")
    lr.assert_close(state[[n - 1, 0, n - 2]], want, ep, "state")


def test_scan_of_many_elements():
    """More than 2^31 elements of x, g and h: the last sequence's rows."""
    T, D, last = (1 << 20) + 300, 2056, 300
    cu = [0, 1 << 20, T]
    x = torch.zeros(T, D, dtype=BF, device=DEV)
    g = torch.zeros(T, D, dtype=BF, device=DEV)
    xl, gl, h0l, _ = _scan_case([0, last], D, BF, True, True, False, seed=6, slow=True)
    x[-last:], g[-last:] = _d(xl), _d(gl)
    x[0] = 1.0                               # the first sequence carries it to its end: g = 0
    h0 = torch.zeros(2, D, device=DEV)
    h0[1] = _d(h0l[0])
    got = layer.scan_forward(kda.Plan(cu, 1), x, g, initial_state=h0)
    h, final = lr.scan(xl.double(), gl.double(), [0, last], _w(h0l), False)
    eh, ef = lr.scan_bound(xl.double(), gl.double(), [0, last], _w(h0l), False)
    lr.assert_close(got["h"][-last:], h, eh, "h")
    lr.assert_close(got["final_state"][1:], final, ef, "final_state")
    assert (got["final_state"][0] == 1).all() and (got["h"][(1 << 20) - 1] == 1).all()
    back = layer.scan_backward(kda.Plan(cu, 1), None, g, got["h"], x, initial_state=h0)
    args = (xl.double(), gl.double(), got["h"][-last:].cpu().double(), [0, last], _w(h0l), False, xl.double(), None)
    want, bounds = lr.scan_backward(*args), lr.scan_backward_bounds(*args)
    for n in ("dx", "dg"):
        lr.assert_close(back[n][-last:], want[n], bounds[n], n)
    lr.assert_close(back["dh0"][1:], want["dh0"], bounds["dh0"], "dh0")
    assert (back["dx"][0] == 1).all() and (back["dh0"][0] == 1).all()


def test_rows_beyond_32_bits():
    """The row-wise operators behind 2^31 elements of one tensor."""
    T, H = 270000, 64                        # 2.2e9 elements of 128-channel heads
    tail = 5
    z = torch.zeros(T, H, 128, dtype=BF, device=DEV)
    zl, b = _randn(tail, H, 128, seed=1, dtype=BF), torch.zeros(T, H, dtype=BF, device=DEV)
    z[-tail:] = _d(zl)
    a_log = torch.zeros(H, device=DEV)
    got = layer.prepare_inputs(z, z, z, b, a_log)
    w = zl.double()
    zero = torch.zeros(tail, H).double()
    want = lr.prepare(w, w, w, zero, torch.zeros(H).double(), None, 1.0, 1e-6)
    bounds = lr.prepare_bounds(want, w, torch.zeros(H).double(), None)
    for n in ("q", "k", "g"):
        lr.assert_close(got[n][-tail:], want[n], bounds[n] + 1e-6 * want[n].abs(), n)
    del got
    weight = torch.ones(128, device=DEV)
    y = layer.output_norm(z, weight, gate=z, residual=z)
    args = dict(o=w, weight=torch.ones(128).double(), gate=w, kind="sigmoid", res_scale=None, residual=w, eps=1e-6)
    lr.assert_close(y[-tail:], lr.output_norm(**args), lr.output_norm_bound(**args), "y")


@pytest.mark.parametrize("D", [1472, 1536, 1540, 8192])
def test_scan_widths(D):
    """Both sides of the window's and the cached accesses' rules (8192 channels
    of 8192 tokens are past the caches)."""
    cu = [0, 100, 8192 if D == 8192 else 700]
    x, g, h0, dev = _scan_case(cu, 64, BF, True, True, False, seed=D, slow=True)
    T = cu[-1]
    dx, dg_, dh0 = (torch.zeros(*s, D, dtype=t, device=DEV) for s, t in (((T,), BF), ((T,), BF), ((2,), F32)))
    at = torch.cat([torch.arange(0, 32), torch.arange(D - 32, D)])     # the first and last channels carry the case
    dx[:, at], dg_[:, at], dh0[:, at] = dev[0], dev[1], _d(h0)
    got = layer.scan_forward(kda.Plan(cu, 1), dx, dg_, initial_state=dh0, tied=True, h_dtype=F32)
    h, final = lr.scan(x.double(), g.double(), cu, _w(h0), True)
    eh, ef = lr.scan_bound(x.double(), g.double(), cu, _w(h0), True)
    lr.assert_close(got["h"][:, at], h, eh, "h")
    lr.assert_close(got["final_state"][:, at], final, ef, "final_state")
    assert not got["h"][:, 32:D - 32].any()
    dh = torch.zeros(T, D, device=DEV)
    part = _randn(T, 64, seed=2)
    dh[:, at] = _d(part)
    back = layer.scan_backward(kda.Plan(cu, 1), dx, dg_, got["h"], dh, initial_state=dh0, tied=True)
    args = (x.double(), g.double(), got["h"][:, at].cpu().double(), cu, _w(h0), True, part.double(), None)
    want, bounds = lr.scan_backward(*args), lr.scan_backward_bounds(*args)
    for n in ("dx", "dg", "dh0"):
        lr.assert_close(back[n][:, at], want[n], bounds[n], n)


# ------------------------------------------------------------- together


def _layer_inputs(T, H, seed):
    raw, a_log, dt_bias = _prepare_inputs(T, H, BF, True, seed)
    raw["gate"] = _randn(T, H, 128, seed=seed + 9, dtype=BF)
    raw["q"][0, 0] = 1.0     # no division of zero by zero in the plain gradient
    a_log = 0.3 * a_log - 2.0
    more = dict(v=_randn(T, H, 128, seed=seed + 10, dtype=BF), z=_randn(T, H, 128, seed=seed + 11, dtype=BF),
                weight=1 + 0.1 * _randn(128, seed=seed + 12), residual=_randn(T, H, 128, seed=seed + 13, dtype=BF),
                res_scale=0.5 + 0.1 * _randn(H, 128, seed=seed + 14))
    return raw, a_log, dt_bias, more


def _layer_run(plan, raw, a_log, dt_bias, m, dy):
    x = layer.prepare_inputs(*raw.values(), a_log, dt_bias)
    f = kda.forward(plan, x["q"], x["k"], m["v"], x["g"], x["beta"])
    y = layer.output_norm(f["o"], m["weight"], gate=m["z"], res_scale=m["res_scale"], residual=m["residual"])
    n = layer.output_norm_backward(dy, f["o"], m["weight"], gate=m["z"], res_scale=m["res_scale"])
    b = kda.backward(plan, x["q"], x["k"], m["v"], x["g"], x["beta"], n["d_o"])
    r = layer.prepare_inputs_backward(*raw.values(), a_log, dt_bias, b["dq"], b["dk"], b["dg"], b["dbeta"])
    return dict(y=y, dv=b["dv"], **{"d_" + k if not k.startswith("d") else k: t for k, t in {**n, **r}.items()})


def test_layer_training_step():
    """One layer forward and backward against automatic differentiation of its
    formulas in 64 bits.  The plain run has no BF16 rounding of q, k, g, beta
    between the operators; each is off by half a step, 2^-8 relative, so the
    results agree to a few 2^-8 of their norm."""
    T, H, cu = 70, 2, [0, 25, 70]
    raw, a_log, dt_bias, m = _layer_inputs(T, H, seed=21)
    dy = _randn(T, H, 128, seed=77, dtype=BF)
    dev = {n: _d(t) for n, t in raw.items()}
    got = _layer_run(kda.Plan(cu, 2), dev, _d(a_log), _d(dt_bias), {n: _d(t) for n, t in m.items()}, _d(dy))
    w = {n: t.double().requires_grad_() for n, t in {**raw, **m, "a_log": a_log, "dt_bias": dt_bias}.items()}
    x = lr.prepare(w["q"], w["k"], w["gate"], w["beta"], w["a_log"], w["dt_bias"], 1.0, 1e-6)
    rows = []
    for n in range(2):
        S = torch.zeros(H, 128, 128, dtype=torch.float64)
        for t in range(cu[n], cu[n + 1]):
            S = torch.exp(x["g"][t])[:, :, None] * S
            u = x["beta"][t][:, None] * (w["v"][t] - (S * x["k"][t][:, :, None]).sum(1))
            S = S + x["k"][t][:, :, None] * u[:, None, :]
            rows.append((S * x["q"][t][:, :, None]).sum(1))
    y = lr.output_norm(torch.stack(rows), w["weight"], w["z"], "sigmoid", w["res_scale"], w["residual"], 1e-6)
    y.backward(dy.double())
    want = dict(y=y.detach(), dv=w["v"].grad, dq_raw=w["q"].grad, dk_raw=w["k"].grad, dgate_raw=w["gate"].grad,
                dbeta_raw=w["beta"].grad, da_log=w["a_log"].grad, ddt_bias=w["dt_bias"].grad, d_gate=w["z"].grad,
                d_weight=w["weight"].grad, d_res_scale=w["res_scale"].grad)
    for n, t in want.items():
        off = (got[n].cpu().double() - t).norm() / t.norm()
        assert off <= 8 * 2.0 ** -8, (n, float(off))


def _replay(fn, outputs, alter):
    """Capture fn, replay it several times with other inputs (``alter(i)``
    changes them in place) and eager work between; every replay must give the
    eager result."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    for i in range(4):
        alter(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outputs()]
        alter(i)
        fn()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got, outputs())):
            assert torch.equal(a, b), (i, j)


def test_capture_decode():
    """A decoding step in a graph: it follows the slots and inputs of each replay."""
    B, H, n = 6, 3, 9
    raw, a_log, dt_bias, m = _layer_inputs(B, H, seed=31)
    raw, m = {k: _d(t) for k, t in raw.items()}, {k: _d(t) for k, t in m.items()}
    a_log, dt_bias = _d(a_log), _d(dt_bias)
    start = _d(_randn(n, H, 128, 128, seed=5))
    state, slots = start.clone(), torch.zeros(B, dtype=torch.int32, device=DEV)
    o = torch.zeros(B, H, 128, device=DEV)
    y = torch.zeros(B, H, 128, dtype=BF, device=DEV)
    sx, sg = (_d(_randn(B, 40, seed=s)) for s in (1, 2))
    pool0 = _d(_randn(n, 40, seed=3))
    pool, sh = pool0.clone(), torch.zeros(B, 40, device=DEV)

    def fn():
        x = layer.prepare_inputs(*raw.values(), a_log, dt_bias)
        layer.step(x["q"], x["k"], m["v"], x["g"], x["beta"], state, slots, o=o)
        layer.output_norm(o, m["weight"], gate=m["z"], out=y)
        layer.scan_step(sx, sg, pool, slots, h=sh, tied=True)

    def alter(i):
        state.copy_(start)
        pool.copy_(pool0)
        o.zero_()
        sh.zero_()
        slots.copy_(torch.tensor([[0, 1, 2, 3, 4, 5], [8, -1, 8, 0, 3, 8], [5, 5, 5, 5, 5, 5], [-1, 9, 1, 0, 7, 2]][i],
                                 dtype=torch.int32))
        raw["q"].copy_(_randn(B, H, 128, seed=i, dtype=BF))
        sg.copy_(-_randn(B, 40, seed=i).abs())

    _replay(fn, lambda: [state, o, y, pool, sh], alter)


@pytest.mark.parametrize("S", [1, 4])
def test_capture_training(S):
    T, H, cu = 130, 2, [0, 60, 130]
    raw, a_log, dt_bias, m = _layer_inputs(T, H, seed=41)
    raw, m = {k: _d(t) for k, t in raw.items()}, {k: _d(t) for k, t in m.items()}
    a_log, dt_bias, dy = _d(a_log), _d(dt_bias), _d(_randn(T, H, 128, seed=1, dtype=BF))
    plan, plan4 = kda.Plan(cu, 2), kda.Plan(cu, S)
    sx, sg, h0 = _d(_randn(T, 24, seed=2)), _d(-_randn(T, 24, seed=3).abs()), _d(_randn(2, 24, seed=4))
    kept = {}

    def fn():
        kept["layer"] = _layer_run(plan, raw, a_log, dt_bias, m, dy)
        f = layer.scan_forward(plan4, sx, sg, initial_state=h0, tied=True)
        kept["scan"] = {**f, **layer.scan_backward(plan4, sx, sg, f["h"], sx, d_final=h0, initial_state=h0, tied=True)}

    plan.device_blob(DEV), plan4.device_blob(DEV)
    graph_out = {}

    def outputs():
        return [t for k in ("layer", "scan") for t in kept[k].values()]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    graph_out = outputs()
    for i in range(4):
        raw["gate"].copy_(_randn(T, H, 128, seed=i, dtype=BF))
        sg.copy_(-_randn(T, 24, seed=i).abs())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in graph_out]
        fn()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got, outputs())):
            assert torch.equal(a, b), (i, j)


def test_other_stream():
    """Calls on a stream of their own, with work queued before and after them."""
    cu, D = [0, 200, 500], 16
    x, g, h0, dev = _scan_case(cu, D, F32, False, True, False, seed=8, slow=True)
    plan = kda.Plan(cu, 5)
    ref = layer.scan_forward(plan, *dev, initial_state=_d(h0))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = {n: torch.full_like(t, -7.0) for n, t in ref.items()}
    stream.wait_stream(torch.cuda.current_stream())
    init = _d(h0)
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        layer.scan_forward(plan, *dev, initial_state=init, out=out, stream=stream)
    stream.synchronize()
    for n in ref:
        assert torch.equal(out[n], ref[n])


def test_two_streams_at_once():
    """Calls that run at the same time, each with its own workspace: scans of
    many tiles, backward sums, steps; every result as when run alone."""
    cu, D = [0, 20000], 512
    plan = kda.Plan(cu, 1)
    plan.device_blob(DEV)
    sets, ref = [], []
    for i in range(2):
        _, _, h0, dev = _scan_case(cu, D, BF, True, True, False, seed=20 + i, slow=True)
        raw, a_log, dt_bias = _prepare_inputs(300, 8, BF, True, seed=30 + i)
        grads = [_d(_randn(300, 8, 128, seed=40 + i)) for _ in range(3)] + [_d(_randn(300, 8, seed=41 + i))]
        sets.append((dev, _d(h0), [_d(t) for t in raw.values()], _d(a_log), _d(dt_bias), grads))

    def work(s, stream=None):
        dev, h0, raw, a_log, dt_bias, grads = s
        f = layer.scan_forward(plan, *dev, initial_state=h0, tied=True, stream=stream)
        b = layer.scan_backward(plan, *dev, f["h"], dev[0], initial_state=h0, tied=True, stream=stream)
        r = layer.prepare_inputs_backward(*raw, a_log, dt_bias, *grads, stream=stream)
        return [*f.values(), *b.values(), *r.values()]

    for s in sets:
        ref.append(work(s))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = [work(s, st) for s, st in zip(sets, streams)]
        for st in streams:
            st.synchronize()
        for a, b in zip(got, ref):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
