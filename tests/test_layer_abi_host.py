"""Host-side refusals of the operators around the recurrence (no GPU needed).

Every call below has at least one bad argument, so nothing is launched and the
fake addresses are never dereferenced: each bad argument must give the
documented status, whatever the others hold."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, SMALL = 0, -1, -4, -5, -8, -9
FAKE, BIG = 1 << 20, 1 << 44
F32, BF16 = 0, 1
NAN, INF = float("nan"), float("inf")


class Call:
    """A C call's arguments by name.  Buffers are name -> [address, bytes] and
    inputs with a stride name -> [address, bytes, stride]."""

    def __init__(self, fn, **args):
        self.fn, self.args = fn, args

    def __call__(self, **change):
        args = {**self.args, **change}
        assert set(args) == set(self.args), set(args) - set(self.args)
        flat = []
        for v in args.values():
            flat += v if isinstance(v, list) else [v]
        return getattr(kda.lib(), self.fn)(*flat, None)


def _buffers(*names):
    return {n: [FAKE, BIG] for n in names}


def _prepare(T=5, H=3, backward=False):
    row, dims = H * 128, dict(T=T, H=H, K=128, dtype=BF16)
    raw = dict(q_raw=[FAKE, BIG, row], k_raw=[FAKE, BIG, row], gate_raw=[FAKE, BIG, row], beta_raw=[FAKE, BIG, H])
    common = {**dims, **raw, **_buffers("a_log", "dt_bias"), "q_scale": 1.0, "eps": 1e-6}
    if not backward:
        return Call("kda_prepare_inputs", **common, **_buffers("q", "k", "g", "beta"))
    return Call("kda_prepare_inputs_backward", **common, **_buffers(
        "dq", "dk", "dg", "dbeta", "dq_raw", "dk_raw", "dgate_raw", "dbeta_raw", "da_log", "ddt_bias", "workspace"))


def _norm(T=5, H=3, V=40, backward=False):
    gate = dict(gate=[FAKE, BIG, H * V], activation=1)
    if not backward:
        return Call("kda_output_norm", T=T, H=H, V=V, o=[FAKE, BIG], o_format=F32, **gate,
                    **_buffers("weight", "res_scale", "residual"), dtype=BF16, eps=1e-6, **_buffers("y"))
    return Call("kda_output_norm_backward", T=T, H=H, V=V, **_buffers("dy", "o"), o_format=F32, **gate,
                **_buffers("weight", "res_scale"), dtype=BF16, eps=1e-6, d_o=[FAKE, BIG], d_o_format=F32,
                **_buffers("d_gate", "d_weight", "d_res_scale", "workspace"))


_PLAN = kda.Plan([0, 3, 10], 2)
_LONG = kda.Plan([0, 3, 300], 2)    # more than one tile of tokens


def _scan(backward=False, plan=_PLAN, D=6, tied=1):
    head = dict(plan=plan.handle, plan_dev=[FAKE, BIG], D=D, dtype=BF16, x=[FAKE, BIG, D], g=[FAKE, BIG, D], tied=tied,
                initial_state=[FAKE, BIG])
    if not backward:
        return Call("kda_scan_forward", **head, h=[FAKE, BIG], h_format=BF16, **_buffers("final_state", "workspace"))
    return Call("kda_scan_backward", **head, **_buffers("h", "dh"), h_format=BF16,
                **_buffers("d_final", "dx", "dg", "d_initial_state", "workspace"))


def _scan_step():
    return Call("kda_scan_step", B=4, D=6, dtype=BF16, **_buffers("x", "g"), tied=0, slots=[FAKE, BIG], num_slots=9,
                **_buffers("state", "state_out", "h"))


def _step():
    return Call("kda_step", B=5, H=3, K=128, V=128, head_begin=0, head_count=3, **_buffers("q", "k", "v", "g", "beta"),
                gate_lower_bound=-INF, slots=[FAKE, BIG], num_slots=9, **_buffers("state", "state_out", "o"),
                o_format=F32)


CALLS = dict(prepare=_prepare(), prepare_bwd=_prepare(backward=True), norm=_norm(), norm_bwd=_norm(backward=True),
             scan=_scan(), scan_bwd=_scan(backward=True), scan_step=_scan_step(), step=_step())

# bytes of each buffer, rows' strides as above
NEED = dict(
    prepare=dict(q_raw=5 * 768, k_raw=5 * 768, gate_raw=5 * 768, beta_raw=30, a_log=12, dt_bias=3 * 512,
                 q=5 * 768, k=5 * 768, g=5 * 768, beta=30),
    prepare_bwd=dict(q_raw=5 * 768, k_raw=5 * 768, gate_raw=5 * 768, beta_raw=30, a_log=12, dt_bias=3 * 512,
                     dq=5 * 1536, dk=5 * 1536, dg=5 * 1536, dbeta=60, dq_raw=5 * 768, dk_raw=5 * 768,
                     dgate_raw=5 * 768, dbeta_raw=30, da_log=12, ddt_bias=3 * 512),
    norm=dict(o=2400, gate=1200, weight=160, res_scale=480, residual=1200, y=1200),
    norm_bwd=dict(dy=1200, o=2400, gate=1200, weight=160, res_scale=480, d_o=2400, d_gate=1200, d_weight=160,
                  d_res_scale=480),
    scan=dict(plan_dev=4 * len(_PLAN.blob), x=120, g=120, initial_state=48, h=120, final_state=48),
    scan_bwd=dict(plan_dev=4 * len(_PLAN.blob), x=120, g=120, initial_state=48, h=120, dh=120, d_final=48, dx=120,
                  dg=120, d_initial_state=48),
    scan_step=dict(x=48, g=48, slots=16, state=216, state_out=216, h=48),
    step=dict(q=3840, k=3840, v=3840, g=3840, beta=30, slots=20, state=9 * 3 * 65536, state_out=9 * 3 * 65536, o=7680),
)
OPTIONAL = dict(prepare={"dt_bias"}, prepare_bwd=set(), norm={"res_scale", "residual"}, norm_bwd=set(),
                scan={"initial_state"}, scan_bwd={"initial_state", "d_final", "d_initial_state"},
                scan_step={"slots"}, step={"slots"})


@pytest.mark.parametrize("call,name", [(c, n) for c in NEED for n in NEED[c]])
def test_buffers(call, name):
    """Null, misaligned and a byte too small, one buffer at a time."""
    c = CALLS[call]
    rest = c.args[name][2:]
    if name not in OPTIONAL[call]:
        assert c(**{name: [None, BIG, *rest]}) == INVALID
    assert c(**{name: [FAKE + 8, BIG, *rest]}) == MISALIGNED
    assert c(**{name: [FAKE, NEED[call][name] - 1, *rest]}) == SMALL


@pytest.mark.parametrize("call", CALLS)
def test_every_buffer_is_checked(call):
    assert set(NEED[call]) | {"workspace"} >= {n for n, v in CALLS[call].args.items() if isinstance(v, list)}


@pytest.mark.parametrize("call,sizes", [(c, s) for c, ss in dict(
    prepare="THK", prepare_bwd="THK", norm="THV", norm_bwd="THV", scan="D", scan_bwd="D", scan_step="BD", step="BHKV",
).items() for s in ss])
def test_sizes(call, sizes):
    c = CALLS[call]
    for v in (0, -1):
        assert c(**{sizes: v}) == INVALID
    if sizes in "KV" and call not in ("norm", "norm_bwd"):
        assert c(**{sizes: 64}) == UNSUPPORTED
    else:
        over = dict(T=(1 << 30) + 1, H=65536, V=8193, B=(1 << 20) + 1, D=(1 << 20) + 1)[sizes]
        assert c(**{sizes: over}) == UNSUPPORTED
    if call in ("norm", "norm_bwd") and sizes == "V":
        assert c(H=4096, V=4097, gate=[FAKE, BIG, 4096 * 4097]) == UNSUPPORTED


@pytest.mark.parametrize("call", ["prepare", "prepare_bwd", "norm", "norm_bwd"])
def test_eps(call):
    for eps in (0.0, -1e-6, NAN, INF):
        assert CALLS[call](eps=eps) == INVALID


@pytest.mark.parametrize("call,name,bad", [
    ("prepare", "dtype", 2), ("prepare_bwd", "dtype", -1), ("norm", "dtype", 2), ("norm", "o_format", 2),
    ("norm", "activation", 3), ("norm_bwd", "d_o_format", 2), ("norm_bwd", "activation", -1), ("scan", "dtype", 2),
    ("scan", "h_format", 2), ("scan", "tied", 2), ("scan_bwd", "h_format", -1), ("scan_bwd", "tied", -1),
    ("scan_step", "dtype", 7), ("scan_step", "tied", 2), ("scan_step", "num_slots", 0), ("step", "num_slots", -3),
    ("step", "o_format", 2), ("step", "gate_lower_bound", NAN), ("step", "gate_lower_bound", 0.5),
    ("prepare", "q_scale", NAN), ("prepare_bwd", "q_scale", INF), ("scan", "plan", None),
])
def test_options(call, name, bad):
    assert CALLS[call](**{name: bad}) == INVALID


@pytest.mark.parametrize("begin,count", [(-1, 1), (0, 0), (0, 4), (3, 1)])
def test_step_head_range(begin, count):
    assert CALLS["step"](head_begin=begin, head_count=count) == INVALID


@pytest.mark.parametrize("call,name,row", [
    ("prepare", "q_raw", 384), ("prepare", "k_raw", 384), ("prepare_bwd", "gate_raw", 384), ("prepare", "beta_raw", 3),
    ("norm", "gate", 120), ("norm_bwd", "gate", 120), ("scan", "x", 6), ("scan", "g", 6), ("scan_bwd", "g", 6)])
def test_strides(call, name, row):
    """Shorter than the row, too long, and bytes counted to the last row's end."""
    c = CALLS[call]
    rows = 10 if "scan" in call else 5
    assert c(**{name: [FAKE, BIG, row - 1]}) == INVALID
    assert c(**{name: [FAKE, BIG, 1 << 31]}) == UNSUPPORTED
    wide = row + 8
    assert c(**{name: [FAKE, 2 * ((rows - 1) * wide + row) - 1, wide]}) == SMALL


def test_prepare_stride_alignment():
    assert CALLS["prepare"](q_raw=[FAKE, BIG, 388]) == MISALIGNED
    assert CALLS["prepare_bwd"](gate_raw=[FAKE, BIG, 385]) == MISALIGNED


def test_optional_pairs():
    """A gradient is asked for exactly where its input is given."""
    none = [None, 0]
    assert CALLS["prepare_bwd"](dt_bias=none) == INVALID
    assert CALLS["prepare_bwd"](ddt_bias=none) == INVALID
    assert CALLS["norm_bwd"](res_scale=none) == INVALID
    assert CALLS["norm_bwd"](d_res_scale=none) == INVALID
    assert CALLS["norm_bwd"](d_gate=none) == INVALID
    assert CALLS["norm"](gate=[None, 0, 0]) == INVALID
    assert CALLS["norm"](activation=0) == INVALID
    assert CALLS["norm_bwd"](activation=0) == INVALID
    # the scan's backward needs x only when tied: here the small buffer behind it is found
    assert _scan(True, tied=0)(x=[None, 0, 0], dg=[FAKE, 1]) == SMALL
    assert _scan(True, tied=1)(x=[None, 0, 0], dg=[FAKE, 1]) == INVALID


@pytest.mark.parametrize("call,need", [
    ("prepare_bwd", lambda: kda.lib().kda_prepare_inputs_backward_workspace_bytes(5, 3, 128)),
    ("norm_bwd", lambda: kda.lib().kda_output_norm_backward_workspace_bytes(5, 3, 40)),
    ("scan_long", lambda: kda.lib().kda_scan_workspace_bytes(_LONG.handle, 6)),
    ("scan_bwd_long", lambda: kda.lib().kda_scan_workspace_bytes(_LONG.handle, 6))])
def test_workspace(call, need):
    size = need()
    assert size > 0
    run = {**CALLS, "scan_long": _scan(plan=_LONG), "scan_bwd_long": _scan(True, _LONG)}[call]
    assert run(workspace=[None, BIG]) == INVALID
    assert run(workspace=[FAKE + 4, BIG]) == MISALIGNED
    assert run(workspace=[FAKE, size - 1]) == WORKSPACE


def test_workspace_sizes():
    L = kda.lib()
    assert L.kda_prepare_inputs_backward_workspace_bytes(0, 3, 128) == 0
    assert L.kda_prepare_inputs_backward_workspace_bytes(5, 3, 64) == 0
    assert L.kda_output_norm_backward_workspace_bytes(5, 3, 8193) == 0
    assert L.kda_output_norm_backward_workspace_bytes(5, 0, 8) == 0
    assert L.kda_scan_workspace_bytes(None, 6) == 0
    assert L.kda_scan_workspace_bytes(_LONG.handle, 0) == 0
    # at most 128 tokens need none; then 12 bytes a channel of whole blocks of
    # 64 and tile of 128 tokens, and a 128-byte ticket a block
    assert L.kda_scan_workspace_bytes(_PLAN.handle, 6) == 0
    assert L.kda_scan_workspace_bytes(kda.Plan([0, 128], 1).handle, 6) == 0
    assert L.kda_scan_workspace_bytes(kda.Plan([0, 129], 1).handle, 6) == 2 * 64 * 12 + 128
    assert L.kda_scan_workspace_bytes(kda.Plan([0, 65536], 1).handle, 4096) == 512 * 4096 * 12 + 64 * 128


def test_pools():
    """state_out is state itself or does not touch it; slots may only be left
    out where every row has one."""
    pool = 9 * 3 * 65536
    for shift in (16, -16, pool - 16, 16 - pool):
        assert CALLS["step"](state=[FAKE + (1 << 24), BIG], state_out=[FAKE + (1 << 24) + shift, BIG]) == INVALID
    assert CALLS["scan_step"](state=[FAKE, BIG], state_out=[FAKE + 208, BIG]) == INVALID
    assert CALLS["step"](slots=[None, 0], num_slots=3) == INVALID
    assert CALLS["scan_step"](slots=[None, 0], num_slots=3) == INVALID


def test_binding_refuses():
    """The Python layer's own checks, before the library is called."""
    q = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
    b, a = torch.zeros(2, 1, dtype=torch.bfloat16), torch.zeros(1)
    with pytest.raises(ValueError, match="needs device tensors"):
        layer.prepare_inputs(q, q, q, b, a)
    with pytest.raises(TypeError, match="q_raw"):
        layer.prepare_inputs(q.half(), q.half(), q.half(), b.half(), a)
    with pytest.raises(TypeError, match="k_raw"):
        layer.prepare_inputs(q, q.float(), q, b, a)
    with pytest.raises(ValueError, match="shape"):
        layer.prepare_inputs(q, q[:1], q, b, a)
    with pytest.raises(ValueError, match="activation"):
        layer.output_norm(q, torch.ones(128), gate=q, activation="tanh")
    with pytest.raises(ValueError, match="without an activation"):
        layer.output_norm(q, torch.ones(128), gate=q, activation="none")
    with pytest.raises(TypeError, match="expected"):
        layer.output_norm(q, torch.ones(128), gate=q, residual=q.float())
    with pytest.raises(TypeError, match="expected"):
        layer.output_norm(q.half(), torch.ones(128))
    with pytest.raises(ValueError, match="tokens"):
        layer.scan_forward(kda.Plan([0, 3], 1), q[:, 0], q[:, 0])


def test_row_strides_of_the_binding():
    """Slices of a wider projection keep their stride; overlapping, transposed
    or scattered rows are refused."""
    wide = torch.zeros(4, 64)
    for t, want in ((wide[:, 8:24], 64), (wide, 64), (wide[:1, :16], 16), (wide[:, :32].view(4, 2, 16), 64)):
        assert layer._row_stride(t, "t") == want
        assert layer._rows(t, t.dtype, t.shape, "t", t.device) == (
            t.data_ptr(), ((t.shape[0] - 1) * want + t[0].numel()) * 4, want)
    for bad in (wide.t(), wide[:, ::2], torch.zeros(1, 8).expand(4, 8), torch.zeros(40).as_strided((4, 8), (4, 1)),
                wide.view(4, 8, 8).transpose(1, 2)):
        with pytest.raises(ValueError, match="dense"):
            layer._row_stride(bad, "t")
