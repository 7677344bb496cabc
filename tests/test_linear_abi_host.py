"""Host-side refusals of linear attention and of the norms and rotation before it
(no GPU needed).

Every call below has at least one bad argument, so nothing is launched and the
fake addresses are never dereferenced: each bad argument must give the
documented status, whatever the others hold."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, SMALL = -1, -4, -5, -8, -9
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


def _rotate(T=5, Hq=4, Hk=2, D=64, R=32, backward=False):
    common = dict(T=T, Hq=Hq, Hk=Hk, D=D, R=R, dtype=BF16, interleaved=0, q_raw=[FAKE, BIG, Hq * D + 8],
                  k_raw=[FAKE, BIG, Hk * D], **_buffers("positions", "inv_freq", "q_weight", "k_weight"), q_scale=1.0,
                  eps=1e-6)
    if not backward:
        return Call("kda_qk_norm_rotate", **common, **_buffers("q", "k"))
    return Call("kda_qk_norm_rotate_backward", **common, **_buffers("dq", "dk"), d_format=F32,
                **_buffers("dq_raw", "dk_raw", "dq_weight", "dk_weight", "workspace"))


def _step():
    return Call("kda_linear_step", B=5, H=6, Hq=2, Hk=3, Hv=6, K=64, V=40, **_buffers("q", "k", "v"), g=[FAKE, BIG, 6],
                g_dtype=F32, slots=[FAKE, BIG], num_slots=9, **_buffers("state", "state_out", "o"), o_format=BF16)


CALLS = dict(rotate=_rotate(), rotate_bwd=_rotate(backward=True), step=_step())

# bytes of each buffer, rows' strides as above
_ROTATE = dict(q_raw=(4 * 264 + 256) * 2, k_raw=5 * 256, positions=20, inv_freq=64, q_weight=256, k_weight=256)
NEED = dict(
    rotate=dict(**_ROTATE, q=5 * 512, k=5 * 256),
    rotate_bwd=dict(**_ROTATE, dq=5 * 1024, dk=5 * 512, dq_raw=5 * 512, dk_raw=5 * 256, dq_weight=256, dk_weight=256),
    step=dict(q=5 * 256, k=5 * 384, v=5 * 480, g=120, slots=20, state=9 * 6 * 64 * 40 * 4,
              state_out=9 * 6 * 64 * 40 * 4, o=5 * 480),
)
OPTIONAL = dict(rotate={"q_weight", "k_weight"}, rotate_bwd=set(), step={"slots"})
# sizes with the value that is one too many, each alone
SIZES = dict(rotate=dict(T=(1 << 30) + 1, Hq=65536, Hk=65536, D=264), rotate_bwd=dict(T=(1 << 30) + 1, Hq=65536, Hk=65536, D=264),
             step=dict(B=(1 << 20) + 1, K=136, V=136))


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


@pytest.mark.parametrize("call,size", [(c, s) for c in SIZES for s in SIZES[c]])
def test_sizes(call, size):
    for v in (0, -1):
        assert CALLS[call](**{size: v}) == INVALID
    assert CALLS[call](**{size: SIZES[call][size]}) == UNSUPPORTED


@pytest.mark.parametrize("call", ["rotate", "rotate_bwd"])
def test_rotate_options(call):
    c = CALLS[call]
    for eps in (0.0, -1e-6, NAN, INF):
        assert c(eps=eps) == INVALID
    for scale in (NAN, INF):
        assert c(q_scale=scale) == INVALID
    for R in (-2, 3, 66):
        assert c(R=R) == INVALID
    assert c(D=60) == UNSUPPORTED
    assert c(interleaved=2) == INVALID
    assert c(dtype=2) == INVALID
    for n in ("q_raw", "k_raw"):
        row = c.args[n][2]
        row = 256 if n == "q_raw" else row
        assert c(**{n: [FAKE, BIG, row - 1]}) == INVALID
        assert c(**{n: [FAKE, BIG, 1 << 31]}) == UNSUPPORTED


def test_rotate_without_rotation_needs_no_positions():
    """R = 0: positions and frequencies may be absent (the short output refuses)."""
    c = CALLS["rotate"]
    assert c(R=0, positions=[None, 0], inv_freq=[None, 0], k=[FAKE, 1]) == SMALL


def test_rotate_backward_options():
    c = CALLS["rotate_bwd"]
    assert c(d_format=2) == INVALID
    for n in ("q_weight", "k_weight", "dq_weight", "dk_weight"):
        assert c(**{n: [None, 0]}) == INVALID
    need = kda.lib().kda_qk_norm_rotate_backward_workspace_bytes(5, 64)
    assert need >= 5 * 2 * 64 * 4
    assert c(workspace=[None, 0]) == INVALID
    assert c(workspace=[FAKE + 8, need]) == MISALIGNED
    assert c(workspace=[FAKE, need - 1]) == WORKSPACE


def test_rotate_workspace_of_bad_sizes():
    size = kda.lib().kda_qk_norm_rotate_backward_workspace_bytes
    assert [size(*a) for a in ((0, 64), (5, 0), (5, 264), (-1, 64))] == [0] * 4


def test_step_options():
    c = CALLS["step"]
    for n, bad in (("H", 0), ("Hq", 0), ("Hk", -1), ("Hv", 0), ("num_slots", 0)):
        assert c(**{n: bad}) == INVALID
    for n in ("Hq", "Hk", "Hv"):
        assert c(**{n: 4}) == INVALID          # 6 heads are no multiple
        assert c(**{n: 12}) == INVALID
    for n in ("K", "V"):
        assert c(**{n: 44}) == UNSUPPORTED
    assert c(H=65536, Hq=1, Hk=1, Hv=1, g=[FAKE, BIG, 65536]) == UNSUPPORTED
    assert c(g_dtype=2) == INVALID and c(o_format=2) == INVALID
    for stride in (1, 5, 7, -1):
        assert c(g=[FAKE, BIG, stride]) == INVALID
    assert c(g=[FAKE, 23, 0]) == SMALL          # one g a head: 24 bytes
    assert c(slots=[None, 0], num_slots=4) == INVALID
    pool = NEED["step"]["state"]
    assert c(state_out=[FAKE + 16, BIG]) == INVALID
    assert c(state_out=[FAKE + pool, BIG], o=[FAKE, 1]) == SMALL


# ---------------------------------------------------------------------------
# kda_linear_forward and kda_linear_backward

T, N, H, HQ, HK, HV, K, V = 300, 3, 6, 2, 3, 6, 64, 40
PLAN = kda.Plan([0, 7, 64, T], 3)


def _linear(backward=False):
    common = dict(plan=PLAN.handle, plan_dev=[FAKE, BIG], H=H, Hq=HQ, Hk=HK, Hv=HV, K=K, V=V,
                  q=[FAKE, BIG, HQ * K + 8], k=[FAKE, BIG, HK * K], v=[FAKE, BIG, HV * V], g=[FAKE, BIG, H + 1],
                  g_dtype=F32, **_buffers("initial_state"))
    if not backward:
        return Call("kda_linear_forward", **common, o=[FAKE, BIG], o_format=BF16, **_buffers("final_state", "workspace"))
    return Call("kda_linear_backward", **common, **_buffers("d_o", "d_final", "dq", "dk", "dv"), grad_format=F32,
                **_buffers("dg", "d_initial_state", "workspace"))


LINEAR = dict(linear=_linear(), linear_bwd=_linear(backward=True))
_STATE = N * H * K * V * 4
_LINEAR_IN = dict(plan_dev=len(PLAN.blob) * 4, q=((T - 1) * (HQ * K + 8) + HQ * K) * 2, k=T * HK * K * 2, v=T * HV * V * 2,
                  g=((T - 1) * (H + 1) + H) * 4, initial_state=_STATE)
LINEAR_NEED = dict(
    linear=dict(**_LINEAR_IN, o=T * H * V * 2, final_state=_STATE),
    linear_bwd=dict(**_LINEAR_IN, d_o=T * H * V * 2, d_final=_STATE, dq=T * HQ * K * 4, dk=T * HK * K * 4,
                    dv=T * HV * V * 4, dg=T * H * 4, d_initial_state=_STATE))
LINEAR_OPTIONAL = {"initial_state", "d_final", "d_initial_state"}


def _linear_workspace(call):
    lib = kda.lib()
    if call == "linear":
        return lib.kda_linear_workspace_bytes(PLAN.handle, H, K, V)
    return lib.kda_linear_backward_workspace_bytes(PLAN.handle, H, HQ, HK, HV, K, V)


@pytest.mark.parametrize("call,name", [(c, n) for c in LINEAR_NEED for n in LINEAR_NEED[c]])
def test_linear_buffers(call, name):
    c = LINEAR[call]
    rest = c.args[name][2:]
    if name not in LINEAR_OPTIONAL:
        assert c(**{name: [None, BIG, *rest]}) == INVALID
    assert c(**{name: [FAKE + 8, BIG, *rest]}) == MISALIGNED
    assert c(**{name: [FAKE, LINEAR_NEED[call][name] - 1, *rest]}) == SMALL


@pytest.mark.parametrize("call", LINEAR)
def test_linear_options(call):
    c = LINEAR[call]
    assert set(LINEAR_NEED[call]) | {"workspace"} == {n for n, v in c.args.items() if isinstance(v, list)}
    assert c(plan=None) == INVALID
    for n in ("H", "Hq", "Hk", "Hv", "K", "V"):
        for bad in (0, -1):
            assert c(**{n: bad}) == INVALID
    for n in ("Hq", "Hk", "Hv"):
        assert c(**{n: 4}) == INVALID and c(**{n: 12}) == INVALID
    for n in ("K", "V"):
        assert c(**{n: 136}) == UNSUPPORTED and c(**{n: 44}) == UNSUPPORTED
    one = dict(Hq=1, Hk=1, Hv=1, q=[FAKE, BIG, K], k=[FAKE, BIG, K], v=[FAKE, BIG, V])
    assert c(H=16385, **one, g=[FAKE, BIG, 16385]) == UNSUPPORTED
    assert c(g_dtype=2) == INVALID
    assert c(**{"o_format" if call == "linear" else "grad_format": 2}) == INVALID
    for n, row in (("q", HQ * K), ("k", HK * K), ("v", HV * V)):
        assert c(**{n: [FAKE, BIG, row - 8]}) == INVALID
        assert c(**{n: [FAKE, BIG, row + 4]}) == MISALIGNED
        assert c(**{n: [FAKE, BIG, (1 << 22) + 8]}) == UNSUPPORTED
    for stride in (H - 1, -1):
        assert c(g=[FAKE, BIG, stride]) == INVALID
    assert c(g=[FAKE, BIG, (1 << 22) + 1]) == UNSUPPORTED
    assert c(g=[FAKE, H * 4 - 1, 0]) == SMALL          # one g a head
    need = _linear_workspace(call)
    assert need > 0
    assert c(workspace=[None, 0]) == INVALID
    assert c(workspace=[FAKE + 8, need]) == MISALIGNED
    assert c(workspace=[FAKE, need - 1]) == WORKSPACE


def test_linear_workspaces():
    lib = kda.lib()
    uncut = kda.Plan([0, 7, 64, T], 1)
    assert lib.kda_linear_workspace_bytes(uncut.handle, H, K, V) == 0
    assert lib.kda_linear_backward_workspace_bytes(uncut.handle, H, HQ, HK, HV, K, V) > 0
    forward = lib.kda_linear_workspace_bytes
    assert [forward(None, H, K, V)] + [forward(PLAN.handle, *a) for a in ((0, K, V), (16385, K, V), (H, 136, V), (H, K, 0))] == [0] * 5
    backward = lib.kda_linear_backward_workspace_bytes
    bad = ((0, 1, 1, 1, K, V), (H, 4, HK, HV, K, V), (H, HQ, HK, HV, 136, V), (H, HQ, HK, HV, K, -8))
    assert [backward(None, H, HQ, HK, HV, K, V)] + [backward(PLAN.handle, *a) for a in bad] == [0] * 5


def test_linear_segments():
    """One where the sequences are short enough, else whole chunks for each segment, at
    most 512 workgroups and 5 sqrt(chunks) segments."""
    count = layer.linear_segments
    assert count([0, 100], 4) == 1 and count([0, 1], 64) == 1
    assert count([0, 65536], 32) == 16 and count([0, 65536], 512) == 1 and count([0, 65536], 1) == 147
    assert count([0, 1024], 1) == 16 and count([0, 1501], 6) == 24 and count([0, 192], 6) == 1
    assert count([0, 64, 16448], 16) == 29
    assert count(list(range(0, 16385, 512)), 16) == 1
    many = list(range(0, 15000, 250))
    assert count([*many, 15900], 16) == 1 and count([*many, 15900], 8) == 63 and count([*many, 20000], 16) == 32


def test_binding_refuses_host_tensors():
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        layer.qk_norm_rotate(q, q)
    with pytest.raises(ValueError, match="device tensors"):
        layer.linear_step(q, q, q, torch.zeros(3, 2), torch.zeros(3, 2, 64, 64))
    plan = kda.Plan([0, 3], 1)
    with pytest.raises(ValueError, match="device tensors"):
        layer.linear_forward(plan, q, q, q, torch.zeros(3, 2))
    with pytest.raises(ValueError, match="device tensors"):
        layer.linear_backward(plan, q, q, q, torch.zeros(2), q)


def test_linear_binding_refusals():
    """Types, shapes and heads that the binding names before any call."""
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    g, plan = torch.zeros(3, 2), kda.Plan([0, 3], 1)
    with pytest.raises(ValueError, match="3 tokens, the plan 4"):
        layer.linear_forward(kda.Plan([0, 4], 1), q, q, q, g)
    with pytest.raises(TypeError, match="v: expected torch.bfloat16"):
        layer.linear_forward(plan, q, q, q.float(), g)
    with pytest.raises(ValueError, match="k: expected shape"):
        layer.linear_forward(plan, q, q[..., :56], q, g)
    with pytest.raises(TypeError, match="g: expected one of"):
        layer.linear_forward(plan, q, q, q, g.double())
    with pytest.raises(ValueError, match="initial_state: expected shape"):
        layer.linear_forward(plan, q, q, q, g, torch.zeros(1, 2, 64, 32))
    with pytest.raises(TypeError, match="grad_dtype"):
        layer.linear_backward(plan, q, q, q, g, q, grad_dtype=torch.float16)
    with pytest.raises(TypeError, match="d_o: expected torch.bfloat16"):
        layer.linear_backward(plan, q, q, q, g, q.float())
    with pytest.raises(ValueError, match="rows must be dense"):
        layer.linear_forward(plan, torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2), q, q, g)
