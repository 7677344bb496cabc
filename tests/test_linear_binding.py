"""What the Python layer holds and asks for around the calls of linear attention and
of the norms and rotation before it (CPU only: the C calls are stubbed)."""
import gc
import weakref

import pytest
import torch

from gated_delta_rule_37_amd import kda, layer

BF, F32 = torch.bfloat16, torch.float32
T, H = 300, 2


def _calls():
    x, g, weight, plan = torch.zeros(T, H, 64, dtype=BF), torch.zeros(T, H), torch.zeros(64), kda.Plan([0, T], 2)
    return dict(
        kda_qk_norm_rotate_backward=lambda **s: layer.qk_norm_rotate_backward(x, x, None, None, weight, weight, x, x, **s),
        kda_linear_forward=lambda **s: layer.linear_forward(plan, x, x, x, g, **s),
        kda_linear_backward=lambda **s: layer.linear_backward(plan, x, x, x, g, x, **s))


def _stubs(monkeypatch, call, empty=None):
    blob = lambda self, device, stream=None: torch.from_numpy(self.blob.copy())  # noqa: E731
    monkeypatch.setattr(kda.Plan, "device_blob", blob)
    monkeypatch.setattr(layer, "_empty", empty or (lambda stream, device, dtype, *shape: torch.empty(*shape, dtype=dtype)))
    monkeypatch.setattr(layer, "_call", call)


@pytest.mark.parametrize("name", _calls())
def test_workspace_outlives_the_call(name, monkeypatch):
    """The workspace belongs to the call until the C function has returned."""
    made, seen = [], []

    def empty(stream, device, dtype, *shape):
        t = torch.empty(*shape, dtype=dtype, device=device)
        if dtype == torch.uint8:
            made.append((weakref.ref(t), t.data_ptr(), t.numel()))
        return t

    def call(called, device, args, stream):
        gc.collect()
        assert called == name
        (ref, address, size), = made
        assert ref() is not None, "the workspace was freed before the call"
        assert tuple(args[-2:]) == (address, size)
        seen.append(called)

    _stubs(monkeypatch, call, empty)
    _calls()[name]()
    assert seen == [name]
    gc.collect()
    assert made[0][0]() is None, "the workspace is kept after the call"


@pytest.mark.parametrize("name", _calls())
def test_everything_is_asked_for_on_the_calls_stream(name, monkeypatch):
    asked = []
    _stubs(monkeypatch, lambda called, device, args, stream: asked.append(stream),
           lambda stream, device, dtype, *shape: asked.append(stream) or torch.empty(*shape, dtype=dtype))
    monkeypatch.setattr(kda.Plan, "device_blob",
                        lambda self, device, stream=None: asked.append(stream) or torch.from_numpy(self.blob.copy()))
    _calls()[name](stream="side")
    assert len(asked) > 3 and set(asked) == {"side"}


def test_uncut_forward_takes_no_workspace(monkeypatch):
    x, g = torch.zeros(T, H, 64, dtype=BF), torch.zeros(T, H)
    seen = []
    _stubs(monkeypatch, lambda called, device, args, stream: seen.append(tuple(args[-2:])))
    layer.linear_forward(kda.Plan([0, T], 1), x, x, x, g)
    assert seen == [(None, 0)]


def test_heads_come_from_the_widest(monkeypatch):
    """H is the most heads of q, k, v and g; the others share."""
    seen = []
    _stubs(monkeypatch, lambda called, device, args, stream: seen.append(args))
    q, v, plan = torch.zeros(T, 2, 64, dtype=BF), torch.zeros(T, 1, 32, dtype=BF), kda.Plan([0, T], 1)
    out = layer.linear_forward(plan, q, v.expand(T, 1, 32).new_zeros(T, 1, 64), v, torch.zeros(6))
    assert out["o"].shape == (T, 6, 32) and out["final_state"].shape == (1, 6, 64, 32)
    grads = layer.linear_backward(plan, q, torch.zeros(T, 1, 64, dtype=BF), v, torch.zeros(6), torch.zeros(T, 6, 32, dtype=BF),
                                  want_dh0=True)
    assert grads["dq"].shape == q.shape and grads["dv"].shape == v.shape and grads["dg"].shape == (6,)
    assert grads["dh0"].shape == (1, 6, 64, 32)
    assert [a[3:9] for a in seen] == [[6, 2, 1, 1, 64, 32]] * 2
