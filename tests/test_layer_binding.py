"""Who holds the memory that the Python layer hands to the library (CPU only:
the C calls are stubbed)."""
import gc
import weakref

import pytest
import torch

from gated_delta_rule_37_amd import kda, layer

BF, F32 = torch.bfloat16, torch.float32


def _calls():
    """Every call that takes a workspace, on CPU tensors."""
    T, H, D = 300, 2, 24
    rows, b = torch.zeros(T, H, 128), torch.zeros(T, H)
    x, plan = torch.zeros(T, D), kda.Plan([0, T], 1)
    return dict(
        kda_prepare_inputs_backward=lambda: layer.prepare_inputs_backward(rows, rows, rows, b, b[0], rows[0], rows, rows,
                                                                          rows, b),
        kda_output_norm_backward=lambda: layer.output_norm_backward(rows, rows, rows[0, 0]),
        kda_scan_forward=lambda: layer.scan_forward(plan, x, x),
        kda_scan_backward=lambda: layer.scan_backward(plan, x, x, x, x))


@pytest.mark.parametrize("name", _calls())
def test_workspace_outlives_the_call(name, monkeypatch):
    """The workspace belongs to the call until the C function has returned: that
    function runs without the interpreter's lock, so another thread could be
    given the same memory on the same stream."""
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

    monkeypatch.setattr(layer, "_empty", empty)
    monkeypatch.setattr(layer, "_call", call)
    _calls()[name]()
    assert seen == [name]
    gc.collect()
    assert made[0][0]() is None, "the workspace is kept after the call"
