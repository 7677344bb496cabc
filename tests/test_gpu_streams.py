"""Memory of calls on another stream than the current one, on the GPU: what a
call allocates and a plan's device copy are not handed on while it runs."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def busy():
    """Keeps a stream busy for some milliseconds with scans of its own."""
    T, D = 32768, 4096
    plan = kda.Plan([0, T], 1)
    x, g = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV), torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)
    out = dict(h=torch.empty_like(x), final_state=torch.empty(1, D, device=DEV))
    plan.device_blob(DEV)
    torch.cuda.synchronize()

    def run(stream):
        for _ in range(60):
            layer.scan_forward(plan, x, g, out=out, stream=stream)
    return run


def test_plan_copy_is_not_handed_on_while_a_stream_reads_it(busy):
    """A plan dropped right after its call on a side stream: as long as that
    stream runs, no new tensor of the current stream has its memory."""
    T, D = 500, 16
    x, g = torch.ones(T, D, device=DEV), torch.full((T, D), -0.1, device=DEV)
    want = layer.scan_forward(kda.Plan([0, 200, T], 1), x, g)
    plan = kda.Plan([0, 200, T], 1)
    at, words = plan.device_blob(DEV).data_ptr(), len(plan.blob)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy(side)
    got = layer.scan_forward(plan, x, g, stream=side)
    del plan
    new = [torch.empty(words, dtype=torch.int32, device=DEV) for _ in range(200)]
    assert not side.query()
    assert at not in {t.data_ptr() for t in new}
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_forward_and_backward_allocate_on_their_stream(busy):
    """kda.forward's and kda.backward's outputs and workspaces on a side stream
    keep their values while the current stream allocates and writes."""
    T, H, cu = 600, 2, [0, 250, 600]
    x = {n: t.to(DEV) for n, t in synth.make_inputs(T, H, 128, 128, seed=3, cu_seqlens=cu, gate_scale=0.05).items()
         if n != "cu_seqlens"}
    ins = [x[n] for n in ("q", "k", "v", "g", "beta")]
    plan = kda.Plan(cu, 2)
    d_o = torch.ones(T, H, 128, device=DEV)

    def work(stream):
        f = kda.forward(plan, *ins, stream=stream)
        return f, kda.backward(plan, *ins, d_o, want_dh0=True, stream=stream)

    want_f, want_b = work(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy(side)
    f, b = work(side)
    sizes = [t.numel() * t.element_size() for t in f.values()] + [
        int(kda.lib().kda_backward_workspace_bytes(plan.handle, H, 128, 128))]
    new = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    assert not side.query()
    side.synchronize()
    assert len(new) == 2 * len(sizes)
    for n in ("o", "final_state"):
        assert torch.equal(f[n], want_f[n]), n
    for n in want_b:
        assert torch.equal(b[n], want_b[n]), n
