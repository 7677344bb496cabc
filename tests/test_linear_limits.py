"""The sizes that linear attention's grids cannot take (CPU only): the calls refuse
them, and the workspace queries, by which a caller allocates first, give 0."""
import pytest

from gated_delta_rule_37_amd import kda

FAKE, BIG, UNSUPPORTED = 1 << 20, 1 << 60, -4
BF16 = 1


def _forward(plan, H, K, V):
    """A call whose buffers are all there, of sizes that are refused."""
    buf = [FAKE, BIG]
    return kda.lib().kda_linear_forward(plan.handle, *buf, H, 1, 1, 1, K, V, *buf, K, *buf, K, *buf, V, *buf, H, BF16, *buf,
                                        *buf, BF16, *buf, *buf, None)


def _backward(plan, H, Hq, Hk, Hv, K, V):
    buf = [FAKE, BIG]
    return kda.lib().kda_linear_backward(plan.handle, *buf, H, Hq, Hk, Hv, K, V, *buf, Hq * K, *buf, Hk * K, *buf, Hv * V,
                                         *buf, H, BF16, *buf, *buf, *buf, *buf, *buf, *buf, BF16, *buf, *buf, *buf, None)


def test_fragments_and_heads():
    """513 sequences of 16384 heads are too many workgroups of 256 threads, 511 are not."""
    lib, H = kda.lib(), 16384
    plan, fits = kda.Plan(list(range(0, 514)), 2), kda.Plan(list(range(0, 1023, 2)), 1)
    assert plan.F * H > 8388607 >= fits.F * H
    assert _forward(plan, H, 8, 8) == UNSUPPORTED and _backward(plan, H, 1, 1, 1, 8, 8) == UNSUPPORTED
    assert lib.kda_linear_workspace_bytes(plan.handle, H, 8, 8) == 0
    assert lib.kda_linear_backward_workspace_bytes(plan.handle, H, 1, 1, 1, 8, 8) == 0
    assert lib.kda_linear_backward_workspace_bytes(fits.handle, H, 1, 1, 1, 8, 8) > 0
    cut = kda.Plan([0, 511], 511)
    assert cut.F * H <= 8388607 and lib.kda_linear_workspace_bytes(cut.handle, H, 8, 8) > 0


@pytest.mark.parametrize("Hq,Hk,Hv", [(8, 16, 16), (16, 8, 16), (16, 16, 8)])
def test_gradients_of_shared_heads(Hq, Hk, Hv):
    """8 heads of 128 channels are 2^31 threads of four at 2^23 tokens, too many; two tokens less fit;
    without shared heads there is no such launch."""
    lib, H = kda.lib(), 16
    plan, less = kda.Plan([0, 1 << 23], 1), kda.Plan([0, (1 << 23) - 2], 1)
    size = lib.kda_linear_backward_workspace_bytes
    assert _backward(plan, H, Hq, Hk, Hv, 128, 128) == UNSUPPORTED
    assert size(plan.handle, H, Hq, Hk, Hv, 128, 128) == 0
    assert size(less.handle, H, Hq, Hk, Hv, 128, 128) > 0 and size(plan.handle, H, H, H, H, 128, 128) > 0
    assert lib.kda_linear_workspace_bytes(plan.handle, H, 128, 128) == 0   # one piece: none needed
