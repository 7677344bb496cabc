"""The norms and rotation of queries and keys on the GPU against their 64-bit
reference, within the reference's bounds (linear_reference states the counts)."""
import pytest
import torch

from gated_delta_rule_37_amd import kda, layer
import layer_reference as lr
import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# the kernel's FP32 eps, as the definition sees it
EPSILON = torch.tensor(1e-5, dtype=F32).double()


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _d(t):
    return None if t is None else t.to(DEV)


def _w(t):
    return None if t is None else t.double()


def _sliced(x, pad):
    """x as the first rows of a wider tensor, ``pad`` elements between them."""
    T = x.shape[0]
    wide = torch.full((T, x[0].numel() + pad), 7.0, dtype=x.dtype, device=DEV)
    wide[:, :x[0].numel()] = x.reshape(T, -1).to(DEV)
    return wide[:, :x[0].numel()].view(x.shape)


# T, Hq, Hk, D, R, dtype, gradients' dtype, interleaved, weights, elements between rows
CASES = [
    (1, 1, 1, 128, 128, BF, BF, False, "qk", 0),
    (3, 5, 2, 128, 64, BF, F32, False, "qk", 8),
    (37, 4, 4, 64, 64, F32, F32, False, "q", 0),
    (37, 4, 1, 64, 32, BF, BF, True, "k", 16),
    (130, 3, 3, 256, 256, BF, BF, False, "qk", 0),
    (5, 2, 2, 256, 254, F32, BF, True, "qk", 4),
    (9, 3, 1, 80, 40, BF, BF, False, "qk", 0),       # R / 2 no whole vectors
    (9, 3, 1, 80, 80, F32, F32, True, "qk", 0),
    (7, 2, 2, 8, 2, BF, BF, False, "qk", 0),
    (7, 2, 2, 8, 8, BF, F32, True, "", 0),
    (11, 1, 7, 24, 0, BF, BF, False, "qk", 8),        # no rotation
    (11, 1, 7, 192, 0, F32, F32, False, "", 0),
    (6, 2, 2, 136, 130, F32, F32, False, "qk", 3),    # rows at any element
    (6, 2, 2, 128, 128, BF, BF, False, "qk", 3),
    (6, 2, 2, 32, 32, BF, BF, False, "qk", 0),
    (6, 3, 3, 96, 96, BF, BF, False, "qk", 0),
    (6, 3, 3, 16, 16, BF, BF, False, "qk", 0),
    (6, 3, 3, 96, 6, F32, BF, False, "qk", 0),
    (2500, 17, 3, 128, 128, BF, BF, False, "qk", 8),
    (4099, 2, 1, 64, 48, BF, F32, True, "qk", 0),
    (300, 40, 8, 128, 96, BF, BF, False, "q", 0),
]


def _case(T, Hq, Hk, D, R, dtype, weights, pad, seed):
    x = dict(q=_randn(T, Hq, D, seed=seed, dtype=dtype, scale=3.0), k=_randn(T, Hk, D, seed=seed + 1, dtype=dtype))
    x["q"][0, 0] = 0                 # a row of zeros
    x["k"][-1, -1] *= 1e-3           # eps counts
    gen = torch.Generator().manual_seed(seed + 2)
    pos = torch.randint(-100, 1 << 22, (T,), generator=gen, dtype=torch.int32)
    pos[0] = 0
    inv = (10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / max(R, 1))).float() if R else None
    w = {n: 1 + 0.5 * _randn(D, seed=seed + 3 + i) if n in weights else None for i, n in enumerate("qk")}
    dev = {n: _sliced(t, pad) if pad else _d(t) for n, t in x.items()}
    return x, pos, inv, w, dev


@pytest.mark.parametrize("T,Hq,Hk,D,R,dtype,d_dtype,interleaved,weights,pad", CASES)
def test_norm_rotate(T, Hq, Hk, D, R, dtype, d_dtype, interleaved, weights, pad):
    x, pos, inv, w, dev = _case(T, Hq, Hk, D, R, dtype, weights, pad, seed=D + T)
    got = layer.qk_norm_rotate(dev["q"], dev["k"], _d(pos) if R else None, _d(inv), _d(w["q"]), _d(w["k"]),
                               q_scale=0.25, eps=1e-5, interleaved=interleaved)
    for n, scale in (("q", 0.25), ("k", 1.0)):
        args = (_w(x[n]), _w(w[n]), scale, EPSILON, pos, inv, interleaved)
        assert got[n].dtype == dtype and got[n].is_contiguous()
        lr.assert_close(got[n], ref.norm_rotate(*args), ref.norm_rotate_bound(*args), n)


@pytest.mark.parametrize("T,Hq,Hk,D,R,dtype,d_dtype,interleaved,weights,pad", CASES)
def test_norm_rotate_backward(T, Hq, Hk, D, R, dtype, d_dtype, interleaved, weights, pad):
    x, pos, inv, w, dev = _case(T, Hq, Hk, D, R, dtype, weights, pad, seed=D + T)
    d = dict(q=_randn(T, Hq, D, seed=50, dtype=d_dtype), k=_randn(T, Hk, D, seed=51, dtype=d_dtype))
    got = layer.qk_norm_rotate_backward(dev["q"], dev["k"], _d(pos) if R else None, _d(inv), _d(w["q"]), _d(w["k"]),
                                        _d(d["q"]), _d(d["k"]), q_scale=0.25, eps=1e-5, interleaved=interleaved)
    for n, scale in (("q", 0.25), ("k", 1.0)):
        args = (_w(d[n]), _w(x[n]), _w(w[n]), scale, EPSILON, pos, inv, interleaved)
        dx, dw = ref.norm_rotate_backward(*args)
        bx, bw = ref.norm_rotate_backward_bounds(*args, heads=Hq + Hk)
        lr.assert_close(got[f"d{n}_raw"], dx, bx, f"d{n}_raw")
        assert (got[f"d{n}_weight"] is None) == (w[n] is None)
        if dw is not None:
            lr.assert_close(got[f"d{n}_weight"], dw, bw, f"d{n}_weight")


def test_rows_stay_apart():
    """A row that holds an infinity or NaN changes no other row, nor its own
    channels behind the rotation but by its mean."""
    x, pos, inv, w, dev = _case(9, 3, 2, 128, 64, F32, "qk", 0, seed=5)
    base = layer.qk_norm_rotate(dev["q"], dev["k"], _d(pos), _d(inv), _d(w["q"]), _d(w["k"]))
    dev["q"][4, 1, 100] = float("nan")
    dev["k"][3, 0, 5] = float("inf")
    got = layer.qk_norm_rotate(dev["q"], dev["k"], _d(pos), _d(inv), _d(w["q"]), _d(w["k"]))
    for n, (t, h) in dict(q=(4, 1), k=(3, 0)).items():
        assert not got[n][t, h].isfinite().all()
        got[n][t, h] = base[n][t, h]
        assert torch.equal(got[n], base[n])


def test_infinite_weight_stays_in_its_channels():
    """A weight that is infinite reaches the channels of its pair, or its own where
    nothing turns."""
    x, pos, inv, w, dev = _case(5, 2, 2, 64, 32, BF, "qk", 0, seed=6)
    w["q"][50] = float("inf")
    w["k"][3] = float("inf")
    got = layer.qk_norm_rotate(dev["q"], dev["k"], _d(pos), _d(inv), _d(w["q"]), _d(w["k"]))
    other = torch.ones(64, dtype=torch.bool)
    other[50] = False
    assert got["q"].cpu()[1:][..., other].isfinite().all()
    other[50], other[3], other[3 + 16] = True, False, False
    assert got["k"].cpu()[..., other].isfinite().all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_and_given_buffers(dtype):
    x, pos, inv, w, dev = _case(70, 3, 2, 128, 128, dtype, "qk", 0, seed=7)
    args = (_d(pos), _d(inv), _d(w["q"]), _d(w["k"]))
    want = layer.qk_norm_rotate(dev["q"], dev["k"], *args)
    out = dict(q=torch.empty_like(dev["q"]), k=torch.empty_like(dev["k"]))
    assert layer.qk_norm_rotate(dev["q"], dev["k"], *args, out=out) is out
    layer.qk_norm_rotate(dev["q"], dev["k"], *args, out=dict(q=dev["q"], k=dev["k"]))
    for n in "qk":
        assert torch.equal(out[n], want[n]) and torch.equal(dev[n], want[n])


def test_far_positions_keep_their_angle():
    """Neighbouring positions two million tokens in differ by the one turn between
    them: angles of q and k cancel but for their distance."""
    D, p0 = 64, 2_000_000
    inv = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float()
    q = _randn(1, 1, D, seed=1).expand(8, 1, D).contiguous()
    k = _randn(1, 1, D, seed=2).expand(8, 1, D).contiguous()
    near, far = (layer.qk_norm_rotate(_d(q), _d(k), _d(torch.arange(8, dtype=torch.int32) + at), _d(inv))
                 for at in (0, p0))
    # each factor is within 32 EPS of the pair's magnitude; the angles themselves are exact to 2^-30
    size = lambda o: ref._both(o.cpu().double(), inv, False)  # noqa: E731
    for d in range(8):
        a, b = ((o["q"][d:].cpu().double() * o["k"][:8 - d].cpu().double()).sum(-1) for o in (near, far))
        bound = 4 * 34 * ref.EPS * (size(near["q"])[d:] * size(near["k"])[:8 - d]).sum(-1)
        assert ((a - b).abs() <= bound).all()


def test_same_bits_and_other_streams():
    x, pos, inv, w, dev = _case(3000, 5, 2, 128, 64, BF, "qk", 8, seed=9)
    d = dict(q=_randn(3000, 5, 128, seed=50, dtype=BF).to(DEV), k=_randn(3000, 2, 128, seed=51, dtype=BF).to(DEV))
    args = (dev["q"], dev["k"], _d(pos), _d(inv), _d(w["q"]), _d(w["k"]))
    want, back = layer.qk_norm_rotate(*args), layer.qk_norm_rotate_backward(*args, d["q"], d["k"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, again = layer.qk_norm_rotate(*args, stream=side), layer.qk_norm_rotate_backward(*args, d["q"], d["k"], stream=side)
    side.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    for n in back:
        assert torch.equal(again[n], back[n]), n


def test_captured():
    """Replays follow what the inputs hold, both directions."""
    x, pos, inv, w, dev = _case(33, 4, 2, 128, 128, BF, "qk", 0, seed=11)
    d = dict(q=_randn(33, 4, 128, seed=50, dtype=BF).to(DEV), k=_randn(33, 2, 128, seed=51, dtype=BF).to(DEV))
    p, f, wq, wk = _d(pos), _d(inv), _d(w["q"]), _d(w["k"])
    args = (dev["q"], dev["k"], p, f, wq, wk)
    layer.qk_norm_rotate(*args), layer.qk_norm_rotate_backward(*args, d["q"], d["k"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, back = layer.qk_norm_rotate(*args), layer.qk_norm_rotate_backward(*args, d["q"], d["k"])
    for i in range(3):
        dev["q"].copy_(_randn(33, 4, 128, seed=60 + i, dtype=BF))
        p.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        want, wanted = layer.qk_norm_rotate(*args), layer.qk_norm_rotate_backward(*args, d["q"], d["k"])
        for a, b in ((got, want), (back, wanted)):
            for n in a:
                assert torch.equal(a[n], b[n]), (i, n)


def test_beyond_32_bit_offsets():
    """Rows behind element 2^31 of a wide projection."""
    T, wide = 70_000, 40_000
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 8 GB")
    row = torch.zeros(T, wide, dtype=BF, device=DEV)
    q, k = row[:, :256].view(T, 2, 128), row[:, 256:384].view(T, 1, 128)
    q.copy_(_randn(T, 2, 128, seed=1, dtype=BF))
    k.copy_(_randn(T, 1, 128, seed=2, dtype=BF))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV)
    got = layer.qk_norm_rotate(q, k, pos, inv)
    want = layer.qk_norm_rotate(q[-64:].contiguous(), k[-64:].contiguous(), pos[-64:].contiguous(), inv)
    for n in "qk":
        assert torch.equal(got[n][-64:], want[n])


def test_refusals():
    q, k = _randn(4, 2, 64, seed=1, dtype=BF).to(DEV), _randn(4, 1, 64, seed=2, dtype=BF).to(DEV)
    pos, inv = torch.arange(4, dtype=torch.int32, device=DEV), torch.ones(16, device=DEV)
    with pytest.raises(ValueError, match="positions"):
        layer.qk_norm_rotate(q, k, None, inv)
    with pytest.raises(TypeError, match="positions"):
        layer.qk_norm_rotate(q, k, pos.long(), inv)
    with pytest.raises(TypeError, match="k_raw"):
        layer.qk_norm_rotate(q, k.float(), pos, inv)
    with pytest.raises(ValueError, match="k_raw"):
        layer.qk_norm_rotate(q, k[:, :, :32].contiguous(), pos, inv)
    with pytest.raises(ValueError, match="cpu"):
        layer.qk_norm_rotate(q, k, pos.cpu(), inv)
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        layer.qk_norm_rotate(q, k, pos, torch.ones(33, device=DEV))
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        layer.qk_norm_rotate(q, k, pos, inv, eps=0.0)
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        layer.qk_norm_rotate(q[:0], k[:0], pos[:0], inv)
    wide = _randn(4, 2, 264, seed=1, dtype=BF).to(DEV)
    with pytest.raises(kda.KdaError, match="UNSUPPORTED"):
        layer.qk_norm_rotate(wide, wide, pos, inv)
    with pytest.raises(ValueError, match="dk"):
        layer.qk_norm_rotate_backward(q, k, pos, inv, None, None, q, q)
    with pytest.raises(TypeError, match="dk"):
        layer.qk_norm_rotate_backward(q, k, pos, inv, None, None, q, k.float())
