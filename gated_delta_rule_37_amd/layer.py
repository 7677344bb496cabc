"""Thin Python binding of the operators around the KDA recurrence.

What one layer runs before and after :func:`kda.forward`, its form for single
tokens, and a recurrence with one state per channel; argument marshalling only,
as in :mod:`.kda` (the kernels are behind ``include/kda.h``, which states each
formula).  Entry points mirror the C names:

* :func:`prepare_inputs`, :func:`prepare_inputs_backward`
  (``kda_prepare_inputs``, ``kda_prepare_inputs_backward``): a layer's raw
  projections to q, k, g and beta
* :func:`output_norm`, :func:`output_norm_backward` (``kda_output_norm``,
  ``kda_output_norm_backward``): the norm of o with its gate, residual and scale
* :func:`scan_forward`, :func:`scan_backward` (``kda_scan_forward``,
  ``kda_scan_backward``): h_t = exp(g_t) h_{t-1} + u_t per channel over packed
  sequences; any plan serves, and one that only they use needs one segment
  (:func:`scan_segments`)
* :func:`scan_step` (``kda_scan_step``) and :func:`step` (``kda_step``): single
  tokens over a pool of states
* :func:`qk_norm_rotate`, :func:`qk_norm_rotate_backward`
  (``kda_qk_norm_rotate``, ``kda_qk_norm_rotate_backward``): queries and keys
  normed per head and turned by their positions
* :func:`linear_forward`, :func:`linear_backward` (``kda_linear_forward``,
  ``kda_linear_backward``): linear attention with a decay for each head over
  packed sequences; any plan serves, :func:`linear_segments` counts the segments
  of one that only they use
* :func:`linear_step` (``kda_linear_step``): its single tokens over a pool of states

A training step of one layer::

    x = layer.prepare_inputs(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias)
    f = kda.forward(plan, x["q"], x["k"], v, x["g"], x["beta"])
    y = layer.output_norm(f["o"], weight, gate=z, activation="sigmoid")
    ...
    n = layer.output_norm_backward(dy, f["o"], weight, gate=z, activation="sigmoid")
    b = kda.backward(plan, x["q"], x["k"], v, x["g"], x["beta"], n["d_o"])
    r = layer.prepare_inputs_backward(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias,
                                      b["dq"], b["dk"], b["dg"], b["dbeta"])

and a decoding step, with ``state`` a pool laid out as kda.forward's
final_state::

    x = layer.prepare_inputs(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias)
    o = layer.step(x["q"], x["k"], v, x["g"], x["beta"], state, slots)
    y = layer.output_norm(o, weight, gate=z, activation="sigmoid")

A layer of linear attention, trained and decoded the same way::

    plan = kda.Plan(cu_seqlens, layer.linear_segments(cu_seqlens, H))
    x = layer.qk_norm_rotate(q_raw, k_raw, positions, inv_freq, q_weight, k_weight, q_scale=K ** -0.5)
    f = layer.linear_forward(plan, x["q"], x["k"], v, g)
    y = layer.output_norm(f["o"], weight, gate=z, activation="silu")
    ...
    n = layer.output_norm_backward(dy, f["o"], weight, gate=z, activation="silu", d_o_dtype=torch.bfloat16)
    b = layer.linear_backward(plan, x["q"], x["k"], v, g, n["d_o"])
    r = layer.qk_norm_rotate_backward(q_raw, k_raw, positions, inv_freq, q_weight, k_weight, b["dq"], b["dk"],
                                      q_scale=K ** -0.5)

    o = layer.linear_step(x["q"], x["k"], v, g, state, slots)     # decoding, state as final_state

Every call enqueues on ``stream`` (default: the current stream of its tensors'
device) and returns without waiting; what it allocates belongs to that stream,
and a plan's device copy waits for it (``Plan.device_blob``, which a capture of
a scan or of linear attention needs called before).  A tensor on another device than the rest raises
ValueError.
"""
from __future__ import annotations

import math

import torch

from . import kda

# element types (kda_dtype) and activations (kda_activation)
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2}

_NULL = (None, 0)
_NULL_ROWS = (None, 0, 0)


def _dtype(t: torch.Tensor, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected one of {list(DTYPES)}, got {t.dtype}")
    return code


# The checks below run on every call, which for one token is most of its time:
# they ask each tensor for as little as they can.
def _buf(t, dtype, shape, name, device):
    """(address, size in bytes) of a dense tensor on ``device``."""
    if t is None:
        return _NULL
    if t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return (t.data_ptr(), t.nbytes)
    raise _refusal(t, dtype, shape, name, device) or ValueError(f"{name}: must be contiguous")


def _refusal(t, dtype, shape, name, device):
    """The error for a tensor of another type, shape or device, else None."""
    if t.dtype != dtype:
        return TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        return ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        return ValueError(f"{name}: on {t.device}, the other tensors on {device}")
    return None


def _made(t):
    """(address, size in bytes) of an output that the call itself allocated."""
    return _NULL if t is None else (t.data_ptr(), t.nbytes)


def _row_stride(t, name):
    """The elements from row t[i] to the next one of a tensor whose rows are
    dense and do not overlap (a slice of a wider tensor's rows)."""
    row = t.numel() // t.shape[0] if t.shape[0] else 0
    if t.is_contiguous():
        return row
    stride = t.stride(0) if t.shape[0] > 1 else row
    if stride < row or not t[0].is_contiguous():
        raise ValueError(f"{name}: rows must be dense and must not overlap")
    return stride


def _rows(t, dtype, shape, name, device):
    """(address, size in bytes, token stride) of a tensor of rows."""
    if t is None:
        return _NULL_ROWS
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise _refusal(t, dtype, shape, name, device)
    n = shape[0]
    if n and t.is_contiguous():
        return (t.data_ptr(), t.nbytes, t.numel() // n)
    strides, row = t.stride(), 1
    for i in range(len(shape) - 1, 0, -1):
        if strides[i] != row:
            break
        row *= shape[i]
    else:   # slices of a wider tensor's rows, the usual case
        if n > 1 and strides[0] >= row:
            return (t.data_ptr(), ((n - 1) * strides[0] + row) * dtype.itemsize, strides[0])
    stride = _row_stride(t, name)
    span = (n - 1) * stride + t.numel() // n if n else 0
    return (t.data_ptr(), span * t.element_size(), stride)


_functions = {}


def _call(name, device, args, stream):
    """One C call on ``stream``, with the tensors' device current."""
    if device.type != "cuda":
        raise ValueError(f"{name}: needs device tensors")
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(kda.lib(), name)
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != 0:
        raise kda.KdaError(status, name)


def _raw(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias, q_scale, eps):
    """T, H, K, the device and the arguments that both directions of the input
    preparation share."""
    T, H, K = q_raw.shape
    dt, dev = q_raw.dtype, q_raw.device
    args = [T, H, K, _dtype(q_raw, "q_raw"),
            *_rows(q_raw, dt, (T, H, K), "q_raw", dev), *_rows(k_raw, dt, (T, H, K), "k_raw", dev),
            *_rows(gate_raw, dt, (T, H, K), "gate_raw", dev), *_rows(beta_raw, dt, (T, H), "beta_raw", dev),
            *_buf(a_log, torch.float32, (H,), "a_log", dev), *_buf(dt_bias, torch.float32, (H, K), "dt_bias", dev),
            float(q_scale), float(eps)]
    return T, H, K, dev, args


def prepare_inputs(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias=None, q_scale=1.0, eps=1e-6, out=None,
                   stream=None):
    """``kda_prepare_inputs``: q and k normalised per head (q times ``q_scale``),
    g = -exp(a_log) softplus(gate_raw + dt_bias), beta = sigmoid(beta_raw), all
    bf16, as dict(q, k, g, beta).  The raw inputs are [T, H, K] (beta_raw
    [T, H]) in bf16 or fp32; their rows may be slices of a wider projection.
    ``out`` gives the buffers to write."""
    T, H, K, dev, args = _raw(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias, q_scale, eps)
    bf = torch.bfloat16
    if out is None:
        out = {n: _empty(stream, dev, bf, T, H, K) for n in ("q", "k", "g")}
        out["beta"] = _empty(stream, dev, bf, T, H)
        for t in out.values():
            args += _made(t)
    else:
        for n in ("q", "k", "g"):
            args += _buf(out[n], bf, (T, H, K), n, dev)
        args += _buf(out["beta"], bf, (T, H), "beta", dev)
    _call("kda_prepare_inputs", dev, args, stream)
    return out


def prepare_inputs_backward(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias, dq, dk, dg, dbeta, q_scale=1.0,
                            eps=1e-6, stream=None):
    """``kda_prepare_inputs_backward``: from the recurrence's gradients (fp32, as
    :func:`kda.backward` returns them) those of the raw inputs (their dtype) and
    parameters (fp32): dict(dq_raw, dk_raw, dgate_raw, dbeta_raw, da_log,
    ddt_bias), ddt_bias None without dt_bias."""
    T, H, K, dev, args = _raw(q_raw, k_raw, gate_raw, beta_raw, a_log, dt_bias, q_scale, eps)
    f32, dt = torch.float32, q_raw.dtype
    for n, t in (("dq", dq), ("dk", dk), ("dg", dg)):
        args += _buf(t, f32, (T, H, K), n, dev)
    args += _buf(dbeta, f32, (T, H), "dbeta", dev)
    out = {n: _empty(stream, dev, dt, T, H, K) for n in ("dq_raw", "dk_raw", "dgate_raw")}
    out["dbeta_raw"] = _empty(stream, dev, dt, T, H)
    out["da_log"] = _empty(stream, dev, f32, H)
    out["ddt_bias"] = None if dt_bias is None else _empty(stream, dev, f32, H, K)
    for n in ("dq_raw", "dk_raw", "dgate_raw", "dbeta_raw", "da_log", "ddt_bias"):
        args += _made(out[n])
    workspace = _scratch(kda.lib().kda_prepare_inputs_backward_workspace_bytes(T, H, K), dev, stream)
    args += _made(workspace)
    _call("kda_prepare_inputs_backward", dev, args, stream)
    return out


def _rotate(q_raw, k_raw, positions, inv_freq, q_weight, k_weight, q_scale, eps, interleaved):
    """The two inputs' shapes, the device and the arguments that both directions
    of the norms and rotation share."""
    T, Hq, D = q_raw.shape
    Hk, dt, dev, f32 = k_raw.shape[1], q_raw.dtype, q_raw.device, torch.float32
    pairs = 0 if inv_freq is None else inv_freq.shape[0]
    if pairs and positions is None:
        raise ValueError("positions: needed with inv_freq")
    args = [T, Hq, Hk, D, 2 * pairs, _dtype(q_raw, "q_raw"), int(bool(interleaved)),
            *_rows(q_raw, dt, (T, Hq, D), "q_raw", dev), *_rows(k_raw, dt, (T, Hk, D), "k_raw", dev),
            *_buf(positions, torch.int32, (T,), "positions", dev), *_buf(inv_freq, f32, (pairs,), "inv_freq", dev),
            *_buf(q_weight, f32, (D,), "q_weight", dev), *_buf(k_weight, f32, (D,), "k_weight", dev),
            float(q_scale), float(eps)]
    return (T, Hq, D), (T, Hk, D), dev, args


def qk_norm_rotate(q_raw, k_raw, positions=None, inv_freq=None, q_weight=None, k_weight=None, q_scale=1.0, eps=1e-6,
                   interleaved=False, out=None, stream=None):
    """``kda_qk_norm_rotate``: q_raw [T, Hq, D] and k_raw [T, Hk, D] (bf16 or
    fp32; rows may be slices of a wider projection) divided by their root mean
    square per head, times their weight [D] (q also times ``q_scale``), then their
    first 2 len(inv_freq) channels turned by positions (int32 [T]) times
    ``inv_freq`` (fp32): channels (i, i + len(inv_freq)) are a pair, or
    (2 i, 2 i + 1) when ``interleaved``.  Without inv_freq nothing turns.  Returns
    dict(q, k) in the inputs' dtype; ``out`` gives the buffers, which may be
    dense inputs themselves."""
    q_shape, k_shape, dev, args = _rotate(q_raw, k_raw, positions, inv_freq, q_weight, k_weight, q_scale, eps,
                                          interleaved)
    dt = q_raw.dtype
    if out is None:
        out = dict(q=_empty(stream, dev, dt, *q_shape), k=_empty(stream, dev, dt, *k_shape))
        args += [*_made(out["q"]), *_made(out["k"])]
    else:
        args += [*_buf(out["q"], dt, q_shape, "q", dev), *_buf(out["k"], dt, k_shape, "k", dev)]
    _call("kda_qk_norm_rotate", dev, args, stream)
    return out


def qk_norm_rotate_backward(q_raw, k_raw, positions, inv_freq, q_weight, k_weight, dq, dk, q_scale=1.0, eps=1e-6,
                            interleaved=False, stream=None):
    """``kda_qk_norm_rotate_backward``: from the gradients of q and k (bf16 or fp32,
    both the same) those of the raw inputs (their dtype) and of the weights (fp32,
    None without them): dict(dq_raw, dk_raw, dq_weight, dk_weight)."""
    q_shape, k_shape, dev, args = _rotate(q_raw, k_raw, positions, inv_freq, q_weight, k_weight, q_scale, eps,
                                          interleaved)
    dt, D, f32 = q_raw.dtype, q_shape[2], torch.float32
    args += [*_buf(dq, dq.dtype, q_shape, "dq", dev), *_buf(dk, dq.dtype, k_shape, "dk", dev), _dtype(dq, "dq")]
    out = dict(dq_raw=_empty(stream, dev, dt, *q_shape), dk_raw=_empty(stream, dev, dt, *k_shape),
               dq_weight=None if q_weight is None else _empty(stream, dev, f32, D),
               dk_weight=None if k_weight is None else _empty(stream, dev, f32, D))
    for t in out.values():
        args += _made(t)
    weights = q_weight is not None or k_weight is not None
    size = kda.lib().kda_qk_norm_rotate_backward_workspace_bytes(q_shape[0], D) if weights else 0
    workspace = _scratch(size, dev, stream)
    args += _made(workspace)
    _call("kda_qk_norm_rotate_backward", dev, args, stream)
    return out


def _empty(stream, device, dtype, *shape):
    """Uninitialised memory of the call's stream."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with kda._allocating_on(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _scratch(size, device, stream):
    """A workspace of ``size`` bytes for one call, or None.  The caller keeps it
    until the C call has returned: only what is enqueued is in stream order, and
    another thread may allocate on the same stream while the call runs."""
    return None if size == 0 else _empty(stream, device, torch.uint8, size)


def _norm(o, weight, gate, activation, res_scale, dtype):
    T, H, V = o.shape
    dev = o.device
    code = ACTIVATIONS.get(activation if gate is not None else "none")
    if code is None:
        raise ValueError(f"activation: expected one of {list(ACTIVATIONS)}, got {activation!r}")
    if gate is not None and code == 0:
        raise ValueError("gate given without an activation")
    gated = [*_rows(gate, dtype, (T, H, V), "gate", dev), code]
    weights = [*_buf(weight, torch.float32, (V,), "weight", dev),
               *_buf(res_scale, torch.float32, (H, V), "res_scale", dev)]
    return T, H, V, dev, gated, weights


def output_norm(o, weight, gate=None, activation="sigmoid", res_scale=None, residual=None, eps=1e-6, dtype=None,
                out=None, stream=None):
    """``kda_output_norm``: residual + res_scale act(gate) weight o / rms(o) per
    (token, head) row of o [T, H, V] (fp32 or bf16).  ``activation`` is "sigmoid"
    or "silu"; ``gate`` None means no gate.  The result has the dtype of gate or
    residual, else ``dtype`` (default: o's); ``out`` gives the buffer, which may
    be the residual itself."""
    for t in (gate, residual, out):
        if t is not None:
            if dtype is not None and t.dtype != dtype:
                raise TypeError(f"gate, residual and out: expected {dtype}, got {t.dtype}")
            dtype = t.dtype
    if dtype is None:
        dtype = o.dtype
    T, H, V, dev, gated, weights = _norm(o, weight, gate, activation, res_scale, dtype)
    if dtype not in DTYPES:
        raise TypeError(f"dtype: expected one of {list(DTYPES)}, got {dtype}")
    if out is None:
        out = _empty(stream, dev, dtype, T, H, V)
    args = [T, H, V, *_buf(o, o.dtype, (T, H, V), "o", dev), _dtype(o, "o"), *gated, *weights,
            *_buf(residual, dtype, (T, H, V), "residual", dev), DTYPES[dtype], float(eps),
            *_buf(out, dtype, (T, H, V), "out", dev)]
    _call("kda_output_norm", dev, args, stream)
    return out


def output_norm_backward(dy, o, weight, gate=None, activation="sigmoid", res_scale=None, eps=1e-6,
                         d_o_dtype=torch.float32, stream=None):
    """``kda_output_norm_backward``: gradients for the cotangent dy as dict(d_o,
    d_gate, d_weight, d_res_scale), those of absent inputs None; the residual's
    gradient is dy.  d_o is fp32, as :func:`kda.backward` takes it, unless
    ``d_o_dtype`` says bfloat16."""
    dtype = dy.dtype
    T, H, V, dev, gated, weights = _norm(o, weight, gate, activation, res_scale, dtype)
    if d_o_dtype not in DTYPES:
        raise TypeError(f"d_o_dtype: expected one of {list(DTYPES)}, got {d_o_dtype}")
    f32 = torch.float32
    out = dict(d_o=_empty(stream, dev, d_o_dtype, T, H, V),
               d_gate=None if gate is None else _empty(stream, dev, dtype, T, H, V),
               d_weight=_empty(stream, dev, f32, V),
               d_res_scale=None if res_scale is None else _empty(stream, dev, f32, H, V))
    workspace = _scratch(kda.lib().kda_output_norm_backward_workspace_bytes(T, H, V), dev, stream)
    args = [T, H, V, *_buf(dy, dtype, (T, H, V), "dy", dev), *_buf(o, o.dtype, (T, H, V), "o", dev), _dtype(o, "o"),
            *gated, *weights, _dtype(dy, "dy"), float(eps), *_made(out["d_o"]),
            DTYPES[d_o_dtype], *_made(out["d_gate"]),
            *_made(out["d_weight"]), *_made(out["d_res_scale"]), *_made(workspace)]
    _call("kda_output_norm_backward", dev, args, stream)
    return out


def scan_segments(cu_seqlens, D: int) -> int:
    """The segment count for a plan that only the scan uses: the scan cuts the
    tokens into tiles by itself, whatever the plan's segments are, so one."""
    return 1


def _scan(plan, x, g, initial_state, tied, stream):
    T, D = g.shape
    if T != plan.T:
        raise ValueError(f"inputs hold {T} tokens, the plan {plan.T}")
    dt, dev = g.dtype, g.device
    blob = plan.device_blob(dev, stream)
    args = [plan.handle, *_buf(blob, torch.int32, (len(plan.blob),), "plan_dev", dev), D, _dtype(g, "g"),
            *_rows(x, dt, (T, D), "x", dev), *_rows(g, dt, (T, D), "g", dev), int(bool(tied)),
            *_buf(initial_state, torch.float32, (plan.N, D), "initial_state", dev)]
    return T, D, dev, args


def scan_forward(plan: kda.Plan, x, g, initial_state=None, tied=False, h_dtype=None, out=None, stream=None):
    """``kda_scan_forward``: h_t = exp(g_t) h_{t-1} + x_t, or + (1 - exp(g_t)) x_t
    when ``tied``, for x and g [T, D] (bf16 or fp32), every sequence of the plan
    from its ``initial_state`` [N, D] (default: zero).  Returns dict(h,
    final_state), h in ``h_dtype`` (default: x's), final_state fp32."""
    T, D, dev, args = _scan(plan, x, g, initial_state, tied, stream)
    if out is None:
        out = dict(h=_empty(stream, dev, g.dtype if h_dtype is None else h_dtype, T, D),
                   final_state=_empty(stream, dev, torch.float32, plan.N, D))
    h = out["h"]
    workspace = _scratch(kda.lib().kda_scan_workspace_bytes(plan.handle, D), dev, stream)
    args += [*_buf(h, h.dtype, (T, D), "h", dev), _dtype(h, "h"),
             *_buf(out["final_state"], torch.float32, (plan.N, D), "final_state", dev),
             *_made(workspace)]
    _call("kda_scan_forward", dev, args, stream)
    return out


def scan_backward(plan: kda.Plan, x, g, h, dh, d_final=None, initial_state=None, tied=False, want_dh0=None,
                  stream=None):
    """``kda_scan_backward``: gradients for the cotangents ``dh`` (in h's dtype) and
    ``d_final`` [N, D] (default: zero) as dict(dx, dg, dh0).  ``h`` is what the
    forward wrote; x is only read when ``tied``.  dh0 (fp32) is None unless
    ``want_dh0`` (default: whether there are initial states)."""
    T, D, dev, args = _scan(plan, x if tied else None, g, initial_state, tied, stream)
    f32 = torch.float32
    want = initial_state is not None if want_dh0 is None else want_dh0
    out = dict(dx=_empty(stream, dev, g.dtype, T, D), dg=_empty(stream, dev, g.dtype, T, D),
               dh0=_empty(stream, dev, f32, plan.N, D) if want else None)
    workspace = _scratch(kda.lib().kda_scan_workspace_bytes(plan.handle, D), dev, stream)
    args += [*_buf(h, h.dtype, (T, D), "h", dev), *_buf(dh, h.dtype, (T, D), "dh", dev), _dtype(h, "h"),
             *_buf(d_final, f32, (plan.N, D), "d_final", dev), *_made(out["dx"]),
             *_made(out["dg"]), *_made(out["dh0"]), *_made(workspace)]
    _call("kda_scan_backward", dev, args, stream)
    return out


def _pool(B, state, slots, state_out, tail, dev):
    """num_slots, the slots' buffer and those of the pool before and after."""
    if state_out is None:
        state_out = state
    shape = (state.shape[0], *tail)
    return state.shape[0], _buf(slots, torch.int32, (B,), "slots", dev), [
        *_buf(state, torch.float32, shape, "state", dev), *_buf(state_out, torch.float32, shape, "state_out", dev)]


def scan_step(x, g, state, slots=None, state_out=None, h=None, tied=False, stream=None):
    """``kda_scan_step``: the next token of B sequences, x and g [B, D], whose
    states lie in the rows ``slots`` (int32 [B], default: row b) of ``state``
    [num_slots, D] fp32, updated in place unless ``state_out`` is given.  A slot
    outside the pool marks an unused row.  Returns h [B, D] in x's dtype
    (``h``: the buffer to write)."""
    B, D = x.shape
    dt, dev = x.dtype, x.device
    if h is None:
        h = _empty(stream, dev, dt, B, D)
    n, slots, pool = _pool(B, state, slots, state_out, (D,), dev)
    args = [B, D, _dtype(x, "x"), *_buf(x, dt, (B, D), "x", dev), *_buf(g, dt, (B, D), "g", dev), int(bool(tied)),
            *slots, n, *pool, *_buf(h, dt, (B, D), "h", dev)]
    _call("kda_scan_step", dev, args, stream)
    return h


def step(q, k, v, g, beta, state, slots=None, state_out=None, o=None, o_dtype=torch.float32, gate_lower_bound=None,
         heads=None, stream=None):
    """``kda_step``: the next token of B sequences, q, k, g [B, H, K], v [B, H, V]
    and beta [B, H] (bf16, as :func:`prepare_inputs` makes them), whose states
    lie in the slots ``slots`` (int32 [B], default: slot b) of ``state``
    [num_slots, H, K, V] fp32, updated in place unless ``state_out`` is given.  A
    slot outside the pool marks an unused row.  Returns o [B, H, V] in
    ``o_dtype`` (``o``: the buffer to write)."""
    B, H, K = k.shape
    V = v.shape[2]
    bf, dev = torch.bfloat16, k.device
    if o is None:
        o = _empty(stream, dev, o_dtype, B, H, V)
    n, slots, pool = _pool(B, state, slots, state_out, (H, K, V), dev)
    bound = float("-inf") if gate_lower_bound is None else float(gate_lower_bound)
    args = [B, H, K, V, *kda._heads(H, heads), *_buf(q, bf, (B, H, K), "q", dev), *_buf(k, bf, (B, H, K), "k", dev),
            *_buf(v, bf, (B, H, V), "v", dev), *_buf(g, bf, (B, H, K), "g", dev), *_buf(beta, bf, (B, H), "beta", dev),
            bound, *slots, n, *pool, *_buf(o, o.dtype, (B, H, V), "o", dev), _dtype(o, "o")]
    _call("kda_step", dev, args, stream)
    return o


def _linear_heads(q, k, v, g):
    """H, Hq, Hk, Hv, K, V: as many states as the most heads of q, k, v and g."""
    Hq, K = q.shape[1:]
    Hk, (Hv, V) = k.shape[1], v.shape[1:]
    return max(Hq, Hk, Hv, g.shape[-1]), Hq, Hk, Hv, K, V


def linear_segments(cu_seqlens, H: int) -> int:
    """The segment count for a plan that only linear attention with ``H`` heads
    uses; one where the sequences are short enough as they are.  A segment and head
    is a workgroup's work, chunk of 64 tokens after chunk, and 512 of them run at
    once: more than 512 segments and heads take a second turn.  Whole chunks are
    shared out, as a part of one costs as much (gradients of 1501 tokens x 6 heads: 8
    segments of 3 chunks 51 us, 12 of 2 45, 24 of 1 46), and no more than 5
    sqrt(chunks), as each segment lengthens the ordered scan between them (8192 x 8: 32
    segments 60 us, 64 76, 128 111; 65536 x 1: 73 134, 147 115, 512 229).  One sequence
    of 65536 x 32: 8 segments 904 us, 16 812, 32 841; gradients of 16384 x 32: 779,
    741, 797.  Of 16384 tokens x 16: 24 equal sequences uncut 64 us, in 32 segments 91,
    24 with one of 2790 179 and 94, 64 with one of 1265 88 and 94."""
    T = int(cu_seqlens[-1])
    chunks = -(-T // 64)
    if chunks < 4:   # 100 tokens in two 25 us for 16, their gradients 47 for 49
        return 1
    S = -(-chunks // math.ceil(chunks / min(-(-512 // H), 5 * math.sqrt(chunks))))
    longest = max(int(b) - int(a) for a, b in zip(cu_seqlens, cu_seqlens[1:]))
    uneven = 1.5 if (len(cu_seqlens) - 1) * H <= 512 else 3   # sequences that fill the GPU as they are
    return S if S > 1 and longest * S > uneven * T else 1


def _linear(plan, q, k, v, g, initial_state, stream):
    """H, the other sizes, the device and the arguments that both directions share."""
    H, Hq, Hk, Hv, K, V = sizes = _linear_heads(q, k, v, g)
    T, bf, dev = q.shape[0], torch.bfloat16, q.device
    if T != plan.T:
        raise ValueError(f"inputs hold {T} tokens, the plan {plan.T}")
    blob = plan.device_blob(dev, stream)
    gates = (*_buf(g, g.dtype, (H,), "g", dev), 0) if g.dim() == 1 else _rows(g, g.dtype, (T, H), "g", dev)
    args = [plan.handle, *_buf(blob, torch.int32, (len(plan.blob),), "plan_dev", dev), *sizes,
            *_rows(q, bf, (T, Hq, K), "q", dev), *_rows(k, bf, (T, Hk, K), "k", dev), *_rows(v, bf, (T, Hv, V), "v", dev),
            *gates, _dtype(g, "g"), *_buf(initial_state, torch.float32, (plan.N, H, K, V), "initial_state", dev)]
    return T, sizes, dev, args


def linear_forward(plan: kda.Plan, q, k, v, g, initial_state=None, o_dtype=torch.bfloat16, out=None, stream=None):
    """``kda_linear_forward``: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t for
    q [T, Hq, K], k [T, Hk, K], v [T, Hv, V] bf16 (rows may be slices of a wider
    projection) and g [T, H] or [H] (fp32 or bf16), every sequence of the plan from
    its ``initial_state`` [N, H, K, V] (default: zero).  There are as many states,
    H, as the most heads of q, k, v and g; a tensor of fewer heads is shared by
    neighbours.  The plan's pieces run in parallel (:func:`linear_segments`).
    Returns dict(o, final_state), o [T, H, V] in ``o_dtype``, final_state fp32."""
    T, (H, Hq, Hk, Hv, K, V), dev, args = _linear(plan, q, k, v, g, initial_state, stream)
    f32 = torch.float32
    if out is None:
        out = dict(o=_empty(stream, dev, o_dtype, T, H, V), final_state=_empty(stream, dev, f32, plan.N, H, K, V))
    o = out["o"]
    workspace = _scratch(kda.lib().kda_linear_workspace_bytes(plan.handle, H, K, V), dev, stream)
    args += [*_buf(o, o.dtype, (T, H, V), "o", dev), _dtype(o, "o"),
             *_buf(out["final_state"], f32, (plan.N, H, K, V), "final_state", dev), *_made(workspace)]
    _call("kda_linear_forward", dev, args, stream)
    return out


def linear_backward(plan: kda.Plan, q, k, v, g, d_o, d_final=None, initial_state=None, want_dh0=None,
                    grad_dtype=torch.bfloat16, stream=None):
    """``kda_linear_backward``: gradients for the cotangents ``d_o`` [T, H, V] (bf16)
    and ``d_final`` [N, H, K, V] (fp32, default: zero) as dict(dq, dk, dv, dg, dh0):
    dq, dk and dv in ``grad_dtype``, dg like g, dh0 (fp32) None unless ``want_dh0``
    (default: whether there are initial states)."""
    T, (H, Hq, Hk, Hv, K, V), dev, args = _linear(plan, q, k, v, g, initial_state, stream)
    if grad_dtype not in DTYPES:
        raise TypeError(f"grad_dtype: expected one of {list(DTYPES)}, got {grad_dtype}")
    f32, state = torch.float32, (plan.N, H, K, V)
    want = initial_state is not None if want_dh0 is None else want_dh0
    out = dict(dq=_empty(stream, dev, grad_dtype, T, Hq, K), dk=_empty(stream, dev, grad_dtype, T, Hk, K),
               dv=_empty(stream, dev, grad_dtype, T, Hv, V), dg=_empty(stream, dev, g.dtype, *g.shape),
               dh0=_empty(stream, dev, f32, *state) if want else None)
    workspace = _scratch(kda.lib().kda_linear_backward_workspace_bytes(plan.handle, H, Hq, Hk, Hv, K, V), dev, stream)
    args += [*_buf(d_o, torch.bfloat16, (T, H, V), "d_o", dev), *_buf(d_final, f32, state, "d_final", dev),
             *_made(out["dq"]), *_made(out["dk"]), *_made(out["dv"]), DTYPES[grad_dtype], *_made(out["dg"]),
             *_made(out["dh0"]), *_made(workspace)]
    _call("kda_linear_backward", dev, args, stream)
    return out


def linear_step(q, k, v, g, state, slots=None, state_out=None, o=None, o_dtype=torch.bfloat16, stream=None):
    """``kda_linear_step``: the next token of B sequences, q [B, Hq, K], k [B, Hk, K]
    and v [B, Hv, V] bf16, g [B, H] or [H] (fp32 or bf16), whose states lie in the
    slots ``slots`` (int32 [B], default: slot b) of ``state`` [num_slots, H, K, V]
    fp32, updated in place unless ``state_out`` is given.  A slot outside the pool
    marks an unused row.  Returns o [B, H, V] in ``o_dtype`` (``o``: the buffer to
    write)."""
    B = q.shape[0]
    H, Hq, Hk, Hv, K, V = _linear_heads(q, k, v, g)
    bf, dev = torch.bfloat16, q.device
    if o is None:
        o = _empty(stream, dev, o_dtype, B, H, V)
    n, slots, pool = _pool(B, state, slots, state_out, (H, K, V), dev)
    fixed = g.dim() == 1
    args = [B, H, Hq, Hk, Hv, K, V, *_buf(q, bf, (B, Hq, K), "q", dev), *_buf(k, bf, (B, Hk, K), "k", dev),
            *_buf(v, bf, (B, Hv, V), "v", dev), *_buf(g, g.dtype, (H,) if fixed else (B, H), "g", dev),
            0 if fixed else H, _dtype(g, "g"), *slots, n, *pool, *_buf(o, o.dtype, (B, H, V), "o", dev), _dtype(o, "o")]
    _call("kda_linear_step", dev, args, stream)
    return o
