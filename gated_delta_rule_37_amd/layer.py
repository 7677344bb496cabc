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

Every call enqueues on ``stream`` (default: the current stream of its tensors'
device) and returns without waiting; what it allocates belongs to that stream,
and a plan's device copy waits for it (``Plan.device_blob``, which a capture of
a scan needs called before).  A tensor on another device than the rest raises
ValueError.
"""
from __future__ import annotations

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
