"""Cases and plain forms of linear attention with a decay for each head, and of the norms and rotation before it.

* ``rotate``: the norms of queries and keys per head and their rotation by position in one pass
  (``layer.qk_norm_rotate`` and its backward).  Per (token, head) row x of D channels n = weight x /
  sqrt(mean(x^2) + eps), q also times q_scale; then the first R channels turn in pairs by position * inv_freq.
* ``linear``: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over packed sequences
  (``layer.linear_forward``, ``layer.linear_backward``), g one number for a token and head, or for a head.
  q, k and v may have fewer heads than the states: head h reads head h // (H // heads).
* ``linear_step``: the same for single tokens over state slots (``layer.linear_step``).

``own`` says whether ``run`` makes the framework's calls or computes the plain form.
"""
import random

import torch

own = False

EPS = 1e-6
CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # decoding eight sequences at far positions: the call's latency counts
        dict(name="rotate_decode_8x8", op="rotate", dir="fwd", T=8, Hq=8, Hk=2, D=128, R=128, dtype="bf16",
             d="bf16", interleaved=False, weight=True, strided=True),
        # a long packed batch, queries and keys slices of one projection, key heads shared
        dict(name="rotate_fwd_32768x32", op="rotate", dir="fwd", T=32768, Hq=32, Hk=8, D=128, R=128, dtype="bf16",
             d="bf16", interleaved=False, weight=True, strided=True),
        # a training step's gradients, half of the channels turned, of an odd length
        dict(name="rotate_bwd_8191x16", op="rotate", dir="bwd", T=8191, Hq=16, Hk=16, D=128, R=64, dtype="bf16",
             d="bf16", interleaved=False, weight=True, strided=False),
        # 32 bits, heads of an odd width, neighbouring channels paired
        dict(name="rotate_fwd_odd_1021x5", op="rotate", dir="fwd", T=1021, Hq=5, Hk=5, D=80, R=40, dtype="fp32",
             d="fp32", interleaved=True, weight=True, strided=False),
        # a short prompt of one sequence with fixed decays: latency
        dict(name="linear_fwd_100x4", op="linear", dir="fwd", T=100, N=1, H=4, Hq=4, Hk=4, Hv=4, K=128, V=128,
             g="head", o="bf16", init=False, strided=False),
        # the longest prompt: one sequence
        dict(name="linear_fwd_65536x32", op="linear", dir="fwd", T=65536, N=1, H=32, Hq=32, Hk=32, Hv=32, K=128,
             V=128, g="fp32", o="bf16", init=False, strided=True),
        # prompts that arrive together and go on from cached states, query and key heads shared by 8 value heads
        dict(name="linear_fwd_packed_16384x16", op="linear", dir="fwd", T=16384, N=24, H=16, Hq=2, Hk=2, Hv=16,
             K=128, V=64, g="fp32", o="bf16", init=True, strided=False),
        # a training step of a packed batch
        dict(name="linear_bwd_16384x32", op="linear", dir="bwd", T=16384, N=4, H=32, Hq=32, Hk=32, Hv=32, K=128,
             V=128, g="fp32", o="bf16", init=True, strided=False),
        # odd lengths, narrow heads of different widths, shared query and key heads, gates in 16 bits
        dict(name="linear_bwd_odd_1501x6", op="linear", dir="bwd", T=1501, N=5, H=6, Hq=2, Hk=2, Hv=6, K=64, V=96,
             g="bf16", o="bf16", init=False, strided=False),
        # decoding one sequence with few heads: latency
        dict(name="linear_step_1x4", op="linear_step", B=1, H=4, Hq=4, Hk=4, Hv=4, K=128, V=128, slots=2, g="fp32",
             o="bf16"),
        # a full server: 256 rows, some of them padding
        dict(name="linear_step_256x32", op="linear_step", B=256, H=32, Hq=32, Hk=32, Hv=32, K=128, V=128, slots=320,
             g="fp32", o="bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "linear", "linear", "linear", "linear_step"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "rotate":
        D = rng.choice([32, 64, 80, 96, 128, 128, 128, 192, 256])
        R = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        Hk, way = rng.randint(1, 16), rng.choice(["fwd", "bwd"])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        T = _log_int(rng, 1, min(32768, (1 << (27 if way == "fwd" else 25)) // ((Hq + Hk) * D)))
        return dict(op=op, dir=way, T=T, Hq=Hq, Hk=Hk, D=D, R=R, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    d=rng.choice(["bf16", "fp32"]), interleaved=flip(), weight=rng.random() < 0.8, strided=flip())
    shared = rng.choice([1, 1, 2, 3, 4])
    H = shared * _log_int(rng, 1, 32 // shared)
    Hq, Hk, Hv = rng.choice([(H // shared, H // shared, H), (H, H // shared, H // shared)])
    heads = dict(H=H, Hq=Hq, Hk=Hk, Hv=Hv, K=rng.choice([128, 128, 64, 8 * rng.randint(1, 16)]),
                 V=rng.choice([128, 128, 64, 8 * rng.randint(1, 16)]), g=rng.choice(["fp32", "fp32", "bf16", "head"]),
                 o=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "linear":
        way = rng.choice(["fwd", "bwd"])
        T = _log_int(rng, 1, min(65536 if way == "fwd" else 16384, (1 << (21 if way == "fwd" else 19)) // H))
        return dict(op=op, dir=way, T=T, N=_log_int(rng, 1, min(T, 64)), **heads, init=flip(), strided=flip())
    B = _log_int(rng, 1, 256)
    return dict(op=op, B=B, slots=B + rng.randint(0, 64), **heads)


def _lengths(T, N, seed):
    """cu_seqlens of N sequences, none empty, over T tokens."""
    cuts = random.Random(seed * 7919 + N).sample(range(1, T), N - 1) if N > 1 else []
    return [0] + sorted(cuts) + [T]


def _slot_rows(c, seed):
    """Distinct state slots of the batch's rows, in no order, about one row in sixteen of a larger batch unused."""
    r = random.Random(seed * 104729 + c["B"])
    slots = r.sample(range(c["slots"]), c["B"])
    return [-1 if c["B"] > 8 and r.random() < 1 / 16 else s for s in slots]


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def rows(T, parts, dtype, strided):
        """Tensors [T, heads, width]; strided: side by side in one projection's rows, padded to 16 bytes."""
        if not strided:
            return [randn(T, h, w, dtype=dtype) for h, w in parts]
        pad = [-(-h * w // 8) * 8 for h, w in parts]
        row, at = randn(T, sum(pad), dtype=dtype), [sum(pad[:i]) for i in range(len(pad))]
        return [row[:, a:a + h * w].view(T, h, w) for a, (h, w) in zip(at, parts)]

    op, s = c["op"], {"case": c}
    bf = torch.bfloat16
    if op == "rotate":
        T, Hq, Hk, D, R, dt = c["T"], c["Hq"], c["Hk"], c["D"], c["R"], DTYPES[c["dtype"]]
        s["q_raw"], s["k_raw"] = rows(T, [(Hq, D), (Hk, D)], dt, c["strided"])
        # positions of sequences that go on from what a cache holds, up to a million tokens in
        start = torch.randint(0, 1 << 20, (), generator=gen, device=dev)
        run_on = torch.arange(T, device=dev) if T > 64 else torch.randint(0, 1 << 19, (T,), generator=gen, device=dev)
        s["positions"] = (start + run_on).to(torch.int32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(R // 2, dtype=torch.float64, device=dev) * 2 / R)).float()
        s["q_weight"], s["k_weight"] = (1 + 0.1 * randn(D) if c["weight"] else None for _ in range(2))
        if c["dir"] == "bwd":
            s["dq"], s["dk"] = randn(T, Hq, D, dtype=DTYPES[c["d"]]), randn(T, Hk, D, dtype=DTYPES[c["d"]])
        return s
    H, K, V = c["H"], c["K"], c["V"]
    # decays from some tokens to some thousands, a rate for each head
    rate = torch.exp(-7 * torch.rand(H, generator=gen, device=dev))
    n = c["T"] if op == "linear" else c["B"]
    q, k, v = rows(n, [(c["Hq"], K), (c["Hk"], K), (c["Hv"], V)], bf, c.get("strided", False))
    # normalised as a norm before the operator leaves them
    q.copy_(q / torch.sqrt((q.float() ** 2).mean(-1, keepdim=True)) * K ** -0.5)
    k.copy_(k / torch.sqrt((k.float() ** 2).mean(-1, keepdim=True)) * K ** -0.5)
    s["q"], s["k"], s["v"] = q, k, v
    if c["g"] == "head":
        s["g"] = -rate
    else:
        s["g"] = (-torch.nn.functional.softplus(randn(n, H)) * rate).to(DTYPES[c["g"]])
    if op == "linear":
        T, N = c["T"], c["N"]
        s["cu"] = _lengths(T, N, seed)
        s["h0"] = randn(N, H, K, V) if c["init"] else None
        s["bounds"] = torch.tensor(s["cu"], device=dev)
        if c["dir"] == "bwd":
            s["d_o"] = randn(T, H, V, dtype=bf)
            s["d_final"] = randn(N, H, K, V)
        if own:
            from gated_delta_rule_37_amd import kda, layer
            s["plan"] = kda.Plan(s["cu"], layer.linear_segments(s["cu"], H))
            s["plan"].device_blob(s["q"].device)
        return s
    # the pool before the step is read, the pool after it written: a pass can be made again
    s["state"] = randn(c["slots"], H, K, V)
    slots = _slot_rows(c, seed)
    s["slots"] = torch.tensor(slots, dtype=torch.int32, device=dev)
    s["rows"] = torch.tensor([i for i, m in enumerate(slots) if m >= 0], device=dev)
    s["state_out"] = s["state"].clone()
    s["out"] = torch.zeros(c["B"], H, V, device=dev, dtype=DTYPES[c["o"]])
    return s


# ------------------------------------------------------------------ plain forms


def _turn(x, cos, sin, R, interleaved):
    """The first R channels of x [T, H, D] in pairs, by angles [T, R / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    r, rest = x[..., :R], x[..., R:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :R // 2], r[..., R // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _plain_rotate(s):
    c = s["case"]
    R, dt = c["R"], DTYPES[c["dtype"]]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = {}
    for n, scale in (("q", c["D"] ** -0.5), ("k", 1.0)):
        x, w = s[n + "_raw"].float(), s[n + "_weight"]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xn = x * r
        if c["dir"] == "fwd":
            y = scale * xn if w is None else scale * xn * w
            out[n] = _turn(y, cos, sin, R, c["interleaved"]).to(dt)
            continue
        m = scale * _turn(s["d" + n].float(), cos, -sin, R, c["interleaved"])
        wm = m if w is None else m * w
        out["d" + n + "_raw"] = (r * (wm - xn * (wm * xn).mean(-1, keepdim=True))).to(dt)
        out["d" + n + "_weight"] = None if w is None else (m * xn).sum((0, 1), dtype=torch.float64).float()
    return out


def _chunks(bounds):
    """Chunks of at most CHUNK tokens, none over a sequence's end: their tokens [M, CHUNK], which of them are, each
    chunk's sequence, and whether it is the sequence's first."""
    length = bounds[1:] - bounds[:-1]
    per = (length + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(len(per), device=bounds.device), per)
    nth = torch.arange(len(seq), device=bounds.device) - (torch.cumsum(per, 0) - per)[seq]
    tokens = (bounds[:-1][seq] + nth * CHUNK)[:, None] + torch.arange(CHUNK, device=bounds.device)
    valid = tokens < bounds[1:][seq][:, None]
    return torch.where(valid, tokens, 0), valid, seq, nth == 0


def _to_chunks(x, tokens, valid, H):
    """[T, heads, W] as [M, H, CHUNK, W] in 32 bits, zero behind a sequence's end."""
    y = x[tokens].float() * valid[:, :, None, None]
    return y.repeat_interleave(H // x.shape[1], 2).transpose(1, 2).contiguous()


def _from_chunks(y, valid, heads):
    """[M, H, CHUNK, W] back to [T, heads, W]: heads that share one are added."""
    y = y.transpose(1, 2)[valid]
    T, H, W = y.shape
    return y if H == heads else y.view(T, heads, H // heads, W).sum(2)


def _states(a, u, first, s0):
    """The state before every chunk, S' = a S + u within each sequence, by doubling over the chunks."""
    a, u = a[..., None, None].clone(), u.clone()
    u[first] += a[first] * s0
    a[first] = 0
    stride = 1
    while stride < len(a):
        u[stride:] += a[stride:] * u[:-stride]
        a[stride:] = a[stride:] * a[:-stride]
        stride *= 2
    before = torch.empty_like(u)
    before[1:] = u[:-1]
    before[first] = s0
    return before, u


def _plain_linear(s):
    c = s["case"]
    H = c["H"]
    tokens, valid, seq, first = _chunks(s["bounds"])
    q, k, v = (_to_chunks(s[n], tokens, valid, H) for n in ("q", "k", "v"))
    g = s["g"].double().expand(c["T"], H)[tokens] * valid[:, :, None]
    G = torch.cumsum(g, 1).transpose(1, 2)                                      # [M, H, CHUNK]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, float("-inf")).float())
    since, until, whole = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float(), torch.exp(G[..., -1]).float()
    s0 = 0.0 if s["h0"] is None else s["h0"]
    before, after = _states(whole, torch.matmul((k * until[..., None]).transpose(-1, -2).contiguous(), v), first, s0)
    kt, qk = k.transpose(-1, -2).contiguous(), None
    qk = torch.matmul(q, kt) * decay
    last = torch.cat([first[1:], first.new_ones(1)])
    if c["dir"] == "fwd":
        o = torch.matmul(qk, v) + since[..., None] * torch.matmul(q, before)
        return {"o": _from_chunks(o, valid, H).to(DTYPES[c["o"]]), "final_state": after[last]}
    do = _to_chunks(s["d_o"], tokens, valid, H)
    # the cotangent of the state after every chunk: the same recurrence from the other end
    back, start = _states(whole.flip(0), torch.matmul((q * since[..., None]).transpose(-1, -2).contiguous(), do).flip(0),
                          last.flip(0), s["d_final"].flip(0))
    after_d, start = back.flip(0), start.flip(0)
    dov = torch.matmul(do, v.transpose(-1, -2).contiguous()) * decay
    from_start = since[..., None] * torch.matmul(do, before.transpose(-1, -2).contiguous())
    dq = torch.matmul(dov, k) + from_start
    from_end = until[..., None] * torch.matmul(v, after_d.transpose(-1, -2).contiguous())
    dk = torch.matmul(dov.transpose(-1, -2).contiguous(), q) + from_end
    dv = torch.matmul(qk.transpose(-1, -2).contiguous(), do) + until[..., None] * torch.matmul(k, after_d)
    # dg_t: what passes from the tokens before t to those from t on, within the chunk and through the states
    pairs = torch.matmul(q, kt) * dov
    pairs = torch.cumsum(pairs.tril(-1), -1) - pairs.tril(-1)                   # [.., i, t]: sum over j < t
    rho, kappa = (q * from_start).sum(-1), (k * from_end).sum(-1)
    dg = (pairs * low).sum(-2) + rho.flip(-1).cumsum(-1).flip(-1) + torch.cumsum(kappa, -1) - kappa
    dg = dg + (whole * (after_d * before).sum((-1, -2)))[..., None]
    dg = _from_chunks(dg[..., None], valid, H)[..., 0]
    bf = torch.bfloat16
    return {"dq": _from_chunks(dq, valid, c["Hq"]).to(bf), "dk": _from_chunks(dk, valid, c["Hk"]).to(bf),
            "dv": _from_chunks(dv, valid, c["Hv"]).to(bf),
            "dg": dg.sum(0, dtype=torch.float64).float() if c["g"] == "head" else dg.to(s["g"].dtype),
            "dh0": None if s["h0"] is None else start[first]}


def _plain_step(s):
    c, rows = s["case"], s["rows"]
    slots = s["slots"][rows].long()
    q, k, v = (s[n][rows].float().repeat_interleave(c["H"] // s[n].shape[1], 1) for n in ("q", "k", "v"))
    g = s["g"].float().expand(c["B"], c["H"])[rows]
    S = s["state"][slots] * torch.exp(g)[..., None, None] + k[..., None] * v[..., None, :]
    s["state_out"][slots] = S
    s["out"][rows] = (S * q[..., None]).sum(-2).to(s["out"].dtype)
    return {"o": s["out"], "state": s["state_out"]}


# ------------------------------------------------------------------ the framework's calls


def _own(s):
    from gated_delta_rule_37_amd import layer
    c = s["case"]
    if c["op"] == "rotate":
        raw = (s["q_raw"], s["k_raw"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"])
        how = dict(q_scale=c["D"] ** -0.5, eps=EPS, interleaved=c["interleaved"])
        if c["dir"] == "fwd":
            return layer.qk_norm_rotate(*raw, **how)
        return layer.qk_norm_rotate_backward(*raw, s["dq"], s["dk"], **how)
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            return layer.linear_forward(s["plan"], s["q"], s["k"], s["v"], s["g"], initial_state=s["h0"],
                                        o_dtype=DTYPES[c["o"]])
        return layer.linear_backward(s["plan"], s["q"], s["k"], s["v"], s["g"], s["d_o"], d_final=s["d_final"],
                                     initial_state=s["h0"])
    layer.linear_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["slots"], state_out=s["state_out"], o=s["out"])
    return {"o": s["out"], "state": s["state_out"]}


PLAIN = {"rotate": _plain_rotate, "linear": _plain_linear, "linear_step": _plain_step}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and exact values


def work(case):
    c, op = case, case["op"]
    if op == "rotate":
        n, e, table = c["T"] * (c["Hq"] + c["Hk"]) * c["D"], SIZE[c["dtype"]], c["T"] * 4 + c["R"] * 2
        w = 2 * c["D"] * 4 if c["weight"] else 0
        if c["dir"] == "fwd":
            return {"bytes": n * 2 * e + table + w, "flops": n * 8}
        return {"bytes": n * (2 * e + SIZE[c["d"]]) + table + 2 * w, "flops": n * 16}
    K, V, H = c["K"], c["V"], c["H"]
    n = c["T"] if op == "linear" else c["B"]
    heads = (c["Hq"] + c["Hk"]) * K + c["Hv"] * V
    gate = H * 4 if c["g"] == "head" else n * H * SIZE[c["g"]]
    if op == "linear":
        state = c["N"] * H * K * V * 4
        if c["dir"] == "fwd":
            b = n * heads * 2 + gate + n * H * V * SIZE[c["o"]] + state * (2 if c["init"] else 1)
            return {"bytes": b, "flops": n * H * K * V * 4}
        b = 2 * n * heads * 2 + 2 * gate + n * H * V * 2 + state * (3 if c["init"] else 1)
        return {"bytes": b, "flops": n * H * K * V * 10}
    return {"bytes": n * H * K * V * 8 + n * heads * 2 + gate + n * H * V * SIZE[c["o"]] + n * 4,
            "flops": n * H * K * V * 5}


def exact(case, seed):
    """The definitions in 64 bits: gradients by differentiation, the attention over all pairs of a sequence's tokens."""
    s = prepare(case, seed)
    s.pop("plan", None)
    c = s["case"]
    if c["op"] == "rotate":
        return _exact_rotate(s, c)
    if c["op"] == "linear":
        return _exact_linear(s, c)
    out, pool = s["out"].double(), s["state"].double()
    where, g = s["slots"].tolist(), s["g"].double()
    of = lambda n, b, h: s[n][b, h * s[n].shape[1] // c["H"]].double()  # noqa: E731
    for b in s["rows"].tolist():
        for h in range(c["H"]):
            e = torch.exp(g[h] if g.dim() == 1 else g[b, h])
            pool[where[b], h] = e * pool[where[b], h] + torch.outer(of("k", b, h), of("v", b, h))
            out[b, h] = torch.mv(pool[where[b], h].t(), of("q", b, h))
    return {"o": out, "state": pool}


def _exact_rotate(s, c):
    """By complex numbers, in pieces of the tokens."""
    T, R, out = c["T"], c["R"], {}
    step = max(1, (1 << 24) // (max(c["Hq"], c["Hk"]) * c["D"]))
    for n, scale in (("q", c["D"] ** -0.5), ("k", 1.0)):
        w = None if s[n + "_weight"] is None else s[n + "_weight"].double().requires_grad_()
        pieces = []
        for t in range(0, T, step):
            x = s[n + "_raw"][t:t + step].double().requires_grad_()
            y = scale * x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS)
            y = y if w is None else y * w
            theta = s["positions"][t:t + step].double()[:, None, None] * s["inv_freq"].double()
            z = y[..., :R].unflatten(-1, (R // 2, 2) if c["interleaved"] else (2, R // 2))
            z = z if c["interleaved"] else z.transpose(-1, -2)
            z = torch.view_as_real(torch.complex(z[..., 0], z[..., 1]) * torch.polar(torch.ones_like(theta), theta))
            z = z if c["interleaved"] else z.transpose(-1, -2)
            y = torch.cat([z.flatten(-2), y[..., R:]], -1)
            if c["dir"] == "bwd":
                y.backward(s["d" + n][t:t + step].double())
                y = x.grad
            pieces.append(y.detach())
        out[n if c["dir"] == "fwd" else "d" + n + "_raw"] = torch.cat(pieces)
        if c["dir"] == "bwd":
            out["d" + n + "_weight"] = None if w is None else w.grad
    return out


def _exact_linear(s, c):
    T, N, H, K, V = (c[n] for n in ("T", "N", "H", "K", "V"))
    if c["dir"] == "bwd":
        leaves = {n: s[n].double().requires_grad_() for n in ("q", "k", "v", "g")}
        if s["h0"] is not None:
            leaves["h0"] = s["h0"].double().requires_grad_()
    else:
        leaves = {n: s[n].double() for n in ("q", "k", "v", "g", "h0") if s[n] is not None}
    o = torch.zeros(T, H, V, dtype=torch.float64, device=s["q"].device)
    final = torch.zeros(N, H, K, V, dtype=torch.float64, device=s["q"].device)
    for n, (lo, hi) in enumerate(zip(s["cu"], s["cu"][1:])):
        for h in range(H):
            q, k, v = (leaves[m][lo:hi, h * leaves[m].shape[1] // H] for m in ("q", "k", "v"))
            g = leaves["g"][h].expand(hi - lo) if c["g"] == "head" else leaves["g"][lo:hi, h]
            G = torch.cumsum(g, 0)
            h0 = leaves["h0"][n, h] if "h0" in leaves else None
            loss = 0.0
            # rows of the triangle, so many that they stay small
            step = max(64, (1 << 26) // (hi - lo))
            for a in range(0, hi - lo, step):
                b = min(a + step, hi - lo)
                rows = torch.arange(a, b, device=G.device)[:, None] >= torch.arange(b, device=G.device)
                d = torch.exp((G[a:b, None] - G[None, :b]).masked_fill(~rows, float("-inf")))
                y = torch.mm(torch.mm(q[a:b], k[:b].t()) * d, v[:b])
                y = y if h0 is None else y + torch.exp(G[a:b, None]) * torch.mm(q[a:b], h0)
                if c["dir"] == "fwd":
                    o[lo + a:lo + b, h] = y
                else:
                    loss = loss + (y * s["d_o"][lo + a:lo + b, h].double()).sum()
            f = torch.mm((k * torch.exp(G[-1] - G)[:, None]).t(), v)
            f = f if h0 is None else f + torch.exp(G[-1]) * h0
            if c["dir"] == "fwd":
                final[n, h] = f
            else:
                (loss + (f * s["d_final"][n, h].double()).sum()).backward()
    if c["dir"] == "fwd":
        return {"o": o, "final_state": final}
    return {"dh0" if n == "h0" else "d" + n: t.grad for n, t in leaves.items()} | ({} if "h0" in leaves else {"dh0": None})
