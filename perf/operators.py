"""The operators around the scan as a user calls them, beside plain torch forms of the same.

Four operators of a layer built from a linear recurrence: the gated linear recurrence itself
(forward, training step, one decode token), the residual addition with RMS norm (to 8 bits with
scales for serving, forward and backward for training), the quantisation of activations to e4m3
with one scale per 128 values, and the projection (matrix product) of such operands.

``own`` selects the library's kernels; otherwise ``run`` evaluates the definitions with
elementary torch operations in 32 bits.
"""
import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

DEV = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0
GROUP = 128
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _size(name):
    return 2 if name == "bf16" else 4


# ---- the cases -------------------------------------------------------------------------


def listed():
    return [
        # one decode token of the served batch: 256 requests, the widest layer of the benchmark
        dict(name="gated_token", op="gated_update", batch=256, dim=5120, dtype="bf16", decay=False, z=True),
        # prefill of the widest layer, sigmoid gate and SiLU output gate
        dict(name="gated_prefill", op="gated_fwd", batch=4, dim=5120, seqlen=4096, dtype="bf16",
             decay=False, z=True),
        # a few channels over a very long sequence, decays given, fp32, length not a multiple of any vector
        dict(name="gated_long_fp32", op="gated_fwd", batch=1, dim=60, seqlen=524287, dtype="fp32",
             decay=True, z=False),
        # a training step of the small layer: forward, then every gradient
        dict(name="gated_train", op="gated_train", batch=8, dim=1536, seqlen=2048, dtype="bf16",
             decay=False, z=True),
        # a decode step's norm in front of an 8-bit projection
        dict(name="norm_fp8_token", op="norm_fp8", rows=256, dim=2560, dtype="bf16", residual="fp32"),
        # the same for a prefill
        dict(name="norm_fp8_prefill", op="norm_fp8", rows=16384, dim=2560, dtype="bf16", residual="fp32"),
        # training: forward and backward with a 16-bit residual stream, a ragged number of rows
        dict(name="norm_train", op="norm_train", rows=16001, dim=768, dtype="bf16", residual="bf16"),
        # the scan's output (channel-major) quantised for the output projection, in prefill
        dict(name="quantize_prefill", op="quantize", batch=4, dim=5120, seqlen=4096, dtype="bf16",
             channel_major=True),
        # the same for one short request of odd length
        dict(name="quantize_short", op="quantize", batch=1, dim=1536, seqlen=333, dtype="bf16",
             channel_major=True),
        # projections: a few tokens of decode, a ragged middle size, the prefill of the widest layer
        dict(name="linear_token", op="linear", batch=16, seqlen=1, k=2560, n=10240, channel_major=False),
        dict(name="linear_ragged", op="linear", batch=3, seqlen=431, k=1536, n=848, channel_major=True),
        dict(name="linear_prefill", op="linear", batch=4, seqlen=4096, k=2560, n=10240,
             channel_major=False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_update", "gated_fwd", "gated_fwd", "gated_train", "norm_fp8", "norm_train",
                     "quantize", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "gated_update":
        return dict(op=op, batch=_log(rng, 1, 256), dim=_log(rng, 64, 5120), dtype=dtype,
                    decay=rng.random() < 0.4, z=rng.random() < 0.5)
    if op in ("gated_fwd", "gated_train"):
        most = 4 * 5120 * 4096 if op == "gated_fwd" else 8 * 1536 * 2048
        dim = _log(rng, 16, 5120)
        seqlen = _log(rng, 1, min(524288, most // dim))
        batch = _log(rng, 1, max(1, min(8, most // (dim * seqlen))))
        return dict(op=op, batch=batch, dim=dim, seqlen=seqlen, dtype=dtype,
                    decay=rng.random() < 0.4, z=rng.random() < 0.5)
    if op in ("norm_fp8", "norm_train"):
        step = 16 if op == "norm_fp8" else rng.choice([1, 8])
        dim = max(step, _log(rng, 64, 5120) // step * step)
        rows = _log(rng, 1, 16384 * 2560 // dim if op == "norm_fp8" else 16001 * 768 // dim)
        return dict(op=op, rows=rows, dim=dim, dtype=dtype, residual=rng.choice(["fp32", dtype]))
    if op == "quantize":
        dim = 16 * _log(rng, 4, 320)
        seqlen = _log(rng, 1, 4096)
        batch = _log(rng, 1, max(1, min(16, 4 * 5120 * 4096 // (dim * seqlen))))
        return dict(op=op, batch=batch, dim=dim, seqlen=seqlen, dtype=dtype,
                    channel_major=rng.random() < 0.6)
    k, n = 16 * _log(rng, 8, 320), _log(rng, 16, 10240)
    tokens = _log(rng, 1, max(1, min(16384, 16384 * 2560 * 10240 // (k * n))))
    batch = rng.choice([1, 2, 3, 4])
    return dict(op=op, batch=batch, seqlen=max(1, tokens // batch), k=k, n=n,
                channel_major=rng.random() < 0.4)


# ---- inputs ----------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = dict(case=dict(case))
    op = case["op"]
    if op.startswith("gated"):
        dt = TYPES[case["dtype"]]
        b, d = case["batch"], case["dim"]
        shape = (b, d) if op == "gated_update" else (b, d, case["seqlen"])
        s["x"] = normal(*shape, dtype=dt)
        if case["decay"]:  # decays given: memories from a few steps to hundreds
            s["gate"] = torch.exp2(-4.0 * uniform(*shape) ** 4 - 0.002).to(dt)
            s["gate_bias"] = None
        else:  # raw gates; the bias starts the channels at memories from 2 to 200 steps
            s["gate"] = normal(*shape, dtype=dt)
            v = torch.exp(math.log(0.005) + (math.log(0.5) - math.log(0.005)) * uniform(d))
            s["gate_bias"] = torch.log(v / (1 - v))
        s["z"] = normal(*shape, dtype=dt) if case["z"] else None
        s["state"] = normal(b, d)
        if op == "gated_train":
            s["dy"] = normal(*shape, dtype=dt)
            s["dlast"] = normal(b, d)
    elif op.startswith("norm"):
        dt, rt = TYPES[case["dtype"]], TYPES[case["residual"]]
        r, d = case["rows"], case["dim"]
        s["x"] = normal(r, d, dtype=dt)
        s["residual"] = (3.0 * normal(r, d)).to(rt)
        s["weight"] = 1.0 + 0.1 * normal(d)
        if op == "norm_train":
            s["dout"] = normal(r, d, dtype=dt)
            s["dres"] = normal(r, d, dtype=rt)
    elif op == "quantize":
        dt = TYPES[case["dtype"]]
        b, d, n = case["batch"], case["dim"], case["seqlen"]
        # token and channel sizes spread as a gated scan's output is
        x = normal(b, d, n) * torch.exp(normal(b, d, 1)) * torch.exp(0.5 * normal(b, 1, n))
        s["x"] = (x if case["channel_major"] else x.transpose(1, 2).reshape(b * n, d)).to(dt).contiguous()
    else:
        t, k, n = case["batch"] * case["seqlen"], case["k"], case["n"]
        s["xq"], s["xs"] = _rows_to_e4m3(normal(t, k) * torch.exp(0.5 * normal(t, 1)))
        s["wq"], s["ws"] = _blocks_to_e4m3(normal(n, k) / math.sqrt(k))
    return s


def _rows_to_e4m3(x):
    """(rows, k) fp32 -> e4m3 values and one scale for each row and 128 columns."""
    r, k = x.shape
    kb = -(-k // GROUP)
    p = torch.nn.functional.pad(x, (0, kb * GROUP - k)).view(r, kb, GROUP)
    amax = p.abs().amax(-1).clamp(min=1e-30)
    q = (p * (E4M3_MAX / amax)[..., None]).reshape(r, kb * GROUP)[:, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), amax / E4M3_MAX


def _blocks_to_e4m3(w):
    """(n, k) fp32 -> e4m3 values and one scale for each block of 128 x 128."""
    n, k = w.shape
    nb, kb = -(-n // GROUP), -(-k // GROUP)
    p = torch.nn.functional.pad(w, (0, kb * GROUP - k, 0, nb * GROUP - n)).view(nb, GROUP, kb, GROUP)
    amax = p.abs().amax((1, 3)).clamp(min=1e-30)
    q = (p * (E4M3_MAX / amax)[:, None, :, None]).reshape(nb * GROUP, kb * GROUP)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), amax / E4M3_MAX


def _of_rows(q, scales):
    """The values that e4m3 rows with a scale per 128 columns stand for, fp32."""
    return q.float() * scales.repeat_interleave(GROUP, dim=1)[:, :q.shape[1]]


# ---- the plain forms -------------------------------------------------------------------


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along the last axis from h = 0, by halving."""
    n = a.shape[-1]
    if n == 1:
        return b
    m = n // 2 * 2
    a1, b1 = a[..., 1:m:2], b[..., 1:m:2]
    odd = _recur(a[..., 0:m:2] * a1, a1 * b[..., 0:m:2] + b1)
    h = torch.empty_like(b)
    h[..., 1:m:2] = odd
    h[..., 0] = b[..., 0]
    h[..., 2::2] = a[..., 2::2] * odd[..., :(n - 1) // 2] + b[..., 2::2]
    return h


def _gates(s):
    """(a, b, sigmoid of the gate or None) in fp32."""
    x, gate = s["x"].float(), s["gate"].float()
    if s["gate_bias"] is None:
        return gate, x, None
    bias = s["gate_bias"] if gate.dim() == 2 else s["gate_bias"][:, None]
    sg = 1.0 / (1.0 + torch.exp(-(gate + bias)))
    return 1.0 - sg, sg * x, sg


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain_update(s):
    a, b, _ = _gates(s)
    h = a * s["state"] + b
    s["state"].copy_(h)
    y = h if s["z"] is None else h * _silu(s["z"].float())
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _plain_states(s):
    a, b, sg = _gates(s)
    b = b.clone()
    b[..., 0] += a[..., 0] * s["state"]
    return a, sg, _recur(a, b)


def _plain_fwd(s):
    _, _, h = _plain_states(s)
    y = h if s["z"] is None else h * _silu(s["z"].float())
    return dict(y=y.to(s["x"].dtype), last_state=h[..., -1].contiguous())


def _plain_train(s):
    dt = s["x"].dtype
    a, sg, h = _plain_states(s)
    g = s["dy"].float()
    r = dict(dz=None)
    if s["z"] is None:
        r["y"] = h.to(dt)
    else:
        z = s["z"].float()
        sz = 1.0 / (1.0 + torch.exp(-z))
        r["y"] = (h * z * sz).to(dt)
        r["dz"] = (g * h * sz * (1.0 + z * (1.0 - sz))).to(dt)
        g = g * z * sz
    r["last_state"] = h[..., -1].contiguous()
    g = g.clone()
    g[..., -1] += s["dlast"]
    later = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1)
    dh = _recur(later.flip(-1), g.flip(-1)).flip(-1)
    before = torch.cat([s["state"][..., None], h[..., :-1]], -1)
    r["dinitial_state"] = a[..., 0] * dh[..., 0]
    r["dgate_bias"] = None
    if sg is None:
        r["dx"], r["dgate"] = dh.to(dt), (dh * before).to(dt)
    else:
        r["dx"] = (sg * dh).to(dt)
        dgate = dh * (s["x"].float() - before) * sg * a
        r["dgate"], r["dgate_bias"] = dgate.to(dt), dgate.sum((0, 2))
    return r


def _plain_norm(s):
    total = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = total.float()
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return total, v, rstd, v * rstd * s["weight"]


def _plain_norm_fp8(s):
    total, _, _, out = _plain_norm(s)
    q, scales = _rows_to_e4m3(out)
    return dict(q=q, scales=scales, residual_out=total)


def _plain_norm_train(s):
    total, v, rstd, out = _plain_norm(s)
    xhat, g = v * rstd, s["dout"].float()
    wg = g * s["weight"]
    dr = s["dres"].float() + rstd * (wg - xhat * (wg * xhat).mean(-1, keepdim=True))
    return dict(out=out.to(s["x"].dtype), residual_out=total, dx=dr.to(s["x"].dtype),
                dresidual=dr.to(s["residual"].dtype), dweight=(g * xhat).sum(0))


def _plain_quantize(s):
    x = s["x"].float()
    if s["case"]["channel_major"]:
        x = x.transpose(1, 2).reshape(-1, x.shape[1])
    q, scales = _rows_to_e4m3(x)
    return dict(q=q, scales=scales)


def _plain_linear(s):
    n, k = s["wq"].shape
    w = s["wq"].float() * s["ws"].repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :k]
    out = torch.matmul(_of_rows(s["xq"], s["xs"]), w.t())
    if s["case"]["channel_major"]:
        out = out.view(s["case"]["batch"], s["case"]["seqlen"], n).transpose(1, 2)
    return dict(out=out.bfloat16().contiguous())


# ---- the library's calls ---------------------------------------------------------------


def _own_update(s):
    from selective_state_space_56_b200 import ops
    y = ops.gated_state_update(s["state"], s["x"], s["gate"], gate_bias=s["gate_bias"], z=s["z"],
                               given_decay=s["case"]["decay"])
    return dict(y=y, state=s["state"])


def _own_fwd(s):
    from selective_state_space_56_b200 import ops
    y, last = ops.gated_scan_fwd(s["x"], s["gate"], gate_bias=s["gate_bias"], z=s["z"],
                                 initial_state=s["state"], given_decay=s["case"]["decay"],
                                 return_last_state=True)
    return dict(y=y, last_state=last)


def _own_train(s):
    from selective_state_space_56_b200 import ops
    decay = s["case"]["decay"]
    kept = torch.empty(ops.gated_scan_checkpoints_size(*s["x"].shape), dtype=torch.uint8, device=DEV)
    y, last = ops.gated_scan_fwd(s["x"], s["gate"], gate_bias=s["gate_bias"], z=s["z"],
                                 initial_state=s["state"], given_decay=decay, return_last_state=True,
                                 checkpoints=kept)
    g = ops.gated_scan_bwd(s["x"], s["gate"], s["dy"], gate_bias=s["gate_bias"], z=s["z"],
                           initial_state=s["state"], dlast_state=s["dlast"], given_decay=decay,
                           checkpoints=kept)
    return dict(y=y, last_state=last, **g)


def _own_norm_fp8(s):
    from selective_state_space_56_b200 import ops
    q, scales, total = ops.add_rms_norm_fp8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    return dict(q=q, scales=scales, residual_out=total)


def _own_norm_train(s):
    from selective_state_space_56_b200 import ops
    out, total = ops.add_rms_norm_fwd(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    g = ops.add_rms_norm_bwd(s["dout"], total, s["weight"], dresidual_out=s["dres"], eps=EPS)
    return dict(out=out, residual_out=total, **g)


def _own_quantize(s):
    from selective_state_space_56_b200 import ops
    q, scales = ops.fp8_quantize(s["x"], channel_major=s["case"]["channel_major"])
    return dict(q=q, scales=scales)


def _own_linear(s):
    from selective_state_space_56_b200 import ops
    seqlen = s["case"]["seqlen"] if s["case"]["channel_major"] else None
    return dict(out=ops.fp8_linear(s["xq"], s["xs"], s["wq"], s["ws"], out_dtype=torch.bfloat16,
                                   channel_major_seqlen=seqlen))


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(gated_update=_own_update, gated_fwd=_own_fwd, gated_train=_own_train,
                    norm_fp8=_own_norm_fp8, norm_train=_own_norm_train, quantize=_own_quantize,
                    linear=_own_linear)[op](state)
    return dict(gated_update=_plain_update, gated_fwd=_plain_fwd, gated_train=_plain_train,
                norm_fp8=_plain_norm_fp8, norm_train=_plain_norm_train, quantize=_plain_quantize,
                linear=_plain_linear)[op](state)


# ---- what a pass cannot do without -----------------------------------------------------


def work(case):
    op = case["op"]
    if op.startswith("gated"):
        rows, e = case["batch"] * case["dim"], _size(case["dtype"])
        bias = 0 if case["decay"] else 4 * case["dim"]
        gate = 0 if case["decay"] else 5  # sigmoid and the two products
        z = 1 if case["z"] else 0
        if op == "gated_update":
            return dict(bytes=rows * (8 + (3 + z) * e) + bias, flops=rows * (2 + gate + 5 * z))
        n = rows * case["seqlen"]
        fwd = dict(bytes=n * (3 + z) * e + rows * 8 + bias, flops=n * (2 + gate + 5 * z))
        if op == "gated_fwd":
            return fwd
        # read x, gate, dy, z and the entering and leaving states' values, write dx, dgate, dz
        return dict(bytes=fwd["bytes"] + n * (5 + 2 * z) * e + rows * 12 + 2 * bias,
                    flops=fwd["flops"] + n * (6 + 2 * gate + 12 * z))
    if op.startswith("norm"):
        r, d, e, f = case["rows"], case["dim"], _size(case["dtype"]), _size(case["residual"])
        if op == "norm_fp8":
            return dict(bytes=r * d * (e + 2 * f + 1) + r * -(-d // GROUP) * 4 + 4 * d, flops=8 * r * d)
        # forward: x, residual -> out, residual_out; backward: dout, residual_out, dresidual_out ->
        # dx and dresidual (one array where their types agree), dweight
        back = e + 2 * f + e + (0 if e == f else f)
        return dict(bytes=r * d * (2 * e + 2 * f + back) + 12 * d, flops=16 * r * d)
    if op == "quantize":
        t, d, e = case["batch"] * case["seqlen"], case["dim"], _size(case["dtype"])
        return dict(bytes=t * d * (e + 1) + t * -(-d // GROUP) * 4, flops=3 * t * d)
    t, k, n = case["batch"] * case["seqlen"], case["k"], case["n"]
    kb = -(-k // GROUP)
    return dict(bytes=t * k + n * k + 4 * kb * (t + -(-n // GROUP)) + 2 * t * n, flops=2 * t * n * k)


# ---- the definitions in 64 bits --------------------------------------------------------


def _sequence(a, b):
    """h_t = a_t h_{t-1} + b_t from h = 0, 64 bits: steps taken one after another inside pieces
    of about sqrt(L) steps, all pieces side by side, then piece after piece."""
    rows, n = a.shape
    c = max(1, math.isqrt(n))
    m = -(-n // c)
    a = torch.nn.functional.pad(a, (0, m * c - n), value=1.0).view(rows, m, c)
    b = torch.nn.functional.pad(b, (0, m * c - n)).view(rows, m, c)
    h, p = torch.empty_like(b), torch.empty_like(a)
    h[:, :, 0], p[:, :, 0] = b[:, :, 0], a[:, :, 0]
    for i in range(1, c):
        h[:, :, i] = a[:, :, i] * h[:, :, i - 1] + b[:, :, i]
        p[:, :, i] = a[:, :, i] * p[:, :, i - 1]
    for j in range(1, m):
        h[:, j] += p[:, j] * h[:, j - 1, -1:]
    return h.view(rows, m * c)[:, :n]


def _exact_gated(s):
    case = s["case"]
    b, d = case["batch"], case["dim"]
    one = case["op"] == "gated_update"
    n = 1 if one else case["seqlen"]
    x, gate = s["x"].double().view(b * d, n), s["gate"].double().view(b * d, n)
    h0 = s["state"].double().view(b * d)
    sg = None
    if case["decay"]:
        a, u = gate, x
    else:
        sg = torch.sigmoid(gate + s["gate_bias"].double().repeat(b)[:, None])
        a, u = torch.sigmoid(-(gate + s["gate_bias"].double().repeat(b)[:, None])), sg * x
    first = torch.zeros_like(u)
    first[:, 0] = a[:, 0] * h0
    h = _sequence(a, u + first)
    z = None if s["z"] is None else s["z"].double().view(b * d, n)
    zs = None if z is None else torch.sigmoid(z)
    y = h if z is None else h * z * zs
    if one:
        return dict(y=y.view(b, d), state=h.view(b, d))
    r = dict(y=y.view(b, d, n), last_state=h[:, -1].reshape(b, d))
    if case["op"] == "gated_fwd":
        return r
    dy = s["dy"].double().view(b * d, n)
    into = dy if z is None else dy * z * zs
    into = into.clone()
    into[:, -1] += s["dlast"].double().view(-1)
    # the adjoint runs backwards: dh_t = into_t + a_{t+1} dh_{t+1}
    back = torch.ones_like(a)
    back[:, 1:] = a[:, 1:].flip(1)
    dh = _sequence(back, into.flip(1)).flip(1)
    prev = torch.empty_like(h)
    prev[:, 0], prev[:, 1:] = h0, h[:, :-1]
    r["dinitial_state"] = (a[:, 0] * dh[:, 0]).view(b, d)
    r["dz"] = None if z is None else (dy * h * (zs + z * zs * torch.sigmoid(-z))).view(b, d, n)
    if sg is None:
        r["dx"], r["dgate"], r["dgate_bias"] = dh.view(b, d, n), (dh * prev).view(b, d, n), None
        return r
    dg = dh * (x - prev) * sg * a
    r["dx"], r["dgate"] = (sg * dh).view(b, d, n), dg.view(b, d, n)
    r["dgate_bias"] = dg.view(b, d, n).sum((0, 2))
    return r


def _exact_groups(v):
    """Rows of 64-bit values in e4m3 with a scale per 128 columns: (values of e4m3, scales)."""
    t, d = v.shape
    q, scales = torch.empty_like(v), []
    for c in range(0, d, GROUP):
        part = v[:, c:c + GROUP]
        scale = part.abs().amax(1, keepdim=True).clamp(min=1e-30) / E4M3_MAX
        # the nearest multiple of the last place of e4m3 (3 bits of fraction, least exponent -6)
        w = part / scale
        step = torch.exp2(torch.floor(torch.log2(w.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, c:c + GROUP] = (torch.round(w / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        scales.append(scale)
    return q, torch.cat(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("gated"):
        return _exact_gated(s)
    if op == "quantize":
        x = s["x"].double()
        q, scales = _exact_groups(x.permute(0, 2, 1).flatten(0, 1) if case["channel_major"] else x)
        return dict(q=q, scales=scales)
    if op == "linear":
        n, k = s["wq"].shape
        at = torch.arange(k, device=DEV) // GROUP
        x = s["xq"].double() * s["xs"].double()[:, at]
        w = s["wq"].double() * s["ws"].double()[torch.arange(n, device=DEV) // GROUP][:, at]
        out = (x @ w.t()).view(case["batch"], case["seqlen"], n)
        return dict(out=out.permute(0, 2, 1) if case["channel_major"] else out.flatten(0, 1))
    total = s["x"].double() + s["residual"].double()
    v = total.to(s["residual"].dtype).double()  # the stream is kept, and normalised, in its own type
    norm = v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)
    out = norm * s["weight"].double()
    if op == "norm_fp8":
        q, scales = _exact_groups(out)
        return dict(q=q, scales=scales, residual_out=v)
    g = s["dout"].double() * s["weight"].double()
    root = torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)
    dv = s["dres"].double() + (g - norm * (g * norm).sum(1, keepdim=True) / v.shape[1]) / root
    return dict(out=out, residual_out=v, dx=dv, dresidual=dv, dweight=(s["dout"].double() * norm).sum(0))
