"""Plain fp64 forms of the layer operators around the scan (numpy, one step after another),
and the error models their GPU tests use.  Test infrastructure only.

Error model of the gated recurrence (u = 2^-24, the fp32 rounding).  The kernel forms
sigmoid(gate + bias) as rcp(1 + ex2(t)), t = fma(gate, -log2 e, -log2 e * bias): t is off by
at most 3 u log2(e) (|gate| + |bias|), ex2.approx by 2^-22 relative, the sum by u, rcp.approx
by 2^-23, so the sigmoid s has relative error rho <= 2^-22 (2 + |gate| + |bias|) and a = 1 - s
absolute error s rho + u.  A product or composition is rounded once per step inside a lane and
at most once more per step in the scan over lanes and chunks, so the computed state is that of
a recurrence whose decays are off by eta_t = s_t rho_t + 4 u a_t and whose inputs by
(rho_t + 32 u) |b_t| (32 covers the roundings on the way through lane, warp and chunk):

    E_t = a_t E_{t-1} + eta_t M_{t-1} + (rho_t + 32 u) |b_t|,   M_t = a_t M_{t-1} + |b_t|.

Given decays have rho = 0.  The adjoint obeys the same recurrence backwards.
"""
import numpy as np

U = 2.0 ** -24


def sigmoid(v):
    v = np.asarray(v, np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def gates(x, gate, bias, decay):
    """(a, b, s, rho) of rows (..., L) in fp64; s is None and rho 0 for given decays."""
    if decay:
        return gate, x, None, np.zeros_like(gate)
    bb = 0.0 if bias is None else bias[:, None]
    v = gate + bb
    s = sigmoid(v)
    return sigmoid(-v), s * x, s, 2.0 ** -22 * (2.0 + np.abs(gate) + np.abs(bb))


def gated_forward(x, gate, bias=None, z=None, h0=None, decay=False):
    """x, gate, z (batch, dim, L) fp64.  Returns a dict: h, y, last, and the error model's
    E, M with initial values E = 0, M = |h0|."""
    a, b, s, rho = gates(x, gate, bias, decay)
    eta = (0.0 if s is None else s * rho) + 4 * U * np.abs(a)
    h, E, M = (np.empty_like(x) for _ in range(3))
    hp = np.zeros(x.shape[:2]) if h0 is None else np.array(h0, np.float64)
    h_init, ep, mp = hp.copy(), np.zeros_like(hp), np.abs(hp)
    for t in range(x.shape[2]):
        ep = np.abs(a[..., t]) * ep + eta[..., t] * mp + (rho[..., t] + 32 * U) * np.abs(b[..., t])
        hp = a[..., t] * hp + b[..., t]
        mp = np.abs(a[..., t]) * mp + np.abs(b[..., t])
        h[..., t], E[..., t], M[..., t] = hp, ep, mp
    zf = np.ones_like(x) if z is None else z * sigmoid(z)
    return dict(h=h, y=h * zf, last=hp, E=E, M=M, E_last=ep, a=a, b=b, s=s, rho=rho, eta=eta,
                zf=zf, h0=h_init)


def gated_backward(x, gate, dy, bias=None, z=None, h0=None, dlast=None, decay=False):
    """Gradients (dict as ops.gated_scan_bwd) and their tolerances before the output rounding
    (dict of the same keys)."""
    f = gated_forward(x, gate, bias, z, h0, decay)
    a, s, rho, h = f["a"], f["s"], f["rho"], f["h"]
    B, D, L = x.shape
    zrho = np.zeros_like(x)
    dsilu = None
    if z is not None:
        sz = sigmoid(z)
        dsilu = sz * (1.0 + z * (1.0 - sz))
        zrho = 2.0 ** -22 * (3.0 + np.abs(z))
    gy = dy * f["zf"]
    e = np.zeros((B, D)) if dlast is None else np.array(dlast, np.float64)
    ee, me = np.zeros_like(e), np.abs(e)
    dh, Ed, Md = (np.empty_like(x) for _ in range(3))
    for t in range(L - 1, -1, -1):
        dh[..., t] = gy[..., t] + e
        Ed[..., t] = ee + (zrho[..., t] + 32 * U) * np.abs(gy[..., t])
        Md[..., t] = np.abs(gy[..., t]) + me
        e = a[..., t] * dh[..., t]
        ee = np.abs(a[..., t]) * Ed[..., t] + f["eta"][..., t] * Md[..., t]
        me = np.abs(a[..., t]) * Md[..., t]
    Ed += 8 * U * Md
    prev = np.concatenate([f["h0"][..., None], h[..., :-1]], -1)
    Ep = np.concatenate([np.zeros((B, D, 1)), f["E"][..., :-1]], -1)
    Mp = np.concatenate([np.abs(f["h0"])[..., None], f["M"][..., :-1]], -1)
    g, tol = dict(dinitial_state=e), dict(dinitial_state=ee + 8 * U * me)
    if z is None:
        g["dz"] = tol["dz"] = None
    else:
        g["dz"] = dy * h * dsilu
        # the derivative of silu: sigmoid off by its rho, 1 - sigmoid by sigmoid rho + u
        tol["dz"] = (np.abs(dy * dsilu) * (f["E"] + 4 * U * f["M"]) + np.abs(dy) * f["M"] *
                     2 * zrho * (1.0 + np.abs(z)))
    if decay:
        g["dx"], tol["dx"] = dh, Ed
        g["dgate"] = dh * prev
        tol["dgate"] = Ed * Mp + Md * (Ep + 4 * U * Mp)
        g["dgate_bias"] = tol["dgate_bias"] = None
        return g, tol
    diff, adiff = x - prev, np.abs(x) + Mp
    g["dx"] = s * dh
    # s enters as 1 - a there: off by s rho + 2 u
    ds = s * rho + 2 * U
    tol["dx"] = s * Ed + ds * Md + 2 * U * np.abs(s) * Md
    g["dgate"] = dh * diff * s * a
    tol["dgate"] = (tol["dx"] * adiff * a + s * Md * (Ep + 4 * U * adiff) * a +
                    s * Md * adiff * (ds + 4 * U * a))
    if bias is None:
        g["dgate_bias"] = tol["dgate_bias"] = None
    else:
        g["dgate_bias"] = g["dgate"].sum((0, 2))
        adds = L / 256.0 + 64 + B  # per lane, per warp, over the rows' partial sums
        tol["dgate_bias"] = tol["dgate"].sum((0, 2)) + adds * U * np.abs(g["dgate"]).sum((0, 2))
    return g, tol


def half_step(dtype, ref):
    """Half a step of rounding to dtype ('bf16' or 'fp32') at |ref|."""
    return np.abs(ref) * (2.0 ** -8 if dtype == "bf16" else U) + 1e-38


def rms_norm(v, weight, eps):
    rstd = 1.0 / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps)
    return v * rstd * weight, rstd


def rms_norm_backward(dout, v, weight, dres, eps):
    _, rstd = rms_norm(v, weight, eps)
    xhat, g = v * rstd, dout * weight
    dv = rstd * (g - xhat * np.mean(g * xhat, -1, keepdims=True))
    if dres is not None:
        dv = dv + dres
    return dv, (dout * xhat).sum(0)


def e4m3_groups(v, group=128):
    """(e4m3 values, scales) of rows v (rows, dim) fp64 by the definition."""
    rows, dim = v.shape
    q = np.empty_like(v)
    scales = np.empty((rows, -(-dim // group)))
    for i, c in enumerate(range(0, dim, group)):
        p = v[:, c:c + group]
        s = np.maximum(np.abs(p).max(1), 1e-30) / 448.0
        q[:, c:c + group], scales[:, i] = round_e4m3(p / s[:, None]), s
    return q, scales


def round_e4m3(w):
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(w), 2.0 ** -6))) - 3)
    return np.clip(np.rint(w / step) * step, -448, 448)


def check(got, ref, tol, what):
    got, ref, tol = (np.asarray(v, np.float64) for v in (got, ref, tol))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d/%d beyond the bound; worst %.3g of it" % (
        what, int(bad.sum()), bad.size, float(np.nanmax(err / np.maximum(tol, 1e-300))))
