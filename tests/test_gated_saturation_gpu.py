"""Gradients and states of the gated recurrence where the gate is far from zero, relative to their own
size: s = sigmoid(v) for a long memory (v down to -40) and 1 - s for an open gate (v up to 40) are
far below 1 there, and neither may be formed from the rounding of the other.

Tolerance (u = 2^-24), for rows of a few steps.  t = fma(gate, -log2 e, -bias log2 e) is off by
3 u log2 e (|gate| + |bias|), so 2^t and with it the smaller of s and 1 - s by 3 u (|gate| + |bias|)
relative; ex2.approx and rcp.approx add 2^-22 and 2^-23, their sum and product 2 u: each of s and
1 - s is off by rho = 2^-22 (2 + |gate| + |bias|) relative at most.  A single step's gradients
  dx = s dh,  dgate = dh (x - h0) s (1 - s),  dh = dy + dlast
are products of at most five such factors, each rounded once: 2 rho + 8 u relative.  dh0 is formed as
(1 - s) dy + (1 - s) dlast, so its bound is relative to those two."""
import numpy as np
import pytest
import torch

from selective_state_space_56_b200 import ops
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
LEVELS = (-40.0, -20.0, -17.0, -12.0, -8.0, -2.0, -0.25, 0.0, 0.25, 2.0, 8.0, 12.0, 17.0, 20.0, 40.0)


def check_rel(got, want, rel, what):
    got = got.double().cpu().numpy().reshape(want.shape)
    ref.check(got, want, rel * np.abs(want) + 1e-37, what)


def problem(b, d, L, level, bias, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(x=n(b, d, L), gate=level + 0.1 * n(b, d, L), dy=n(b, d, L), h0=n(b, d), dlast=n(b, d), bias=None)
    if bias:  # half of the level in the bias
        p["gate"] -= 0.5 * level
        p["bias"] = torch.full((d,), 0.5 * level)
    return p


def gates(p):
    gate = p["gate"].double().numpy()
    b = np.zeros(gate.shape[1]) if p["bias"] is None else p["bias"].double().numpy()
    v = gate + b[:, None]
    return ref.sigmoid(v), ref.sigmoid(-v), 2.0 ** -22 * (2 + np.abs(gate) + np.abs(b)[:, None])


@pytest.mark.parametrize("bias", [False, True], ids=["gate", "gate_and_bias"])
@pytest.mark.parametrize("level", LEVELS)
@pytest.mark.parametrize("rows", [300, 5000], ids=["team", "alone"])
def test_one_step(cuda_ok, rows, level, bias):
    """Rows of a single step: every gradient is a product, so the bound is relative."""
    p = problem(1, rows, 1, level, bias, seed=rows)
    c = {k: None if v is None else v.to(DEV) for k, v in p.items()}
    s, a, rho = (v[0, :, 0] for v in gates(p))
    x, h0 = p["x"].double().numpy()[0, :, 0], p["h0"].double().numpy()[0]
    dh = p["dy"].double().numpy()[0, :, 0] + p["dlast"].double().numpy()[0]
    # dh = dy + dlast is one fp32 addition: relative error u; x - h0 likewise
    rel = 2 * rho + 8 * U
    g = ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], c["bias"], None, c["h0"], c["dlast"])
    check_rel(g["dx"], s * dh, rel, "dx")
    both = np.abs(p["dy"].double().numpy()[0, :, 0]) + np.abs(p["dlast"].double().numpy()[0])
    ref.check(g["dinitial_state"].double().cpu().numpy()[0], a * dh, rel * a * both + 1e-37, "dinitial_state")
    check_rel(g["dgate"], dh * (x - h0) * s * a, rel, "dgate")
    if bias:
        check_rel(g["dgate_bias"], dh * (x - h0) * s * a, rel, "dgate_bias")
    # the forward's two terms are relative to their own sizes
    tol = (rho + 4 * U) * (s * np.abs(x) + a * np.abs(h0)) + 1e-37
    y, last = ops.gated_scan_fwd(c["x"], c["gate"], c["bias"], None, c["h0"], return_last_state=True)
    want = s * x + a * h0
    ref.check(y.double().cpu().numpy()[0, :, 0], want, tol, "y")
    ref.check(last.double().cpu().numpy()[0], want, tol, "last")
    state = c["h0"].clone()
    out = ops.gated_state_update(state, c["x"][..., 0].contiguous(), c["gate"][..., 0].contiguous(), c["bias"])
    ref.check(state.double().cpu().numpy()[0], want, tol, "updated state")
    ref.check(out.double().cpu().numpy()[0], want, tol, "updated y")


@pytest.mark.parametrize("z", [False, True], ids=["no_z", "z"])
@pytest.mark.parametrize("level", [-20.0, -14.0, -10.0])
@pytest.mark.parametrize("shape", [(1, 2500, 257), (2, 30, 700), (1, 3, 9000)], ids=lambda s: "%dx%dx%d" % s)
def test_long_memories(cuda_ok, shape, level, z):
    """Rows of many steps whose states hardly decay: dx and dgate are s times sums of order one, so
    their errors are relative to s."""
    b, d, L = shape
    p = problem(b, d, L, level, True, seed=L)
    p["z"] = torch.randn(b, d, L, generator=torch.Generator().manual_seed(7)) if z else None
    c = {k: None if v is None else v.to(DEV) for k, v in p.items()}
    n = lambda k: None if p[k] is None else p[k].double().numpy()  # noqa: E731
    got = ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], c["bias"], c["z"], c["h0"], c["dlast"])
    f = ref.gated_forward(n("x"), n("gate"), n("bias"), n("z"), n("h0"))
    zf, (s, a, rho) = f["zf"], gates(p)
    gy, M = n("dy") * zf, np.empty_like(zf)
    dh, e, m = np.empty_like(gy), n("dlast"), np.abs(n("dlast"))
    for t in range(L - 1, -1, -1):
        dh[..., t], M[..., t] = gy[..., t] + e, np.abs(gy[..., t]) + m
        e, m = a[..., t] * dh[..., t], a[..., t] * M[..., t]
    prev = np.concatenate([n("h0")[..., None], f["h"][..., :-1]], -1)
    # Each decay is off by u / 2 + s rho, a composition is rounded at most three times a step on its
    # way (lane, warp, chunk) and silu is off by 2^-22 (3 + |z|): sums of L terms of magnitude M are
    # off by at most their share below; s and 1 - s as above.
    zr = 0.0 if p["z"] is None else 2.0 ** -22 * (3 + np.abs(n("z")))
    sums = (L * (4 * U + (s * rho).max()) + 40 * U) * M.max() + np.max(zr * np.abs(gy)) * L
    ref.check(got["dx"].double().cpu().numpy(), s * dh, s * sums + (2 * rho + 8 * U) * np.abs(s * dh), "dx")
    states = f["E"].max() + 8 * U * f["M"].max()
    dgate = dh * (n("x") - prev) * s * a
    tol = s * (sums * (np.abs(n("x")) + np.abs(prev)) + states * M) + (2 * rho + 12 * U) * np.abs(dgate)
    ref.check(got["dgate"].double().cpu().numpy(), dgate, tol + 4 * U * s * M * (np.abs(n("x")) + np.abs(prev)), "dgate")
