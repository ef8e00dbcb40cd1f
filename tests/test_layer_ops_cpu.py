"""Host checks of the layer operators' C entry points (nothing is launched: fake pointers that
are never dereferenced), and of the fp64 forms their GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from selective_state_space_56_b200 import build as s6build
from selective_state_space_56_b200 import ops
from tests import layer_ref as ref

OK, NULL, DIMS, ALIGN, DTYPE, WORKSPACE, FLAGS = 0, -1, -2, -3, -4, -5, -8
P = 16 * 1024  # a fake, aligned, never dereferenced address


@pytest.fixture(scope="module")
def lib():
    s6build.build()
    return ops.load_library()


def fwd(lib, dims=(2, 3, 100), ck=None, ckb=0, i=0, o=0, flags=0, **kw):
    a = dict(x=P, gate=P, bias=None, z=None, h0=None, y=P, last=None)
    a.update(kw)
    return lib.mamba_gated_scan_fwd(a["x"], a["gate"], a["bias"], a["z"], a["h0"], a["y"], a["last"],
                                    ck, ckb, ops.GatedDims(*dims), i, o, flags, None)


def bwd(lib, dims=(2, 5000, 100), ws=P, wsb=1 << 40, ck=None, ckb=0, i=0, flags=0, **kw):
    a = dict(x=P, gate=P, bias=None, z=None, h0=None, dy=P, dlast=None, dx=P, dg=P, dz=None, db=None,
             dh0=None)
    a.update(kw)
    return lib.mamba_gated_scan_bwd(a["x"], a["gate"], a["bias"], a["z"], a["h0"], a["dy"], a["dlast"],
                                    a["dx"], a["dg"], a["dz"], a["db"], a["dh0"], ck, ckb,
                                    ops.GatedDims(*dims), i, ws, wsb, flags, None)


@pytest.mark.parametrize("field", ["x", "gate", "y"])
def test_gated_forward_null(lib, field):
    assert fwd(lib, **{field: None}) == NULL


@pytest.mark.parametrize("field", ["x", "gate", "bias", "z", "h0", "y", "last"])
def test_gated_forward_alignment(lib, field):
    assert fwd(lib, **{field: P + 8}) == ALIGN


@pytest.mark.parametrize("dims", [(0, 3, 8), (2, 0, 8), (2, 3, -1), (1 << 40, 1 << 40, 8), (1, 1, 1 << 62),
                                  (1 << 16, 1 << 16, 8)])
def test_gated_dims(lib, dims):
    assert fwd(lib, dims=dims) == DIMS
    assert bwd(lib, dims=dims) == DIMS
    assert lib.mamba_gated_scan_checkpoints_size(ops.GatedDims(*dims)) == 0
    assert lib.mamba_gated_scan_bwd_workspace_size(ops.GatedDims(*dims)) == 0


def test_gated_other_refusals(lib):
    assert fwd(lib, i=2) == DTYPE and fwd(lib, o=-1) == DTYPE and bwd(lib, i=7) == DTYPE
    assert fwd(lib, flags=1) == FLAGS and bwd(lib, flags=4) == FLAGS
    need = ops.gated_scan_checkpoints_size(2, 3, 100)
    assert need > 0 and fwd(lib, ck=P, ckb=need - 1) == WORKSPACE
    assert fwd(lib, ck=P + 4, ckb=need) == ALIGN


@pytest.mark.parametrize("field", ["x", "gate", "dy", "dx", "dg"])
def test_gated_backward_null(lib, field):
    assert bwd(lib, **{field: None}) == NULL


def test_gated_backward_gradients_match_inputs(lib):
    assert bwd(lib, z=P) == NULL and bwd(lib, dz=P) == NULL
    assert bwd(lib, bias=P) == NULL and bwd(lib, db=P) == NULL
    assert bwd(lib, bias=P, db=P, flags=2) == NULL  # given decays: the bias has no gradient
    assert bwd(lib, ws=None, wsb=0) == WORKSPACE
    assert bwd(lib, dh0=P + 2) == ALIGN
    need = ops.gated_scan_checkpoints_size(2, 5000, 100)
    assert bwd(lib, ck=P, ckb=need - 4) == WORKSPACE


def test_gated_update_refusals(lib):
    f = lambda st=P, x=P, g=P, y=P, b=2, d=8, dt=1, fl=0: lib.mamba_gated_state_update(  # noqa: E731
        st, x, g, None, None, y, b, d, dt, fl, None)
    assert [f(st=None), f(x=None), f(g=None), f(y=None)] == [NULL] * 4
    assert [f(b=0), f(d=0), f(b=1 << 40, d=1 << 40)] == [DIMS] * 3
    assert f(dt=3) == DTYPE and f(fl=1) == FLAGS and f(y=P + 1) == ALIGN


def test_norm_refusals(lib):
    def f(x=P, r=None, w=P, o=P, ro=None, rows=2, dim=64, xt=0, rt=0, ot=0):
        return lib.mamba_add_rms_norm_fwd(x, r, w, 1e-5, o, ro, rows, dim, xt, rt, ot, None)

    def f8(x=P, q=P, s=P, dim=64):
        return lib.mamba_add_rms_norm_fp8(x, None, P, 1e-5, q, s, None, 2, dim, 0, 0, None)

    def fb(d=P, v=P, dx=P, dw=P, rows=2, dim=64, ws=P, wsb=1 << 30):
        return lib.mamba_add_rms_norm_bwd(d, v, P, None, 1e-5, dx, None, dw, rows, dim, 0, 0, ws, wsb, None)

    assert [f(x=None), f(w=None), f(o=None), f(r=P)] == [NULL] * 4
    assert [f(rows=-1), f(dim=0), f(dim=16385), f(rows=1 << 33)] == [DIMS] * 4
    assert [f(xt=2), f(rt=2), f(ot=2)] == [DTYPE] * 3
    assert f(o=P + 4) == ALIGN
    assert [f8(q=None), f8(s=None)] == [NULL] * 2 and f8(dim=40) == DIMS
    assert [fb(d=None), fb(v=None), fb(dx=None), fb(dw=None)] == [NULL] * 4
    assert fb(ws=None) == WORKSPACE and fb(wsb=8) == WORKSPACE and fb(dim=0) == DIMS
    assert lib.mamba_add_rms_norm_bwd_workspace_size(2, 0) == 0


def test_fp8_refusals(lib):
    def q(x=P, o=P, s=P, b=1, d=64, L=4, cm=0, dt=0):
        return lib.mamba_fp8_quantize(x, o, s, b, d, L, cm, dt, None)

    def w(x=P, n=4, k=32, dt=0):
        return lib.mamba_fp8_quantize_weight(x, P, P, n, k, dt, None)

    def lin(x=P, xs=P, wq=P, ws=P, o=P, t=4, n=8, k=32, L=0, dt=0):
        return lib.mamba_fp8_linear(x, xs, wq, ws, o, t, n, k, L, dt, None)

    assert [q(x=None), q(o=None), q(s=None)] == [NULL] * 3
    assert [q(d=8), q(d=40), q(b=-1, L=-4), q(cm=1, b=70000), q(b=1 << 40, L=1 << 40)] == [DIMS] * 5
    assert q(dt=2) == DTYPE and q(s=P + 8) == ALIGN
    assert w(x=None) == NULL and [w(n=0), w(k=24)] == [DIMS] * 2 and w(dt=5) == DTYPE
    assert [lin(x=None), lin(xs=None), lin(wq=None), lin(ws=None), lin(o=None)] == [NULL] * 5
    assert [lin(t=-1), lin(n=0), lin(k=24), lin(L=-1), lin(L=3), lin(t=1 << 32)] == [DIMS] * 6
    assert lin(dt=9) == DTYPE and lin(wq=P + 8) == ALIGN


def test_wrappers_refuse_cpu_tensors():
    import torch
    x = torch.zeros(2, 16, 4)
    for call in (lambda: ops.gated_scan_fwd(x, x), lambda: ops.gated_scan_bwd(x, x, x),
                 lambda: ops.gated_state_update(x[..., 0], x[..., 0], x[..., 0]),
                 lambda: ops.add_rms_norm_fwd(x, torch.ones(4)), lambda: ops.add_rms_norm_fp8(x, torch.ones(4)),
                 lambda: ops.add_rms_norm_bwd(x, x, torch.ones(4)), lambda: ops.fp8_quantize(x[0]),
                 lambda: ops.fp8_quantize_weight(x[0]),
                 lambda: ops.fp8_linear(x[0], x[0], x[0], x[0])):
        with pytest.raises(ValueError):
            call()


# ---- the fp64 forms themselves ----------------------------------------------------------


def _problem(decay, z, seed=0, L=9):
    r = np.random.default_rng(seed)
    x, gate, dy = (r.standard_normal((2, 3, L)) for _ in range(3))
    if decay:
        gate = r.uniform(-0.3, 1.0, gate.shape)
    return dict(x=x, gate=gate, bias=None if decay else r.standard_normal(3),
                z=r.standard_normal(x.shape) if z else None, h0=r.standard_normal((2, 3))), dy, \
        r.standard_normal((2, 3))


@pytest.mark.parametrize("decay", [False, True])
@pytest.mark.parametrize("z", [False, True])
def test_reference_gradients_against_differences(decay, z):
    p, dy, dlast = _problem(decay, z)

    def loss(q):
        f = ref.gated_forward(q["x"], q["gate"], q["bias"], q["z"], q["h0"], decay)
        return (f["y"] * dy).sum() + (f["last"] * dlast).sum()

    g, _ = ref.gated_backward(p["x"], p["gate"], dy, p["bias"], p["z"], p["h0"], dlast, decay)
    names = dict(x="dx", gate="dgate", bias="dgate_bias", z="dz", h0="dinitial_state")
    eps = 1e-5
    for name, grad in names.items():
        if p[name] is None:
            assert g[grad] is None
            continue
        for i in np.ndindex(p[name].shape):
            up, down = dict(p), dict(p)
            up[name], down[name] = p[name].copy(), p[name].copy()
            up[name][i] += eps
            down[name][i] -= eps
            assert abs((loss(up) - loss(down)) / (2 * eps) - g[grad][i]) < 1e-7, (name, i)


def test_reference_is_the_gated_rnn_of_the_selective_scan():
    """The sigmoid form is the exact zero-order-hold scan with N = 1, A = -1, B = C = 1 (Mamba,
    Selection mechanism), as the scan's oracle computes it."""
    import oracle
    p, _, _ = _problem(False, False, L=12)
    one = np.ones((2, 1, 12))
    y, _ = oracle.selective_scan(p["x"], p["gate"], -np.ones((3, 1)), one, one, delta_bias=p["bias"], zoh=True)
    f = ref.gated_forward(p["x"], p["gate"], p["bias"])
    assert np.abs(f["y"] - y).max() < 1e-12


def test_reference_e4m3_rounding_is_torchs():
    import torch
    v = torch.cat([torch.linspace(-448, 448, 4001), torch.logspace(-12, 2, 500), torch.zeros(1)])
    want = v.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_e4m3(v.double().numpy()), want)


def test_reference_norm_gradients_against_differences():
    r = np.random.default_rng(1)
    v, w, dout, dres = r.standard_normal((2, 5)), r.standard_normal(5), r.standard_normal((2, 5)), r.standard_normal((2, 5))
    loss = lambda v, w: (ref.rms_norm(v, w, 1e-5)[0] * dout).sum() + (v * dres).sum()  # noqa: E731
    dv, dw = ref.rms_norm_backward(dout, v, w, dres, 1e-5)
    eps = 1e-6
    for i in np.ndindex(v.shape):
        d = np.zeros_like(v)
        d[i] = eps
        assert abs((loss(v + d, w) - loss(v - d, w)) / (2 * eps) - dv[i]) < 1e-7
    for i in range(5):
        d = np.zeros_like(w)
        d[i] = eps
        assert abs((loss(v, w + d) - loss(v, w - d)) / (2 * eps) - dw[i]) < 1e-7


def test_ctypes_signatures_take_addresses(lib):
    assert ctypes.sizeof(ops.GatedDims) == 24
