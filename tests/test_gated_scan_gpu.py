"""Gated linear recurrence on the GPU against the fp64 recurrence (tests/layer_ref.py, which
derives the error bounds used here): forward, backward, decode update, both forms, split
rows, odd lengths, graphs, streams, edge values."""
import numpy as np
import pytest
import torch

from selective_state_space_56_b200 import ops
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def problem(b, d, L, dtype, decay, z=True, bias=True, h0=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]

    def normal(*s):
        return torch.randn(*s, generator=g)

    p = dict(x=normal(b, d, L).to(dt), dy=normal(b, d, L).to(dt),
             z=normal(b, d, L).to(dt) if z else None,
             h0=normal(b, d) if h0 else None, dlast=normal(b, d) if h0 else None)
    if decay:
        p["gate"] = (1.0 - 1.2 * torch.rand(b, d, L, generator=g) ** 3).to(dt)  # in [-0.2, 1]
        p["bias"] = None
    else:
        p["gate"] = normal(b, d, L).to(dt)
        p["bias"] = -4.0 * torch.rand(d, generator=g) if bias else None
    return p


def dev(p):
    return {k: None if v is None else v.to(DEV) for k, v in p.items()}


def compare(p, dtype, decay, out_dtype=None, checkpoints=True):
    c, h = dev(p), {k: n64(v) for k, v in p.items()}
    b, d, L = p["x"].shape
    ck = torch.empty(ops.gated_scan_checkpoints_size(b, d, L), dtype=torch.uint8, device=DEV)
    y, last = ops.gated_scan_fwd(c["x"], c["gate"], c["bias"], c["z"], c["h0"], given_decay=decay,
                                 out_dtype=None if out_dtype is None else TYPES[out_dtype],
                                 return_last_state=True, checkpoints=ck)
    f = ref.gated_forward(h["x"], h["gate"], h["bias"], h["z"], h["h0"], decay)
    zr = 0.0 if p["z"] is None else 2.0 ** -22 * (3.0 + np.abs(h["z"]))
    tol = np.abs(f["zf"]) * (f["E"] + (zr + 4 * ref.U) * f["M"])
    ref.check(n64(y), f["y"], tol + ref.half_step(out_dtype or dtype, f["y"]), "y")
    ref.check(n64(last), f["last"], f["E_last"] + 4 * ref.U * np.abs(f["last"]), "last_state")
    got = ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], c["bias"], c["z"], c["h0"], c["dlast"],
                             given_decay=decay, checkpoints=ck if checkpoints else None)
    g, t = ref.gated_backward(h["x"], h["gate"], h["dy"], h["bias"], h["z"], h["h0"], h["dlast"],
                              decay)
    for k in g:
        if g[k] is None:
            assert got[k] is None, k
            continue
        kind = dtype if k in ("dx", "dgate", "dz") else "fp32"
        ref.check(n64(got[k]), g[k], t[k] * 1.01 + ref.half_step(kind, g[k]), k)
    return y, last, got


SHAPES = [(1, 1, 1), (2, 3, 2), (1, 5, 7), (2, 3, 8), (3, 7, 9), (2, 4, 255), (1, 9, 256),
          (2, 5, 257), (1, 3, 263), (2, 6, 1000), (1, 2, 4099)]


@pytest.mark.parametrize("decay", [False, True], ids=["sigmoid", "decay"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%dx%d" % s)
def test_gated_scan_shapes(cuda_ok, shape, dtype, decay):
    compare(problem(*shape, dtype, decay, seed=sum(shape)), dtype, decay)


@pytest.mark.parametrize("decay", [False, True], ids=["sigmoid", "decay"])
@pytest.mark.parametrize("z", [False, True], ids=["no_z", "z"])
@pytest.mark.parametrize("h0", [False, True], ids=["zero", "h0"])
def test_gated_scan_options(cuda_ok, decay, z, h0):
    p = problem(2, 6, 300, "bf16", decay, z=z, bias=False, h0=h0, seed=9)
    compare(p, "bf16", decay, out_dtype="fp32", checkpoints=False)
    p = problem(2, 6, 300, "fp32", decay, z=z, h0=h0, seed=10)
    compare(p, "fp32", decay, out_dtype="bf16", checkpoints=False)


@pytest.mark.parametrize("decay", [False, True], ids=["sigmoid", "decay"])
def test_gated_scan_few_long_rows(cuda_ok, decay):
    """Few long rows: a cluster of CTAs walks each; a length whose last chunk only some rows
    touch."""
    p = problem(1, 3, 70001, "fp32", decay, seed=3)
    compare(p, "fp32", decay)
    compare(p, "fp32", decay, checkpoints=False)


def test_gated_scan_enough_rows(cuda_ok):
    """Rows enough for one warp each in the backward and nearly so in the forward, ending inside a
    vector."""
    compare(problem(2, 1200, 301, "bf16", False, seed=4), "bf16", False)


@pytest.mark.parametrize("rows", [1, 20, 75, 149, 300, 700, 2400])
@pytest.mark.parametrize("L", [600, 5003])
def test_gated_scan_rows_by_teams(cuda_ok, rows, L):
    """Every way of sharing a row: clusters of 8 down to 1 CTAs, 16 down to 1 warps."""
    compare(problem(1, rows, L, "bf16", rows % 2 == 0, seed=rows), "bf16", rows % 2 == 0)


@pytest.mark.parametrize("decay", [False, True], ids=["sigmoid", "decay"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("z", [False, True], ids=["no_z", "z"])
@pytest.mark.parametrize("rows,L", [(1186, 513), (1203, 1029), (1190, 1536), (60, 2605)])
def test_gated_scan_chunks_ahead(cuda_ok, rows, L, z, dtype, decay):
    """Rows of more chunks than a warp keeps on their way, walked alone and by teams."""
    compare(problem(1, rows, L, dtype, decay, z=z, seed=rows), dtype, decay)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,L", [(1190, 777), (1190, 41), (40, 1541)])
def test_gated_scan_nan_stays_in_its_row(cuda_ok, rows, L, dtype):
    """Vectors that two rows share: what one row holds there does not reach the other."""
    p = dev(problem(1, rows, L, dtype, False, bias=False, seed=5))
    bad = {k: None if v is None else v.clone() for k, v in p.items()}
    for k in ("x", "gate", "z", "dy"):
        bad[k][0, 7] = float("nan")
    keep = [i for i in range(rows) if i != 7]
    out = []
    for c in (p, bad):
        y, last = ops.gated_scan_fwd(c["x"], c["gate"], None, c["z"], c["h0"], return_last_state=True)
        g = ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], None, c["z"], c["h0"], c["dlast"])
        out.append([y, last, g["dx"], g["dgate"], g["dz"], g["dinitial_state"]])
    for clean, got in zip(*out):
        assert torch.equal(clean[:, keep], got[:, keep])
    assert torch.isnan(out[1][0][0, 7]).all()


def test_gated_scan_gradients_against_differences(cuda_ok):
    """Central differences of the GPU forward (fp32, summed in fp64) in random directions."""
    p = problem(1, 4, 40, "fp32", False, seed=5)
    c = dev(p)
    g = ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], c["bias"], c["z"], c["h0"], c["dlast"])
    names = dict(x="dx", gate="dgate", z="dz", bias="dgate_bias", h0="dinitial_state")

    def loss(q):
        y, last = ops.gated_scan_fwd(q["x"], q["gate"], q["bias"], q["z"], q["h0"],
                                     return_last_state=True)
        return float((y.double() * c["dy"].double()).sum() + (last.double() * c["dlast"].double()).sum())

    eps = 2.0 ** -6
    for name, grad in names.items():
        v = torch.randn(c[name].shape, generator=torch.Generator().manual_seed(6)).to(DEV)
        up, down = dict(c), dict(c)
        up[name], down[name] = c[name] + eps * v, c[name] - eps * v
        diff = (loss(up) - loss(down)) / (2 * eps)
        want = float((g[grad].double() * v.double()).sum())
        # third-order term of the difference (eps^2 / 6 times a third derivative of order |v|^3,
        # under 2 here) and the forward's fp32 error (160 sums off by under 1e-5 each) over 2 eps
        scale = float((g[grad].double().abs() * v.double().abs()).sum())
        assert abs(diff - want) <= 2e-3 * scale + 160 * 1e-6 / eps, (name, diff, want)


def test_gated_scan_equal_calls_equal_bits(cuda_ok):
    c = dev(problem(2, 70, 3001, "bf16", False, seed=7))
    run = lambda: ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], c["bias"], c["z"], c["h0"])  # noqa: E731
    first = run()
    for _ in range(3):
        again = run()
        for k in first:
            assert torch.equal(first[k], again[k]), k


def test_gated_scan_neighbouring_rows_do_not_leak(cuda_ok):
    """A row of NaN or infinities leaves the rows beside it as they are, at a length where they
    share vectors."""
    c = dev(problem(1, 5, 259, "bf16", False, seed=8))
    clean = ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], c["bias"], c["z"], c["h0"])
    y0 = ops.gated_scan_fwd(c["x"], c["gate"], c["bias"], c["z"], c["h0"])
    for value in (float("nan"), float("inf")):
        q = dict(c)
        for k in ("x", "gate", "dy", "z"):
            q[k] = c[k].clone()
            q[k][0, 2] = value
        y = ops.gated_scan_fwd(q["x"], q["gate"], q["bias"], q["z"], q["h0"])
        g = ops.gated_scan_bwd(q["x"], q["gate"], q["dy"], q["bias"], q["z"], q["h0"])
        for r in (0, 1, 3, 4):
            assert torch.equal(y[0, r], y0[0, r])
            for k in ("dx", "dgate", "dz", "dinitial_state"):
                assert torch.equal(g[k][0, r], clean[k][0, r]), (k, r, value)
            assert torch.equal(g["dgate_bias"][r], clean["dgate_bias"][r])


def test_gated_scan_padding_and_resets(cuda_ok):
    """Given decays: a = 1, b = 0 hold the state, a = 0 forgets it (within the rounding of
    another association, which the error model bounds); saturated gates keep (s = 0) or
    replace (s = 1) it exactly."""
    x = torch.randn(1, 2, 600, generator=torch.Generator().manual_seed(1)).to(DEV)
    a = torch.full_like(x, 0.5)
    a[0, :, 300:] = 1.0
    x[0, :, 300:] = 0.0
    f = ref.gated_forward(n64(x), n64(a), decay=True)
    tol = f["E"] + 4 * ref.U * f["M"] + ref.half_step("fp32", f["h"])
    y, last = ops.gated_scan_fwd(x, a, given_decay=True, return_last_state=True)
    ref.check(n64(y), f["h"], tol, "held state")
    ref.check(n64(last), f["last"], tol[..., -1], "last held state")
    a[0, :, 100] = 0.0
    f = ref.gated_forward(n64(x[..., 100:]), n64(a[..., 100:]), decay=True)
    y = ops.gated_scan_fwd(x, a, given_decay=True)
    ref.check(n64(y[..., 100:]), f["h"], f["E"] + 4 * ref.U * f["M"] + ref.half_step("fp32", f["h"]),
              "after a reset")
    gate = torch.full_like(x, -3e4)
    h0 = torch.randn(1, 2, device=DEV)
    y = ops.gated_scan_fwd(x, gate, initial_state=h0)
    assert torch.equal(y, h0[..., None].expand_as(y))
    y = ops.gated_scan_fwd(x, -gate, initial_state=h0)
    assert torch.equal(y, x)


def test_gated_scan_empty_sequence(cuda_ok):
    x = torch.empty(2, 3, 0, device=DEV)
    h0 = torch.randn(2, 3, device=DEV)
    y, last = ops.gated_scan_fwd(x, x, initial_state=h0, return_last_state=True)
    assert y.shape == (2, 3, 0) and torch.equal(last, h0)
    _, last = ops.gated_scan_fwd(x, x, return_last_state=True)
    assert float(last.abs().max()) == 0.0
    g = ops.gated_scan_bwd(x, x, x, gate_bias=torch.zeros(3, device=DEV), dlast_state=h0)
    assert torch.equal(g["dinitial_state"], h0) and float(g["dgate_bias"].abs().max()) == 0.0


@pytest.mark.parametrize("decay", [False, True], ids=["sigmoid", "decay"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 64), (5, 1000)], ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gated_update_equals_recurrence(cuda_ok, shape, dtype, decay):
    b, d = shape
    p = problem(b, d, 5, dtype, decay, seed=b * d)
    h = {k: n64(v) for k, v in p.items()}
    f = ref.gated_forward(h["x"], h["gate"], h["bias"], h["z"], h["h0"], decay)
    state = p["h0"].to(DEV)
    for t in range(5):
        y = ops.gated_state_update(state, *(p[k][..., t].contiguous().to(DEV) for k in ("x", "gate")),
                                   gate_bias=None if p["bias"] is None else p["bias"].to(DEV),
                                   z=p["z"][..., t].contiguous().to(DEV), given_decay=decay)
        tol = f["E"][..., t] + 4 * ref.U * f["M"][..., t]
        ref.check(n64(state), f["h"][..., t], tol, "state")
        zt = h["z"][..., t]
        ref.check(n64(y), f["y"][..., t], np.abs(f["zf"][..., t]) * (tol + 2.0 ** -22 * (3 + np.abs(zt)) *
                  f["M"][..., t]) + ref.half_step(dtype, f["y"][..., t]), "y")


def test_gated_graphs_and_streams(cuda_ok):
    """A captured forward and backward, replayed on new inputs, equal the eager calls; two graphs
    with workspaces of their own replay side by side on two streams."""
    probs = [dev(problem(1, 40, 5000, "bf16", False, seed=s)) for s in (1, 2)]

    def step(c, ck):
        y, last = ops.gated_scan_fwd(c["x"], c["gate"], c["bias"], c["z"], c["h0"],
                                     return_last_state=True, checkpoints=ck)
        g = ops.gated_scan_bwd(c["x"], c["gate"], c["dy"], c["bias"], c["z"], c["h0"], checkpoints=ck)
        return dict(g, y=y, last=last)

    size = ops.gated_scan_checkpoints_size(1, 40, 5000)
    eager = [step(c, torch.empty(size, dtype=torch.uint8, device=DEV)) for c in probs]
    graphs, outs = [], []
    for c in probs:
        ck = torch.empty(size, dtype=torch.uint8, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(c, ck)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c, ck))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        for k in e:
            assert torch.equal(e[k], o[k]), k
    del graphs
