"""Thin ctypes binding over the C ABI in include/mamba_s6.h (argument marshalling only).

Every function here checks that its tensors sit on one CUDA device with the
layouts the ABI expects, allocates any output the caller did not pass (with
torch), and forwards raw device pointers plus the current torch stream to
``libmamba_s6.so``.  All arithmetic runs in the library's CUDA kernels; there is
no fallback: if the library is missing or the ABI rejects the call, a
``MambaError`` is raised.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmamba_s6.so")

MAMBA_F32, MAMBA_BF16 = 0, 1
MAMBA_FLAG_EXACT_ZOH = 1
MAMBA_FLAG_GIVEN_DECAY = 2
_DTYPES = {torch.float32: MAMBA_F32, torch.bfloat16: MAMBA_BF16}


class MambaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (where, status_string(status), status))


class ScanDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("dim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("seqlen", ctypes.c_int64)]


class GatedDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("dim", ctypes.c_int64), ("seqlen", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None
_native = None


def _load_native(lib):
    """The native marshalling of the layer operators' calls, or None where it is not built for
    this torch."""
    path = os.path.join(_HERE, "_native-%s.so" % torch.__version__)
    if not os.path.exists(path):
        return None
    try:
        spec = importlib.util.spec_from_file_location("_native", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except ImportError:
        return None
    if mod.torch_version != torch.__version__:
        return None
    mod.set_error(MambaError)
    mod.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in mod.names()})
    return mod


def load_library():
    """Load libmamba_s6.so (build it first with ``python -m selective_state_space_56_b200.build``)."""
    global _lib, _native
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError("libmamba_s6.so is not built (run: python -m "
                                  "selective_state_space_56_b200.build)")
            lib = ctypes.CDLL(LIB_PATH)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
            lib.mamba_selective_scan_workspace_size.restype = ctypes.c_size_t
            lib.mamba_selective_scan_workspace_size.argtypes = [ScanDims]
            lib.mamba_selective_scan_fwd.restype = i32
            lib.mamba_selective_scan_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp,
                                                     ScanDims, i32, i32, vp, ctypes.c_size_t, vp]
            lib.mamba_selective_scan_bwd_workspace_size.restype = ctypes.c_size_t
            lib.mamba_selective_scan_bwd_workspace_size.argtypes = [ScanDims]
            lib.mamba_selective_scan_bwd.restype = i32
            lib.mamba_selective_scan_bwd.argtypes = [vp] * 8 + [i32] + [vp] * 9 + [
                ScanDims, i32, vp, ctypes.c_size_t, vp]
            lib.mamba_selective_scan_bwd_ex.restype = i32
            lib.mamba_selective_scan_bwd_ex.argtypes = [vp] * 8 + [i32] + [vp] * 9 + [
                ScanDims, i32, vp, ctypes.c_size_t, ctypes.c_uint, vp]
            u32 = ctypes.c_uint
            lib.mamba_selective_scan_fwd_ex.restype = i32
            lib.mamba_selective_scan_fwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, vp,
                                                        vp, ScanDims, i32, i32, vp,
                                                        ctypes.c_size_t, u32, vp]
            lib.mamba_selective_scan_fwd_train.restype = i32
            lib.mamba_selective_scan_fwd_train.argtypes = [vp] * 8 + [i32, vp, vp, ScanDims, i32,
                                                               i32, vp, ctypes.c_size_t, vp,
                                                               ctypes.c_size_t, vp]
            lib.mamba_selective_scan_bwd_from_checkpoints.restype = i32
            lib.mamba_selective_scan_bwd_from_checkpoints.argtypes = [vp] * 8 + [i32] + [vp] * 9 + [
                ScanDims, i32, vp, ctypes.c_size_t, vp]
            lib.mamba_selective_scan_fwd_train_ex.restype = i32
            lib.mamba_selective_scan_fwd_train_ex.argtypes = [vp] * 8 + [
                i32, vp, vp, ScanDims, i32, i32, vp, ctypes.c_size_t, vp, ctypes.c_size_t, u32, vp]
            lib.mamba_selective_scan_bwd_from_checkpoints_ex.restype = i32
            lib.mamba_selective_scan_bwd_from_checkpoints_ex.argtypes = [vp] * 8 + [i32] + [vp] * 9 + [
                ScanDims, i32, vp, ctypes.c_size_t, u32, vp]
            lib.mamba_selective_scan_fwd_init.restype = i32
            lib.mamba_selective_scan_fwd_init.argtypes = [vp] * 8 + [i32] + [vp] * 3 + [
                ScanDims, i32, i32, vp, ctypes.c_size_t, u32, vp]
            lib.mamba_selective_scan_summary.restype = i32
            lib.mamba_selective_scan_summary.argtypes = [vp] * 6 + [i32, vp, vp, ScanDims, i32, vp,
                                                                 ctypes.c_size_t, u32, vp]
            lib.mamba_selective_scan_fold.restype = i32
            lib.mamba_selective_scan_fold.argtypes = [vp] * 4 + [i64] * 4 + [vp, vp, vp]
            lib.mamba_selective_state_update_ex.restype = i32
            lib.mamba_selective_state_update_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                            i32, vp, i64, i64, i64, i32, u32, vp]
            lib.mamba_causal_conv1d_fwd.restype = i32
            lib.mamba_causal_conv1d_fwd.argtypes = [vp] * 6 + [i64, i64, i64, i32, i32, i32, vp]
            lib.mamba_causal_conv1d_update.restype = i32
            lib.mamba_causal_conv1d_update.argtypes = [vp] * 5 + [i64, i64, i32, i32, i32, vp]
            lib.mamba_causal_conv1d_bwd.restype = i32
            lib.mamba_causal_conv1d_bwd.argtypes = [vp] * 9 + [i64, i64, i64, i32, i32, i32, vp]
            lib.mamba_selective_state_update.restype = i32
            lib.mamba_selective_state_update.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                                                         vp, i64, i64, i64, i32, vp]
            size, f32 = ctypes.c_size_t, ctypes.c_float
            for name in ("checkpoints", "bwd_workspace"):
                fn = getattr(lib, "mamba_gated_scan_%s_size" % name)
                fn.restype, fn.argtypes = size, [GatedDims]
            lib.mamba_diag_gated_team.restype = i32
            lib.mamba_diag_gated_team.argtypes = [GatedDims, i32] + [ctypes.POINTER(ctypes.c_int)] * 2
            lib.mamba_add_rms_norm_bwd_workspace_size.restype = size
            lib.mamba_add_rms_norm_bwd_workspace_size.argtypes = [i64, i64]
            for name, args in (
                    ("gated_scan_fwd", [vp] * 8 + [size, GatedDims, i32, i32, u32, vp]),
                    ("gated_scan_bwd", [vp] * 13 + [size, GatedDims, i32, vp, size, u32, vp]),
                    ("gated_state_update", [vp] * 6 + [i64, i64, i32, u32, vp]),
                    ("add_rms_norm_fwd", [vp] * 3 + [f32, vp, vp, i64, i64, i32, i32, i32, vp]),
                    ("add_rms_norm_fp8", [vp] * 3 + [f32, vp, vp, vp, i64, i64, i32, i32, vp]),
                    ("add_rms_norm_bwd", [vp] * 4 + [f32] + [vp] * 3 + [i64, i64, i32, i32, vp,
                                                                        size, vp]),
                    ("fp8_quantize", [vp] * 3 + [i64, i64, i64, i32, i32, vp]),
                    ("fp8_quantize_weight", [vp] * 3 + [i64, i64, i32, vp]),
                    ("fp8_linear", [vp] * 5 + [i64] * 4 + [i32, vp])):
                fn = getattr(lib, "mamba_" + name)
                fn.restype, fn.argtypes = i32, args
            lib.mamba_status_string.restype = ctypes.c_char_p
            lib.mamba_status_string.argtypes = [i32]
            lib.mamba_check_device_error.restype = i32
            lib.mamba_check_device_error.argtypes = [i32, vp]
            lib.mamba_diag_wait_timeout.restype = i32
            lib.mamba_diag_wait_timeout.argtypes = [i64, vp]
            lib.mamba_diag_wait_timeout_in.restype = i32
            lib.mamba_diag_wait_timeout_in.argtypes = [i32, i64, vp]
            lib.mamba_diag_exp2.restype = i32
            lib.mamba_diag_exp2.argtypes = [vp, vp, vp, vp, i64, vp]
            lib.mamba_diag_throughput.restype = i32
            lib.mamba_diag_throughput.argtypes = [i32, i64, i64, vp, vp]
            lib.mamba_abi_version.restype = i32
            lib.mamba_abi_version.argtypes = []
            _native = _load_native(lib)
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    try:
        return load_library().mamba_status_string(int(status)).decode()
    except ImportError:
        return "status %d" % status


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(t, name, device, shape=None, dtypes=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))


def check_device_error(clear: bool = True, device=None) -> None:
    """Raise MambaError if a bounded device-side wait gave up since the last clear."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        rc = load_library().mamba_check_device_error(int(bool(clear)), _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_check_device_error")


def diag_wait_timeout(limit_cycles: int = 2_000_000, device=None, part: int = 0) -> None:
    """Launch one bounded device wait that nothing completes (it gives up after
    limit_cycles SM clocks and sets the device error word of the scans, part 0, the projection,
    1, or the gated recurrence, 2); for testing detection."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        rc = load_library().mamba_diag_wait_timeout_in(int(part), int(limit_cycles), _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_diag_wait_timeout_in")


def diag_exp2(x):
    """2^x of a float32 CUDA tensor via (FMA-pipe polynomial, SFU ex2.approx, exp2f)."""
    if x.dtype != torch.float32 or x.device.type != "cuda" or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    outs = [torch.empty_like(x) for _ in range(3)]
    with torch.cuda.device(x.device):
        rc = load_library().mamba_diag_exp2(_ptr(x), _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]),
                                            x.numel(), _stream_handle(x.device))
    if rc != 0:
        raise MambaError(rc, "mamba_diag_exp2")
    return tuple(outs)


THROUGHPUT_KINDS = {"sfu_ex2": 0, "ffma": 1, "ffma2": 2}


def diag_throughput(kind: str, blocks: int, iters: int, sink):
    """Launch the pipe-throughput probe (kind "sfu_ex2", "ffma" or "ffma2") on the current
    stream; sink is a float32 CUDA tensor of at least blocks * 256 elements.  Returns the
    number of fp32 results the launch computes (the caller times it)."""
    k = THROUGHPUT_KINDS[kind]
    if sink.dtype != torch.float32 or sink.device.type != "cuda" or sink.numel() < blocks * 256:
        raise ValueError("sink must be a float32 CUDA tensor of at least blocks * 256 elements")
    with torch.cuda.device(sink.device):
        rc = load_library().mamba_diag_throughput(k, int(blocks), int(iters), _ptr(sink),
                                                  _stream_handle(sink.device))
    if rc != 0:
        raise MambaError(rc, "mamba_diag_throughput")
    return blocks * 256 * iters * (16 if k == 2 else 8)


def selective_scan_workspace_size(batch: int, dim: int, dstate: int, seqlen: int) -> int:
    """Bytes of workspace ``mamba_selective_scan_fwd`` needs for these sizes (0 if none)."""
    return int(load_library().mamba_selective_scan_workspace_size(
        ScanDims(batch, dim, dstate, seqlen)))


def selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True,
                       out_dtype=None, y=None, last_state=None, return_last_state=False,
                       workspace=None, exact_zoh=False, initial_state=None, checkpoints=None):
    """Fused selective scan.  u, delta, z: (batch, dim, L); A: (dim, N) fp32;
    B, C: (batch, N, L); D, delta_bias: (dim) fp32.  Returns y (batch, dim, L)
    [and last_state (batch, dim, N) fp32].  exact_zoh: Bbar = (exp(Delta A) - 1) / A * B
    instead of Delta * B.  initial_state: (batch, dim, N) fp32 state before the sequence
    (zero when None).  checkpoints: a uint8 CUDA tensor of at least
    selective_scan_bwd_workspace_size(...) bytes to record the backward's checkpoints in
    (a training forward, also with exact_zoh; not with initial_state)."""
    if not isinstance(u, torch.Tensor) or u.dim() != 3:
        raise ValueError("u must be a (batch, dim, L) tensor")
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("selective_scan_fwd runs on CUDA tensors only")
    b, d, L = u.shape
    N = A.shape[1] if A.dim() == 2 else -1
    in_dt = u.dtype
    if in_dt not in _DTYPES:
        raise ValueError("unsupported input dtype %s" % in_dt)
    out_dt = in_dt if out_dtype is None else out_dtype
    if out_dt not in _DTYPES:
        raise ValueError("unsupported output dtype %s" % out_dt)
    _check(u, "u", dev, (b, d, L), (in_dt,))
    _check(delta, "delta", dev, (b, d, L), (in_dt,))
    _check(z, "z", dev, (b, d, L), (in_dt,))
    _check(A, "A", dev, (d, N), (torch.float32,))
    _check(B, "B", dev, (b, N, L), (in_dt,))
    _check(C, "C", dev, (b, N, L), (in_dt,))
    _check(D, "D", dev, (d,), (torch.float32,))
    _check(delta_bias, "delta_bias", dev, (d,), (torch.float32,))
    if y is None:
        y = torch.empty((b, d, L), dtype=out_dt, device=dev)
    _check(y, "y", dev, (b, d, L), (out_dt,))
    if last_state is None and return_last_state:
        last_state = torch.empty((b, d, N), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", dev, (b, d, N), (torch.float32,))
    _check(initial_state, "initial_state", dev, (b, d, N), (torch.float32,))
    lib = load_library()
    dims = ScanDims(b, d, N, L)
    need = int(lib.mamba_selective_scan_workspace_size(dims))
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
            int(bool(delta_softplus)), _ptr(y), _ptr(last_state), dims, _DTYPES[in_dt],
            _DTYPES[out_dt], _ptr(workspace), ws_bytes)
    flags = MAMBA_FLAG_EXACT_ZOH if exact_zoh else 0
    if checkpoints is not None and initial_state is not None:
        raise ValueError("checkpoints are recorded by a forward from h = 0 only")
    with torch.cuda.device(dev):
        if checkpoints is not None:
            _check(checkpoints, "checkpoints", dev)
            rc = lib.mamba_selective_scan_fwd_train_ex(
                *args, _ptr(checkpoints), checkpoints.numel() * checkpoints.element_size(),
                flags, _stream_handle(dev))
        elif initial_state is not None:
            rc = lib.mamba_selective_scan_fwd_init(*args[:9], _ptr(initial_state), *args[9:], flags,
                                                   _stream_handle(dev))
        elif exact_zoh:
            rc = lib.mamba_selective_scan_fwd_ex(*args, flags, _stream_handle(dev))
        else:
            rc = lib.mamba_selective_scan_fwd(*args, _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_selective_scan_fwd")
    if return_last_state:
        return y, last_state
    return y


def selective_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None,
                       delta_softplus=True, workspace=None, checkpoints=None, exact_zoh=False):
    """Gradients of ``selective_scan_fwd`` for the upstream gradient dy (batch, dim, L),
    in the inputs' dtype.  Returns a dict with du, ddelta, dz (input dtype, dz None
    without a gate), dA (dim, N), dB, dC (batch, N, L), dD, ddelta_bias (dim) in fp32
    (None where the input is None).  checkpoints: the buffer a training forward
    (selective_scan_fwd(..., checkpoints=...)) filled for the same inputs; the backward
    then skips its own checkpointing pass (with the exact_zoh the forward used).
    exact_zoh: the gradients of the exact zero-order-hold forward
    (``selective_scan_fwd(..., exact_zoh=True)``)."""
    if not isinstance(u, torch.Tensor) or u.dim() != 3:
        raise ValueError("u must be a (batch, dim, L) tensor")
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("selective_scan_bwd runs on CUDA tensors only")
    b, d, L = u.shape
    N = A.shape[1] if A.dim() == 2 else -1
    dt = u.dtype
    if dt not in _DTYPES:
        raise ValueError("unsupported input dtype %s" % dt)
    for t, name, shape, dts in ((u, "u", (b, d, L), (dt,)), (delta, "delta", (b, d, L), (dt,)),
                                (z, "z", (b, d, L), (dt,)), (dy, "dy", (b, d, L), (dt,)),
                                (A, "A", (d, N), (torch.float32,)), (B, "B", (b, N, L), (dt,)),
                                (C, "C", (b, N, L), (dt,)), (D, "D", (d,), (torch.float32,)),
                                (delta_bias, "delta_bias", (d,), (torch.float32,))):
        _check(t, name, dev, shape, dts)
    f32 = torch.float32
    g = dict(du=torch.empty((b, d, L), dtype=dt, device=dev),
             ddelta=torch.empty((b, d, L), dtype=dt, device=dev),
             dz=None if z is None else torch.empty((b, d, L), dtype=dt, device=dev),
             dA=torch.empty((d, N), dtype=f32, device=dev),
             dB=torch.empty((b, N, L), dtype=f32, device=dev),
             dC=torch.empty((b, N, L), dtype=f32, device=dev),
             dD=None if D is None else torch.empty(d, dtype=f32, device=dev),
             ddelta_bias=None if delta_bias is None else torch.empty(d, dtype=f32, device=dev))
    lib = load_library()
    dims = ScanDims(b, d, N, L)
    if checkpoints is not None:
        _check(checkpoints, "checkpoints", dev)
        with torch.cuda.device(dev):
            rc = lib.mamba_selective_scan_bwd_from_checkpoints_ex(
                _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                _ptr(delta_bias), int(bool(delta_softplus)), _ptr(dy), _ptr(g["du"]),
                _ptr(g["ddelta"]), _ptr(g["dz"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]),
                _ptr(g["dD"]), _ptr(g["ddelta_bias"]), dims, _DTYPES[dt], _ptr(checkpoints),
                checkpoints.numel() * checkpoints.element_size(),
                MAMBA_FLAG_EXACT_ZOH if exact_zoh else 0, _stream_handle(dev))
        if rc != 0:
            raise MambaError(rc, "mamba_selective_scan_bwd_from_checkpoints")
        return g
    need = int(lib.mamba_selective_scan_bwd_workspace_size(dims))
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with torch.cuda.device(dev):
        rc = lib.mamba_selective_scan_bwd_ex(
            _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
            int(bool(delta_softplus)), _ptr(dy), _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dz"]),
            _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["ddelta_bias"]),
            dims, _DTYPES[dt], _ptr(workspace), ws_bytes,
            MAMBA_FLAG_EXACT_ZOH if exact_zoh else 0, _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_selective_scan_bwd_ex")
    return g


def selective_scan_bwd_workspace_size(batch: int, dim: int, dstate: int, seqlen: int) -> int:
    """Bytes of workspace ``mamba_selective_scan_bwd`` needs (the chunk checkpoints)."""
    return int(load_library().mamba_selective_scan_bwd_workspace_size(
        ScanDims(batch, dim, dstate, seqlen)))


def selective_state_update(state, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                           delta_softplus=True, y=None, exact_zoh=False):
    """One decode token, in place on ``state`` (batch, dim, N) fp32.
    u, delta, z: (batch, dim); B, C: (batch, N); A: (dim, N).  Returns y (batch, dim).
    exact_zoh: Bbar = (exp(Delta A) - 1) / A * B instead of Delta * B."""
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be a (batch, dim, N) tensor")
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("selective_state_update runs on CUDA tensors only")
    b, d, N = state.shape
    io_dt = u.dtype
    if io_dt not in _DTYPES:
        raise ValueError("unsupported dtype %s" % io_dt)
    _check(state, "state", dev, (b, d, N), (torch.float32,))
    _check(u, "u", dev, (b, d), (io_dt,))
    _check(delta, "delta", dev, (b, d), (io_dt,))
    _check(z, "z", dev, (b, d), (io_dt,))
    _check(A, "A", dev, (d, N), (torch.float32,))
    _check(B, "B", dev, (b, N), (io_dt,))
    _check(C, "C", dev, (b, N), (io_dt,))
    _check(D, "D", dev, (d,), (torch.float32,))
    _check(delta_bias, "delta_bias", dev, (d,), (torch.float32,))
    if y is None:
        y = torch.empty((b, d), dtype=io_dt, device=dev)
    _check(y, "y", dev, (b, d), (io_dt,))
    args = (_ptr(state), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
            _ptr(delta_bias), int(bool(delta_softplus)), _ptr(y), b, d, N, _DTYPES[io_dt])
    lib = load_library()
    with torch.cuda.device(dev):
        if exact_zoh:
            rc = lib.mamba_selective_state_update_ex(*args, MAMBA_FLAG_EXACT_ZOH,
                                                     _stream_handle(dev))
        else:
            rc = lib.mamba_selective_state_update(*args, _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_selective_state_update")
    return y


def causal_conv1d_fwd(x, weight, bias=None, initial_state=None, silu=True, out=None,
                      return_final_state=False):
    """Causal depthwise conv1d (+ SiLU).  x: (batch, dim, L) bf16/fp32; weight: (dim, K)
    fp32, 1 <= K <= 4; bias: (dim) fp32; initial_state: (batch, dim, K-1) x.dtype.
    Returns out (batch, dim, L) [and the final state (batch, dim, K-1)]."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a (batch, dim, L) tensor")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("causal_conv1d_fwd runs on CUDA tensors only")
    b, d, L = x.shape
    K = weight.shape[1] if weight.dim() == 2 else -1
    dt = x.dtype
    if dt not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dt)
    _check(x, "x", dev, (b, d, L), (dt,))
    _check(weight, "weight", dev, (d, K), (torch.float32,))
    _check(bias, "bias", dev, (d,), (torch.float32,))
    _check(initial_state, "initial_state", dev, (b, d, K - 1), (dt,))
    if out is None:
        out = torch.empty((b, d, L), dtype=dt, device=dev)
    _check(out, "out", dev, (b, d, L), (dt,))
    fin = None
    if return_final_state and K > 1:
        fin = torch.empty((b, d, K - 1), dtype=dt, device=dev)
    with torch.cuda.device(dev):
        rc = load_library().mamba_causal_conv1d_fwd(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(out), _ptr(fin),
            b, d, L, K, int(bool(silu)), _DTYPES[dt], _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_causal_conv1d_fwd")
    if return_final_state:
        return out, fin
    return out


def causal_conv1d_update(conv_state, x, weight, bias=None, silu=True, out=None):
    """One decode token: conv_state (batch, dim, K-1) is updated in place; x (batch, dim).
    Returns out (batch, dim)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a (batch, dim) tensor")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("causal_conv1d_update runs on CUDA tensors only")
    b, d = x.shape
    K = weight.shape[1] if weight.dim() == 2 else -1
    dt = x.dtype
    if dt not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dt)
    _check(x, "x", dev, (b, d), (dt,))
    _check(weight, "weight", dev, (d, K), (torch.float32,))
    _check(bias, "bias", dev, (d,), (torch.float32,))
    _check(conv_state, "conv_state", dev, (b, d, K - 1), (dt,))
    if out is None:
        out = torch.empty((b, d), dtype=dt, device=dev)
    _check(out, "out", dev, (b, d), (dt,))
    with torch.cuda.device(dev):
        rc = load_library().mamba_causal_conv1d_update(
            _ptr(conv_state), _ptr(x), _ptr(weight), _ptr(bias), _ptr(out), b, d, K,
            int(bool(silu)), _DTYPES[dt], _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_causal_conv1d_update")
    return out


def causal_conv1d_bwd(x, weight, dout, bias=None, initial_state=None, silu=True):
    """Gradients of sum(out * dout) for ``causal_conv1d_fwd`` with the same x, weight, bias,
    initial_state and silu.  Returns a dict: dx (batch, dim, L) x.dtype, dweight (dim, K)
    fp32, dbias (dim) fp32 (None without a bias), dinitial_state (batch, dim, K-1) x.dtype
    (None without an initial state)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a (batch, dim, L) tensor")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("causal_conv1d_bwd runs on CUDA tensors only")
    b, d, L = x.shape
    K = weight.shape[1] if weight.dim() == 2 else -1
    dt = x.dtype
    if dt not in _DTYPES:
        raise ValueError("unsupported dtype %s" % dt)
    _check(x, "x", dev, (b, d, L), (dt,))
    _check(dout, "dout", dev, (b, d, L), (dt,))
    _check(weight, "weight", dev, (d, K), (torch.float32,))
    _check(bias, "bias", dev, (d,), (torch.float32,))
    _check(initial_state, "initial_state", dev, (b, d, K - 1), (dt,))
    g = dict(dx=torch.empty((b, d, L), dtype=dt, device=dev),
             dweight=torch.empty((d, K), dtype=torch.float32, device=dev),
             dbias=None if bias is None else torch.empty(d, dtype=torch.float32, device=dev),
             dinitial_state=None if (initial_state is None or K < 2)
             else torch.empty((b, d, K - 1), dtype=dt, device=dev))
    with torch.cuda.device(dev):
        rc = load_library().mamba_causal_conv1d_bwd(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(dout), _ptr(g["dx"]),
            _ptr(g["dweight"]), _ptr(g["dbias"]), _ptr(g["dinitial_state"]), b, d, L, K,
            int(bool(silu)), _DTYPES[dt], _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_causal_conv1d_bwd")
    return g


def selective_scan_summary(u, delta, A, B, C, delta_bias=None, delta_softplus=True,
                           exact_zoh=False, workspace=None):
    """Summary of a sequence segment for the associative combine: (h_end (batch, dim, N),
    delta_sum (batch, dim)), the state after the segment from zero and its summed step."""
    if not isinstance(u, torch.Tensor) or u.dim() != 3:
        raise ValueError("u must be a (batch, dim, L) tensor")
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("selective_scan_summary runs on CUDA tensors only")
    b, d, L = u.shape
    N = A.shape[1] if A.dim() == 2 else -1
    dt = u.dtype
    if dt not in _DTYPES:
        raise ValueError("unsupported input dtype %s" % dt)
    for t, name, shape, dts in ((u, "u", (b, d, L), (dt,)), (delta, "delta", (b, d, L), (dt,)),
                                (A, "A", (d, N), (torch.float32,)), (B, "B", (b, N, L), (dt,)),
                                (C, "C", (b, N, L), (dt,)),
                                (delta_bias, "delta_bias", (d,), (torch.float32,))):
        _check(t, name, dev, shape, dts)
    h_end = torch.empty((b, d, N), dtype=torch.float32, device=dev)
    dsum = torch.empty((b, d), dtype=torch.float32, device=dev)
    lib = load_library()
    dims = ScanDims(b, d, N, L)
    need = int(lib.mamba_selective_scan_workspace_size(dims))
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with torch.cuda.device(dev):
        rc = lib.mamba_selective_scan_summary(
            _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(delta_bias),
            int(bool(delta_softplus)), _ptr(h_end), _ptr(dsum), dims, _DTYPES[dt],
            _ptr(workspace), ws_bytes, MAMBA_FLAG_EXACT_ZOH if exact_zoh else 0,
            _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_selective_scan_summary")
    return h_end, dsum


def selective_scan_fold(h_ends, delta_sums, A, h0=None, return_delta_sum=False):
    """Apply summaries h_ends (count, batch, dim, N), delta_sums (count, batch, dim) in order
    to h0 (batch, dim, N) or zero; returns the resulting state [and the total step]."""
    dev = A.device
    if dev.type != "cuda":
        raise ValueError("selective_scan_fold runs on CUDA tensors only")
    cnt, b, d, N = h_ends.shape
    _check(h_ends, "h_ends", dev, (cnt, b, d, N), (torch.float32,))
    _check(delta_sums, "delta_sums", dev, (cnt, b, d), (torch.float32,))
    _check(A, "A", dev, (d, N), (torch.float32,))
    _check(h0, "h0", dev, (b, d, N), (torch.float32,))
    h_out = torch.empty((b, d, N), dtype=torch.float32, device=dev)
    s_out = torch.empty((b, d), dtype=torch.float32, device=dev) if return_delta_sum else None
    with torch.cuda.device(dev):
        rc = load_library().mamba_selective_scan_fold(
            _ptr(h_ends) if cnt else None, _ptr(delta_sums) if cnt else None, _ptr(A), _ptr(h0),
            cnt, b, d, N, _ptr(h_out), _ptr(s_out), _stream_handle(dev))
    if rc != 0:
        raise MambaError(rc, "mamba_selective_scan_fold")
    return (h_out, s_out) if return_delta_sum else h_out


# ---- The gated linear recurrence --------------------------------------------------------


def _cuda_device(t, name, where, ndim):
    if not isinstance(t, torch.Tensor) or t.dim() not in ndim:
        raise ValueError("%s must be a tensor of %s dimensions" % (name, " or ".join(map(str, ndim))))
    if not t.is_cuda:
        raise ValueError("%s runs on CUDA tensors only" % where)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.get_device()


def _is(t, name, dev, shape, dtype):
    """t is a contiguous tensor of this shape and dtype on CUDA device dev; its address."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    _check(t, name, torch.device("cuda", dev), shape, (dtype,))
    raise TypeError("%s must be a torch.Tensor" % name)


def _output(t, name, like, dev, shape, dtype):
    """The caller's output, checked, or a new one; and its address."""
    if t is None:
        t = _new(like, shape, dtype)
        return t, t.data_ptr()
    return t, _is(t, name, dev, shape, dtype)


def _maybe(t, name, dev, shape, dtype):
    return None if t is None else _is(t, name, dev, shape, dtype)


def _buffer(t, name, dev):
    """Address and bytes of a caller's buffer (or None)."""
    if t is None:
        return None, 0
    _check(t, name, torch.device("cuda", dev))
    return t.data_ptr(), t.numel() * t.element_size()


def _dtype(dt, what):
    code = _DTYPES.get(dt)
    if code is None:
        raise ValueError("unsupported %s dtype %s" % (what, dt))
    return code


def _new(like, shape, dtype):
    """A new contiguous tensor on like's device (torch.empty_like, where it will do, takes half
    the time of torch.empty)."""
    if like.shape == shape and like.is_contiguous():
        return torch.empty_like(like) if like.dtype is dtype else torch.empty_like(like, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=like.device)


# The raw handle of a device's current stream: torch.cuda.current_stream builds a Stream object
# around it (2.2 us against 0.1).
_calls = {}
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(name, dev, *args):
    """One library call on device dev's current stream; raises MambaError for a non-zero status."""
    fn = _calls.get(name) or _calls.setdefault(name, getattr(load_library(), name))
    if dev == _current_device():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != 0:
        raise MambaError(rc, name)


def gated_scan_checkpoints_size(batch: int, dim: int, seqlen: int) -> int:
    """Bytes of the checkpoints ``gated_scan_fwd`` can record for ``gated_scan_bwd``."""
    return int(load_library().mamba_gated_scan_checkpoints_size(GatedDims(batch, dim, seqlen)))


def gated_scan_bwd_workspace_size(batch: int, dim: int, seqlen: int) -> int:
    """Bytes of workspace ``gated_scan_bwd`` needs for these sizes."""
    return int(load_library().mamba_gated_scan_bwd_workspace_size(GatedDims(batch, dim, seqlen)))


def _workspace(workspace, need, like, dev):
    """(the tensor, which the caller keeps until the call has returned, its address, its bytes)"""
    if workspace is None and need > 0:
        workspace = _new(like, need, torch.uint8)
    return (workspace, *_buffer(workspace, "workspace", dev))


def diag_gated_team(batch: int, dim: int, seqlen: int, backward: bool = False) -> tuple:
    """(warps of a CTA, CTAs of a cluster) that walk a row together for these sizes."""
    warps, ctas = ctypes.c_int(), ctypes.c_int()
    rc = load_library().mamba_diag_gated_team(GatedDims(batch, dim, seqlen), int(bool(backward)),
                                              ctypes.byref(warps), ctypes.byref(ctas))
    if rc != 0:
        raise MambaError(rc, "mamba_diag_gated_team")
    return warps.value, ctas.value


def gated_scan_fwd(x, gate, gate_bias=None, z=None, initial_state=None, given_decay=False,
                   out_dtype=None, y=None, last_state=None, return_last_state=False,
                   checkpoints=None):
    """Gated linear recurrence h_t = (1 - s_t) h_{t-1} + s_t x_t with s_t = sigmoid(gate_t +
    gate_bias), or h_t = gate_t h_{t-1} + x_t with given_decay; y_t = h_t silu(z_t) (h_t
    without z).  x, gate, z: (batch, dim, L); gate_bias: (dim) fp32; initial_state: (batch,
    dim) fp32 (zero when None).  Returns y (batch, dim, L) [and last_state (batch, dim) fp32].
    checkpoints: a uint8 CUDA tensor of gated_scan_checkpoints_size(...) bytes to record what
    ``gated_scan_bwd`` starts from."""
    flags = MAMBA_FLAG_GIVEN_DECAY if given_decay else 0
    if _native is not None and y is None and last_state is None and out_dtype is None:
        r = _native.gated_scan_fwd(x, gate, gate_bias, z, initial_state, checkpoints, flags,
                                   bool(return_last_state))
        if r is not None:
            return r if return_last_state else r[0]
    dev = _cuda_device(x, "x", "gated_scan_fwd", (3,))
    b, d, L = shape = x.shape
    in_dt, f32 = x.dtype, torch.float32
    out_dt = in_dt if out_dtype is None else out_dtype
    in_code, out_code = _dtype(in_dt, "input"), _dtype(out_dt, "output")
    y, yp = _output(y, "y", x, dev, shape, out_dt)
    lp = None
    if last_state is not None or return_last_state:
        last_state, lp = _output(last_state, "last_state", x, dev, (b, d), f32)
    ck, ck_bytes = _buffer(checkpoints, "checkpoints", dev)
    _run("mamba_gated_scan_fwd", dev, x.data_ptr(), _is(gate, "gate", dev, shape, in_dt),
         _maybe(gate_bias, "gate_bias", dev, (d,), f32), _maybe(z, "z", dev, shape, in_dt),
         _maybe(initial_state, "initial_state", dev, (b, d), f32), yp, lp, ck, ck_bytes,
         GatedDims(b, d, L), in_code, out_code, flags)
    return (y, last_state) if return_last_state else y


def gated_scan_bwd(x, gate, dy, gate_bias=None, z=None, initial_state=None, dlast_state=None,
                   given_decay=False, checkpoints=None, workspace=None):
    """Gradients of sum(y dy) + sum(last_state dlast_state) for ``gated_scan_fwd`` with the
    same inputs.  Returns a dict: dx, dgate, dz (batch, dim, L) in the inputs' dtype (dz None
    without z), dgate_bias (dim) fp32 (None without a bias or with given_decay),
    dinitial_state (batch, dim) fp32.  checkpoints: the buffer the forward filled for the same
    inputs; without it the backward makes one more pass over x and gate."""
    flags = MAMBA_FLAG_GIVEN_DECAY if given_decay else 0
    if _native is not None and workspace is None:
        r = _native.gated_scan_bwd(x, gate, dy, gate_bias, z, initial_state, dlast_state, checkpoints,
                                   flags)
        if r is not None:
            return dict(dx=r[0], dgate=r[1], dz=r[2], dgate_bias=r[3], dinitial_state=r[4])
    dev = _cuda_device(x, "x", "gated_scan_bwd", (3,))
    b, d, L = shape = x.shape
    dt, f32 = x.dtype, torch.float32
    code = _dtype(dt, "input")
    g = dict(dx=_new(x, shape, dt), dgate=_new(x, shape, dt),
             dz=None if z is None else _new(x, shape, dt),
             dgate_bias=None if gate_bias is None or given_decay else _new(x, (d,), f32),
             dinitial_state=_new(x, (b, d), f32))
    ck, ck_bytes = _buffer(checkpoints, "checkpoints", dev)
    dims = GatedDims(b, d, L)
    need = (_lib or load_library()).mamba_gated_scan_bwd_workspace_size(dims)
    workspace, ws, ws_bytes = _workspace(workspace, need, x, dev)
    _run("mamba_gated_scan_bwd", dev, x.data_ptr(), _is(gate, "gate", dev, shape, dt),
         _maybe(gate_bias, "gate_bias", dev, (d,), f32), _maybe(z, "z", dev, shape, dt),
         _maybe(initial_state, "initial_state", dev, (b, d), f32), _is(dy, "dy", dev, shape, dt),
         _maybe(dlast_state, "dlast_state", dev, (b, d), f32), g["dx"].data_ptr(),
         g["dgate"].data_ptr(), _addr(g["dz"]), _addr(g["dgate_bias"]), g["dinitial_state"].data_ptr(), ck, ck_bytes,
         dims, code, ws, ws_bytes, flags)
    return g


def gated_state_update(state, x, gate, gate_bias=None, z=None, given_decay=False, y=None):
    """One decode token of the gated recurrence, in place on ``state`` (batch, dim) fp32;
    x, gate, z: (batch, dim).  Returns y (batch, dim)."""
    flags = MAMBA_FLAG_GIVEN_DECAY if given_decay else 0
    if _native is not None and y is None:
        r = _native.gated_state_update(state, x, gate, gate_bias, z, flags)
        if r is not None:
            return r
    dev = _cuda_device(state, "state", "gated_state_update", (2,))
    b, d = shape = state.shape
    f32 = torch.float32
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dt = x.dtype
    code = _dtype(dt, "input")
    xp = _is(x, "x", dev, shape, dt)
    y, yp = _output(y, "y", x, dev, shape, dt)
    _run("mamba_gated_state_update", dev, _is(state, "state", dev, shape, f32), xp,
         _is(gate, "gate", dev, shape, dt), _maybe(gate_bias, "gate_bias", dev, (d,), f32),
         _maybe(z, "z", dev, shape, dt), yp, b, d, code, flags)
    return y


def _addr(t):
    return None if t is None else t.data_ptr()


# ---- Residual addition with RMS norm ----------------------------------------------------


def _norm_inputs(x, weight, residual, residual_out, where):
    """(device, dim, rows, dtype codes, the addresses of x, residual, weight, residual_out, and
    residual_out itself)"""
    dev = _cuda_device(x, "x", where, (2, 3))
    shape, dt = x.shape, x.dtype
    d = shape[-1]
    code = rcode = _dtype(dt, "input")
    rt, rp = dt, None
    if residual is not None:
        if not isinstance(residual, torch.Tensor):
            raise TypeError("residual must be a torch.Tensor")
        rt = residual.dtype
        rcode = _dtype(rt, "residual")
        rp = _is(residual, "residual", dev, shape, rt)
    op = None
    if residual is not None or residual_out is not None:
        like = x if residual is None else residual
        residual_out, op = _output(residual_out, "residual_out", like, dev, shape, rt)
    rows = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    return (dev, d, rows, code, rcode, x.data_ptr(), rp,
            _is(weight, "weight", dev, (d,), torch.float32), op, residual_out)


def add_rms_norm_fwd(x, weight, residual=None, eps=1e-5, out_dtype=None, out=None,
                     residual_out=None):
    """v = residual + x (in the residual's dtype); out = v / sqrt(mean v^2 + eps) * weight.
    x, residual: (..., dim) of 2 or 3 dimensions, weight: (dim) fp32.  Returns (out, v);
    without a residual v is x."""
    if _native is not None and out_dtype is None and out is None and residual_out is None:
        r = _native.add_rms_norm_fwd(x, weight, residual, eps)
        if r is not None:
            return r if residual is not None else (r[0], x)
    dev, d, rows, code, rcode, xp, rp, wp, op, residual_out = _norm_inputs(
        x, weight, residual, residual_out, "add_rms_norm_fwd")
    out_dt = x.dtype if out_dtype is None else out_dtype
    ocode = _dtype(out_dt, "output")
    out, outp = _output(out, "out", x, dev, x.shape, out_dt)
    _run("mamba_add_rms_norm_fwd", dev, xp, rp, wp, eps, outp, op, rows, d, code, rcode, ocode)
    return out, x if residual_out is None else residual_out


def add_rms_norm_fp8(x, weight, residual=None, eps=1e-5, q=None, scales=None, residual_out=None):
    """``add_rms_norm_fwd`` with the output in e4m3: returns (q (..., dim) float8_e4m3fn,
    scales (..., ceil(dim / 128)) fp32, v), out = q * scale.  dim a multiple of 16."""
    if _native is not None and q is None and scales is None and residual_out is None:
        r = _native.add_rms_norm_fp8(x, weight, residual, eps)
        if r is not None:
            return r if residual is not None else (r[0], r[1], x)
    dev, d, rows, code, rcode, xp, rp, wp, op, residual_out = _norm_inputs(
        x, weight, residual, residual_out, "add_rms_norm_fp8")
    q, scales, qp, sp = _fp8_outputs(x, q, scales, x.shape[:-1], d, dev)
    _run("mamba_add_rms_norm_fp8", dev, xp, rp, wp, eps, qp, sp, op, rows, d, code, rcode)
    return q, scales, x if residual_out is None else residual_out


def _fp8_outputs(like, q, scales, lead, d, dev):
    """e4m3 rows and their scales (new ones where None), and their addresses."""
    qs, ss = (*lead, d), (*lead, (d + 127) // 128)
    q, qp = _output(q, "q", like, dev, qs, torch.float8_e4m3fn)
    scales, sp = _output(scales, "scales", like, dev, ss, torch.float32)
    return q, scales, qp, sp


def add_rms_norm_bwd(dout, residual_out, weight, dresidual_out=None, eps=1e-5, workspace=None):
    """Gradients of ``add_rms_norm_fwd`` from the v it returned.  dout: (..., dim) in x's
    dtype; dresidual_out: the gradient arriving at v from elsewhere, in its dtype.  Returns a
    dict: dx (dout's dtype), dresidual (v's dtype; the same tensor where the dtypes agree),
    dweight (dim) fp32."""
    if _native is not None and workspace is None:
        r = _native.add_rms_norm_bwd(dout, residual_out, weight, dresidual_out, eps)
        if r is not None:
            return dict(dx=r[0], dresidual=r[0] if r[1] is None else r[1], dweight=r[2])
    dev = _cuda_device(dout, "dout", "add_rms_norm_bwd", (2, 3))
    shape, dt, f32 = dout.shape, dout.dtype, torch.float32
    d = shape[-1]
    code = _dtype(dt, "input")
    if not isinstance(residual_out, torch.Tensor):
        raise TypeError("residual_out must be a torch.Tensor")
    rt = residual_out.dtype
    rcode = _dtype(rt, "residual")
    dx = _new(dout, shape, dt)
    dres = None if rt == dt else _new(dout, shape, rt)
    dw = _new(dout, (d,), f32)
    rows = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    need = (_lib or load_library()).mamba_add_rms_norm_bwd_workspace_size(rows, d)
    workspace, ws, ws_bytes = _workspace(workspace, need, dout, dev)
    _run("mamba_add_rms_norm_bwd", dev, dout.data_ptr(),
         _is(residual_out, "residual_out", dev, shape, rt), _is(weight, "weight", dev, (d,), f32),
         _maybe(dresidual_out, "dresidual_out", dev, shape, rt), eps, dx.data_ptr(), _addr(dres),
         dw.data_ptr(), rows, d, code, rcode, ws, ws_bytes)
    return dict(dx=dx, dresidual=dx if dres is None else dres, dweight=dw)


# ---- 8-bit operands and the projections -------------------------------------------------


def fp8_quantize(x, channel_major=False, q=None, scales=None):
    """Activations to e4m3 with a scale for each token and 128 channels: x (tokens, dim), or
    (batch, dim, L) with channel_major (the layout of the scans' y).  Returns (q (tokens, dim)
    float8_e4m3fn, scales (tokens, ceil(dim / 128)) fp32), tokens = batch * L in the latter
    case.  dim a multiple of 16."""
    if _native is not None and q is None and scales is None:
        r = _native.fp8_quantize(x, bool(channel_major))
        if r is not None:
            return r
    dev = _cuda_device(x, "x", "fp8_quantize", (3,) if channel_major else (2,))
    code = _dtype(x.dtype, "input")
    b, d, L = x.shape if channel_major else (1, x.shape[1], x.shape[0])
    q, scales, qp, sp = _fp8_outputs(x, q, scales, (b * L,), d, dev)
    _run("mamba_fp8_quantize", dev, x.data_ptr(), qp, sp, b, d, L,
         1 if channel_major else 0, code)
    return q, scales


def fp8_quantize_weight(w):
    """Weights (n, k) to e4m3 with a scale for each block of 128 x 128: returns (q (n, k)
    float8_e4m3fn, scales (ceil(n / 128), ceil(k / 128)) fp32).  k a multiple of 16."""
    dev = _cuda_device(w, "w", "fp8_quantize_weight", (2,))
    code = _dtype(w.dtype, "input")
    n, k = w.shape
    q = _new(w, (n, k), torch.float8_e4m3fn)
    scales = _new(w, ((n + 127) // 128, (k + 127) // 128), torch.float32)
    _run("mamba_fp8_quantize_weight", dev, w.data_ptr(), q.data_ptr(),
         scales.data_ptr(), n, k, code)
    return q, scales


def fp8_linear(xq, x_scales, wq, w_scales, out_dtype=torch.bfloat16, channel_major_seqlen=None,
               out=None):
    """The projection x w^T of operands in e4m3 (``fp8_quantize`` / ``add_rms_norm_fp8`` and
    ``fp8_quantize_weight``): xq (tokens, k), wq (n, k).  Returns (tokens, n), or with
    channel_major_seqlen = L the layout of the conv's and the scans' inputs, (tokens / L, n, L)."""
    code = _dtype(out_dtype, "output")
    if _native is not None and out is None:
        L = channel_major_seqlen
        if L is None or (type(L) is int and L > 0):
            r = _native.fp8_linear(xq, x_scales, wq, w_scales, code, L or 0)
            if r is not None:
                return r
    dev = _cuda_device(xq, "xq", "fp8_linear", (2,))
    t, k = xq.shape
    n = wq.shape[0] if isinstance(wq, torch.Tensor) and wq.dim() == 2 else -1
    f8, f32, kb = torch.float8_e4m3fn, torch.float32, (k + 127) // 128
    L, shape = 0, (t, n)
    if channel_major_seqlen is not None:
        L = int(channel_major_seqlen)
        if L < 1 or t % L != 0:
            raise ValueError("channel_major_seqlen must be positive and divide the %d tokens" % t)
        shape = (t // L, n, L)
    ptrs = (_is(xq, "xq", dev, (t, k), f8), _is(x_scales, "x_scales", dev, (t, kb), f32),
            _is(wq, "wq", dev, (n, k), f8), _is(w_scales, "w_scales", dev, ((n + 127) // 128, kb), f32))
    out, outp = _output(out, "out", xq, dev, shape, out_dtype)
    _run("mamba_fp8_linear", dev, *ptrs, outp, t, n, k, L, code)
    return out
