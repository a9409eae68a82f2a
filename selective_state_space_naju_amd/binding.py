"""ctypes binding of libnaju.so (argument marshalling only).

Every step of the computation runs in the HIP kernels of ``libnaju.so``;
this module checks tensor shapes/dtypes, allocates outputs and the
workspace with PyTorch, and passes raw device pointers plus the current
HIP stream through the C ABI declared in ``include/naju.h``.  If the
library is missing the import of any entry point raises -- there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libnaju.so")

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = range(5)
F32, BF16 = 0, 1
OP_SCAN_FWD, OP_SCAN_BWD, OP_BLOCK_FWD, OP_BLOCK_BWD = range(4)
D_CONV = 4

# every function the header declares (the CPU tests check the exports)
EXPORTS = ("naju_workspace_bytes", "naju_ckpt_bytes", "naju_workspace_init",
           "naju_workspace_check", "naju_scan_fwd", "naju_scan_bwd", "naju_block_fwd",
           "naju_block_bwd", "naju_scan_step", "naju_block_step", "naju_mixer_workspace_bytes",
           "naju_mixer_fwd", "naju_mixer_bwd_workspace_bytes", "naju_mixer_bwd",
           "naju_scan_fwd_noalloc", "naju_embed_fwd", "naju_embed_bwd_workspace_bytes",
           "naju_embed_bwd", "naju_distill_fwd", "naju_distill_bwd", "naju_distill_fwd_bwd",
           "naju_logits_workspace_bytes", "naju_logits_process", "naju_w4_linear", "naju_w4_quantize",
           "naju_last_error", "naju_version")


class NajuError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("naju status %d: %s" % (status, msg))
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("d_inner", ctypes.c_int64), ("d_state", ctypes.c_int64),
                ("d_conv", ctypes.c_int32), ("io", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Loads libnaju.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError("libnaju.so not found at %s; build it with "
                              "`python -m selective_state_space_naju_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        dp = ctypes.POINTER(Dims)
        L.naju_workspace_bytes.argtypes = [ctypes.c_int, dp]
        L.naju_workspace_bytes.restype = sz
        L.naju_ckpt_bytes.argtypes = [dp]
        L.naju_ckpt_bytes.restype = sz
        L.naju_workspace_init.argtypes = [vp, sz, vp]
        L.naju_workspace_init.restype = st
        L.naju_workspace_check.argtypes = [vp, sz, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.naju_workspace_check.restype = st
        L.naju_scan_fwd.argtypes = [dp] + [vp] * 11 + [sz, vp]
        L.naju_scan_fwd.restype = st
        L.naju_block_fwd.argtypes = [dp] + [vp] * 15 + [sz, vp]
        L.naju_block_fwd.restype = st
        L.naju_scan_bwd.argtypes = [dp] + [vp] * 18 + [sz, vp]
        L.naju_scan_bwd.restype = st
        L.naju_block_bwd.argtypes = [dp] + [vp] * 24 + [sz, vp]
        L.naju_block_bwd.restype = st
        L.naju_scan_step.argtypes = [dp] + [vp] * 9
        L.naju_scan_step.restype = st
        L.naju_block_step.argtypes = [dp] + [vp] * 12
        L.naju_block_step.restype = st
        L.naju_mixer_workspace_bytes.argtypes = [dp, ctypes.c_int64]
        L.naju_mixer_workspace_bytes.restype = sz
        L.naju_mixer_fwd.argtypes = [dp, ctypes.c_int64] + [vp] * 16 + [sz, vp]
        L.naju_mixer_fwd.restype = st
        L.naju_mixer_bwd_workspace_bytes.argtypes = [dp, ctypes.c_int64]
        L.naju_mixer_bwd_workspace_bytes.restype = sz
        L.naju_mixer_bwd.argtypes = [dp, ctypes.c_int64] + [vp] * 28 + [sz, vp, sz, vp]
        L.naju_mixer_bwd.restype = st
        L.naju_scan_fwd_noalloc.argtypes = [dp] + [vp] * 12
        L.naju_scan_fwd_noalloc.restype = st
        i64, i32, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        L.naju_embed_fwd.argtypes = [i64, i64, i64, i32, vp, vp, f32, vp, vp]
        L.naju_embed_fwd.restype = st
        L.naju_embed_bwd_workspace_bytes.argtypes = [i64, i64, i64]
        L.naju_embed_bwd_workspace_bytes.restype = sz
        L.naju_embed_bwd.argtypes = [i64, i64, i64, i32, vp, vp, f32, i32, vp, vp, sz, vp]
        L.naju_embed_bwd.restype = st
        L.naju_distill_fwd.argtypes = [i64, i64, i64, i32, vp, i64, vp, vp, f32] + [vp] * 3
        L.naju_distill_fwd.restype = st
        L.naju_distill_bwd.argtypes = [i64, i64, i64, i32, vp, i64, vp, vp, f32, vp, vp, vp, i64,
                                       vp]
        L.naju_distill_bwd.restype = st
        L.naju_distill_fwd_bwd.argtypes = [i64, i64, i64, i32, vp, i64, vp, vp, f32, vp, vp, vp,
                                           vp, i64, vp]
        L.naju_distill_fwd_bwd.restype = st
        L.naju_logits_workspace_bytes.argtypes = [i64]
        L.naju_logits_workspace_bytes.restype = sz
        L.naju_logits_process.argtypes = ([i64, i64, i32, vp, i64, vp, i64] + [vp] * 6 +
                                          [i64, vp, vp, vp, vp, sz, vp])
        L.naju_logits_process.restype = st
        L.naju_w4_linear.argtypes = [i64, i64, i64, i64] + [vp] * 8
        L.naju_w4_linear.restype = st
        L.naju_w4_quantize.argtypes = [i64, i64, i64, i32] + [vp] * 5
        L.naju_w4_quantize.restype = st
        L.naju_last_error.argtypes = []
        L.naju_last_error.restype = ctypes.c_char_p
        L.naju_version.argtypes = []
        L.naju_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def last_error() -> str:
    return lib().naju_last_error().decode()


def check(status: int) -> None:
    if status != OK:
        raise NajuError(status, last_error())


def check_workspace(ws) -> None:
    """Raises if a cross-workgroup wait of a call that used `ws` gave up (its
    results are then invalid).  Synchronises the workspace's device."""
    flags = ws.error_flags()
    if flags:
        raise NajuError(EHIP, "a cross-workgroup wait gave up (workspace error flags 0x%x): "
                              "results invalid" % flags)


def make_dims(batch, seqlen, d_inner, d_state, io, d_conv=D_CONV) -> Dims:
    return Dims(int(batch), int(seqlen), int(d_inner), int(d_state), int(d_conv), int(io))


def workspace_bytes(op: int, dims: Dims) -> int:
    return int(lib().naju_workspace_bytes(op, ctypes.byref(dims)))


def ckpt_bytes(dims: Dims) -> int:
    return int(lib().naju_ckpt_bytes(ctypes.byref(dims)))


def _p(t):
    return None if t is None else t.data_ptr()


def stream_handle(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev) -> int:
    """The current stream's handle on dev (a device of tensors), without building a stream
    object: 4 us less a call, which single-token calls notice."""
    index = dev.index
    if index is None:  # (no device of a GPU's tensor)
        raise ValueError("tensors must be on a GPU, got %s" % dev)
    if _raw_stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream(index)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_its_device(fn):
    """An entry point that runs with its first tensor's device current.  The library launches on
    the current device, and the default stream's handle is 0 on every device: called from another
    one, a kernel would run there, on memory that is not its own."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, **kw):
        t = args[0] if args else kw.get(first)
        device = t.get_device() if t is not None else -1  # (-1 in host memory)
        if device < 0 or device == _current_device():
            return fn(*args, **kw)
        with torch.cuda.device(device):
            return fn(*args, **kw)
    return call


class Workspace:
    """A zero-initialised device workspace (reused across calls on one stream)."""

    def __init__(self, nbytes: int, device):
        n = max(256, (int(nbytes) + 255) // 256 * 256)
        self.tensor = torch.zeros(n, dtype=torch.uint8, device=device)
        self.nbytes = n

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    def error_flags(self) -> int:
        return _error_flags(self.tensor, self.nbytes)


@_on_its_device
def _error_flags(ws: torch.Tensor, nbytes: int) -> int:
    out = ctypes.c_uint32(0)
    check(lib().naju_workspace_check(_p(ws), nbytes, stream_handle(ws.device), ctypes.byref(out)))
    return int(out.value)


_ws_cache: dict = {}


def _cached_workspace(key, nbytes, dev) -> Workspace:
    """The workspace kept for key, made at its first use.  One made under graph capture is not
    kept: its zero fill is a node of that graph and has not run for anybody else."""
    ws = _ws_cache.get(key)
    if ws is None:
        ws = Workspace(nbytes(), dev)
        if not torch.cuda.is_current_stream_capturing():
            _ws_cache[key] = ws
    return ws


def workspace(op: int, dims: Dims, device) -> Workspace:
    """Cached workspace per (device, stream, op, dims): a workspace is only ever
    reused by calls with the same layout, on one stream."""
    dev = torch.device(device)
    key = (dev.index, torch.cuda.current_stream(dev).cuda_stream, op, dims.batch, dims.seqlen,
           dims.d_inner, dims.d_state, dims.d_conv, dims.io)
    return _cached_workspace(key, lambda: workspace_bytes(op, dims), dev)


def _io_of(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("activations must be float32 or bfloat16, got %s" % t.dtype)


def _req(t, name, shape, dtype, device):
    if (t is not None and t.shape == shape and t.dtype == dtype and t.device == device
            and t.is_contiguous()):
        return t
    if t is None:
        raise ValueError("%s is required" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _opt(t, name, shape, dtype, device):
    return None if t is None else _req(t, name, shape, dtype, device)


# ------------------------------------------------------------------ entry points
@_on_its_device
def scan_fwd(h, a, b, B, C, D, x0=None, *, return_ckpt=False, ws=None, check_errors=False):
    """y, x_final (, ckpt) = naju_scan_fwd(h, a, b, B, C, D, x0).

    check_errors=True synchronises and raises if a look-back wait gave up (the
    library sets an error bit in the workspace instead of hanging)."""
    Bt, L, Di = h.shape
    N = B.shape[-1]
    dt, dev = h.dtype, h.device
    io = _io_of(h)
    for nm, t in (("h", h), ("a", a), ("b", b)):
        _req(t, nm, (Bt, L, Di), dt, dev)
    _req(B, "B", (Bt, L, N), dt, dev)
    _req(C, "C", (Bt, L, N), dt, dev)
    _req(D, "D", (Di,), torch.float32, dev)
    _opt(x0, "x0", (Bt, Di, N), torch.float32, dev)
    dims = make_dims(Bt, L, Di, N, io)
    y = torch.empty((Bt, L, Di), dtype=dt, device=dev)
    xf = torch.empty((Bt, Di, N), dtype=torch.float32, device=dev)
    ck = None
    if return_ckpt:
        ck = torch.empty(ckpt_bytes(dims) // 4, dtype=torch.float32, device=dev)
    ws = ws or workspace(OP_SCAN_FWD, dims, dev)
    check(lib().naju_scan_fwd(ctypes.byref(dims), _p(h), _p(a), _p(b), _p(B), _p(C), _p(D),
                              _p(x0), _p(y), _p(xf), _p(ck), ws.ptr, ws.nbytes,
                              stream_handle(dev)))
    if check_errors:
        check_workspace(ws)
    return (y, xf, ck) if return_ckpt else (y, xf)


@_on_its_device
def block_fwd(u, z, conv_w, a, b, B, C, D, x0=None, conv_state=None, *, return_ckpt=False,
              ws=None, check_errors=False):
    """y, x_final, conv_state_out (, ckpt) = naju_block_fwd(...) (check_errors: as for
    scan_fwd)."""
    Bt, L, Di = u.shape
    N = B.shape[-1]
    dt, dev = u.dtype, u.device
    io = _io_of(u)
    for nm, t in (("u", u), ("z", z), ("a", a), ("b", b)):
        _req(t, nm, (Bt, L, Di), dt, dev)
    _req(B, "B", (Bt, L, N), dt, dev)
    _req(C, "C", (Bt, L, N), dt, dev)
    _req(D, "D", (Di,), torch.float32, dev)
    _req(conv_w, "conv_w", (Di, D_CONV), torch.float32, dev)
    _opt(x0, "x0", (Bt, Di, N), torch.float32, dev)
    _opt(conv_state, "conv_state", (Bt, D_CONV - 1, Di), dt, dev)
    dims = make_dims(Bt, L, Di, N, io)
    y = torch.empty((Bt, L, Di), dtype=dt, device=dev)
    xf = torch.empty((Bt, Di, N), dtype=torch.float32, device=dev)
    cso = torch.empty((Bt, D_CONV - 1, Di), dtype=dt, device=dev)
    ck = None
    if return_ckpt:
        ck = torch.empty(ckpt_bytes(dims) // 4, dtype=torch.float32, device=dev)
    ws = ws or workspace(OP_BLOCK_FWD, dims, dev)
    check(lib().naju_block_fwd(ctypes.byref(dims), _p(u), _p(z), _p(conv_w), _p(conv_state),
                               _p(a), _p(b), _p(B), _p(C), _p(D), _p(x0), _p(y), _p(xf),
                               _p(cso), _p(ck), ws.ptr, ws.nbytes, stream_handle(dev)))
    if check_errors:
        check_workspace(ws)
    return (y, xf, cso, ck) if return_ckpt else (y, xf, cso)


@_on_its_device
def scan_bwd(h, a, b, B, C, D, dy, x0=None, dx_final=None, ckpt=None, *, want_dx0=True,
             ws=None):
    """Gradients of naju_scan_fwd: dict(dh, da, db, dB, dC, dD, dx0)."""
    Bt, L, Di = h.shape
    N = B.shape[-1]
    dt, dev = h.dtype, h.device
    io = _io_of(h)
    for nm, t in (("h", h), ("a", a), ("b", b), ("dy", dy)):
        _req(t, nm, (Bt, L, Di), dt, dev)
    _req(B, "B", (Bt, L, N), dt, dev)
    _req(C, "C", (Bt, L, N), dt, dev)
    _req(D, "D", (Di,), torch.float32, dev)
    _opt(x0, "x0", (Bt, Di, N), torch.float32, dev)
    _opt(dx_final, "dx_final", (Bt, Di, N), torch.float32, dev)
    dims = make_dims(Bt, L, Di, N, io)
    out = {k: torch.empty((Bt, L, Di), dtype=dt, device=dev) for k in ("dh", "da", "db")}
    out["dB"] = torch.empty((Bt, L, N), dtype=dt, device=dev)
    out["dC"] = torch.empty((Bt, L, N), dtype=dt, device=dev)
    out["dD"] = torch.empty((Di,), dtype=torch.float32, device=dev)
    out["dx0"] = torch.empty((Bt, Di, N), dtype=torch.float32, device=dev) if want_dx0 else None
    ws = ws or workspace(OP_SCAN_BWD, dims, dev)
    check(lib().naju_scan_bwd(ctypes.byref(dims), _p(h), _p(a), _p(b), _p(B), _p(C), _p(D),
                              _p(x0), _p(ckpt), _p(dy), _p(dx_final), _p(out["dh"]),
                              _p(out["da"]), _p(out["db"]), _p(out["dB"]), _p(out["dC"]),
                              _p(out["dD"]), _p(out["dx0"]), ws.ptr, ws.nbytes,
                              stream_handle(dev)))
    return out


@_on_its_device
def block_bwd(u, z, conv_w, a, b, B, C, D, dy, x0=None, dx_final=None, conv_state=None,
              ckpt=None, *, want_dx0=True, want_dconv_state=True, ws=None):
    """Gradients of naju_block_fwd: dict(du, dz, dconv_w, dconv_state, da, db, dB, dC, dD, dx0)."""
    Bt, L, Di = u.shape
    N = B.shape[-1]
    dt, dev = u.dtype, u.device
    io = _io_of(u)
    for nm, t in (("u", u), ("z", z), ("a", a), ("b", b), ("dy", dy)):
        _req(t, nm, (Bt, L, Di), dt, dev)
    _req(B, "B", (Bt, L, N), dt, dev)
    _req(C, "C", (Bt, L, N), dt, dev)
    _req(D, "D", (Di,), torch.float32, dev)
    _req(conv_w, "conv_w", (Di, D_CONV), torch.float32, dev)
    _opt(x0, "x0", (Bt, Di, N), torch.float32, dev)
    _opt(dx_final, "dx_final", (Bt, Di, N), torch.float32, dev)
    _opt(conv_state, "conv_state", (Bt, D_CONV - 1, Di), dt, dev)
    dims = make_dims(Bt, L, Di, N, io)
    out = {k: torch.empty((Bt, L, Di), dtype=dt, device=dev) for k in ("du", "dz", "da", "db")}
    out["dB"] = torch.empty((Bt, L, N), dtype=dt, device=dev)
    out["dC"] = torch.empty((Bt, L, N), dtype=dt, device=dev)
    out["dD"] = torch.empty((Di,), dtype=torch.float32, device=dev)
    out["dconv_w"] = torch.empty((Di, D_CONV), dtype=torch.float32, device=dev)
    out["dconv_state"] = (torch.empty((Bt, D_CONV - 1, Di), dtype=dt, device=dev)
                          if want_dconv_state else None)
    out["dx0"] = torch.empty((Bt, Di, N), dtype=torch.float32, device=dev) if want_dx0 else None
    ws = ws or workspace(OP_BLOCK_BWD, dims, dev)
    check(lib().naju_block_bwd(ctypes.byref(dims), _p(u), _p(z), _p(conv_w), _p(conv_state),
                               _p(a), _p(b), _p(B), _p(C), _p(D), _p(x0), _p(ckpt), _p(dy),
                               _p(dx_final), _p(out["du"]), _p(out["dz"]), _p(out["dconv_w"]),
                               _p(out["dconv_state"]), _p(out["da"]), _p(out["db"]),
                               _p(out["dB"]), _p(out["dC"]), _p(out["dD"]), _p(out["dx0"]),
                               ws.ptr, ws.nbytes, stream_handle(dev)))
    return out


@_on_its_device
def scan_step(h, a, b, B, C, D, x):
    """y = naju_scan_step(h, a, b, B, C, D, x); x ([Bt, Di, N] fp32) is updated in place."""
    Bt, Di = h.shape
    N = B.shape[-1]
    dt, dev = h.dtype, h.device
    io = _io_of(h)
    for nm, t in (("h", h), ("a", a), ("b", b)):
        _req(t, nm, (Bt, Di), dt, dev)
    _req(B, "B", (Bt, N), dt, dev)
    _req(C, "C", (Bt, N), dt, dev)
    _req(D, "D", (Di,), torch.float32, dev)
    _req(x, "x", (Bt, Di, N), torch.float32, dev)
    dims = make_dims(Bt, 1, Di, N, io)
    y = torch.empty((Bt, Di), dtype=dt, device=dev)
    check(lib().naju_scan_step(ctypes.byref(dims), _p(h), _p(a), _p(b), _p(B), _p(C), _p(D),
                               _p(x), _p(y), stream_handle(dev)))
    return y


@_on_its_device
def block_step(u, z, conv_w, conv_state, a, b, B, C, D, x):
    """y = naju_block_step(...); x and conv_state ([Bt, K-1, Di]) are updated in place."""
    Bt, Di = u.shape
    N = B.shape[-1]
    dt, dev = u.dtype, u.device
    io = _io_of(u)
    for nm, t in (("u", u), ("z", z), ("a", a), ("b", b)):
        _req(t, nm, (Bt, Di), dt, dev)
    _req(B, "B", (Bt, N), dt, dev)
    _req(C, "C", (Bt, N), dt, dev)
    _req(D, "D", (Di,), torch.float32, dev)
    _req(conv_w, "conv_w", (Di, D_CONV), torch.float32, dev)
    _req(conv_state, "conv_state", (Bt, D_CONV - 1, Di), dt, dev)
    _req(x, "x", (Bt, Di, N), torch.float32, dev)
    dims = make_dims(Bt, 1, Di, N, io)
    y = torch.empty((Bt, Di), dtype=dt, device=dev)
    check(lib().naju_block_step(ctypes.byref(dims), _p(u), _p(z), _p(conv_w), _p(conv_state),
                                _p(a), _p(b), _p(B), _p(C), _p(D), _p(x), _p(y),
                                stream_handle(dev)))
    return y


@_on_its_device
def mixer_fwd(xn, W_u, W_z, conv_w, W_a, a_bias, W_b, b_bias, W_B, W_C, D, W_out, res=None,
              conv_state=None, *, ws=None):
    """out = naju_mixer_fwd(...): the mixer layer around the block scan (bf16)."""
    Bt, L, dm = xn.shape
    Di = W_u.shape[1]
    N = W_B.shape[1]
    dt, dev = xn.dtype, xn.device
    if dt != torch.bfloat16:
        raise TypeError("the mixer layer takes bfloat16 activations and weights")
    _req(xn, "xn", (Bt, L, dm), dt, dev)
    _opt(res, "res", (Bt, L, dm), dt, dev)
    _req(W_u, "W_u", (dm, Di), dt, dev)
    _req(W_z, "W_z", (dm, Di), dt, dev)
    _req(conv_w, "conv_w", (Di, D_CONV), torch.float32, dev)
    _opt(conv_state, "conv_state", (Bt, D_CONV - 1, Di), dt, dev)
    _req(W_a, "W_a", (Di, Di), dt, dev)
    _req(W_b, "W_b", (Di, Di), dt, dev)
    _req(a_bias, "a_bias", (Di,), torch.float32, dev)
    _req(b_bias, "b_bias", (Di,), torch.float32, dev)
    _req(W_B, "W_B", (Di, N), dt, dev)
    _req(W_C, "W_C", (Di, N), dt, dev)
    _req(D, "D", (Di,), torch.float32, dev)
    _req(W_out, "W_out", (Di, dm), dt, dev)
    dims = make_dims(Bt, L, Di, N, BF16)
    out = torch.empty((Bt, L, dm), dtype=dt, device=dev)
    if ws is None:
        d = torch.device(dev)
        key = (d.index, torch.cuda.current_stream(d).cuda_stream, "mixer", Bt, L, dm, Di, N)
        ws = _cached_workspace(
            key, lambda: int(lib().naju_mixer_workspace_bytes(ctypes.byref(dims), dm)), d)
    check(lib().naju_mixer_fwd(ctypes.byref(dims), dm, _p(xn), _p(res), _p(W_u), _p(W_z),
                               _p(conv_w), _p(conv_state), _p(W_a), _p(a_bias), _p(W_b),
                               _p(b_bias), _p(W_B), _p(W_C), _p(D), _p(W_out), _p(out), ws.ptr,
                               ws.nbytes, stream_handle(dev)))
    return out


@_on_its_device
def mixer_bwd(xn, W_u, W_z, conv_w, W_a, a_bias, W_b, b_bias, W_B, W_C, D, W_out, d_out,
              conv_state=None, *, fwd_ws=None, ws=None):
    """Gradients of naju_mixer_fwd for upstream d_out (the residual's is d_out); fwd_ws:
    the Workspace a mixer_fwd call on the same inputs used (its intermediates are reused):
    dict(dxn, dW_u, dW_z, dconv_w, dconv_state, dW_a, da_bias, dW_b, db_bias, dW_B, dW_C,
    dD, dW_out), fp32 except dconv_state (bf16, only with conv_state)."""
    Bt, L, dm = xn.shape
    Di = W_u.shape[1]
    N = W_B.shape[1]
    dt, dev = xn.dtype, xn.device
    if dt != torch.bfloat16:
        raise TypeError("the mixer layer takes bfloat16 activations and weights")
    _req(d_out, "d_out", (Bt, L, dm), dt, dev)
    for nm, t, shp in (("xn", xn, (Bt, L, dm)), ("W_u", W_u, (dm, Di)), ("W_z", W_z, (dm, Di)),
                       ("W_a", W_a, (Di, Di)), ("W_b", W_b, (Di, Di)), ("W_B", W_B, (Di, N)),
                       ("W_C", W_C, (Di, N)), ("W_out", W_out, (Di, dm))):
        _req(t, nm, shp, dt, dev)
    for nm, t, shp in (("conv_w", conv_w, (Di, D_CONV)), ("a_bias", a_bias, (Di,)),
                       ("b_bias", b_bias, (Di,)), ("D", D, (Di,))):
        _req(t, nm, shp, torch.float32, dev)
    _opt(conv_state, "conv_state", (Bt, D_CONV - 1, Di), dt, dev)
    dims = make_dims(Bt, L, Di, N, BF16)
    f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)  # noqa: E731
    g = dict(dxn=f32(Bt, L, dm), dW_u=f32(dm, Di), dW_z=f32(dm, Di), dconv_w=f32(Di, D_CONV),
             dW_a=f32(Di, Di), da_bias=f32(Di), dW_b=f32(Di, Di), db_bias=f32(Di),
             dW_B=f32(Di, N), dW_C=f32(Di, N), dD=f32(Di), dW_out=f32(Di, dm))
    g["dconv_state"] = (torch.empty((Bt, D_CONV - 1, Di), dtype=dt, device=dev)
                        if conv_state is not None else None)
    if ws is None:
        d = torch.device(dev)
        key = (d.index, torch.cuda.current_stream(d).cuda_stream, "mixer_bwd", Bt, L, dm, Di, N)
        ws = _cached_workspace(
            key, lambda: int(lib().naju_mixer_bwd_workspace_bytes(ctypes.byref(dims), dm)), d)
    check(lib().naju_mixer_bwd(ctypes.byref(dims), dm, _p(xn), _p(W_u), _p(W_z), _p(conv_w),
                               _p(conv_state), _p(W_a), _p(a_bias), _p(W_b), _p(b_bias),
                               _p(W_B), _p(W_C), _p(D), _p(W_out), _p(d_out), _p(g["dxn"]),
                               _p(g["dW_u"]), _p(g["dW_z"]), _p(g["dconv_w"]),
                               _p(g["dconv_state"]), _p(g["dW_a"]), _p(g["da_bias"]),
                               _p(g["dW_b"]), _p(g["db_bias"]), _p(g["dW_B"]), _p(g["dW_C"]),
                               _p(g["dD"]), _p(g["dW_out"]),
                               fwd_ws.ptr if fwd_ws is not None else None,
                               fwd_ws.nbytes if fwd_ws is not None else 0, ws.ptr, ws.nbytes,
                               stream_handle(dev)))
    return g


# ------------------------------------------------- around the mixer layer
def _logits_records(R, dev, stream) -> Workspace:
    """naju_logits_process's zero-filled records of R rows.  Calls leave them zero, so one buffer
    per stream serves them all and is replaced by a larger one as rows grow (the allocator hands
    the old one out in stream order).  A call under graph capture has records of its own, with
    their fill in the graph: replays come in any order, and on any stream."""
    if torch.cuda.is_current_stream_capturing():
        return Workspace(lib().naju_logits_workspace_bytes(R), dev)
    key = (dev.index, stream, "logits")
    rows, ws = _ws_cache.get(key, (-1, None))
    if R > rows:
        rows = 1 << max(8, (R - 1).bit_length())
        nbytes = lib().naju_logits_workspace_bytes(rows)
        ws = Workspace(nbytes, dev)
        if nbytes > 0:  # (else the call refuses that many rows)
            _ws_cache[key] = (rows, ws)
    return ws


@_on_its_device
def embed_fwd(ids, W, scale=1.0):
    """out = naju_embed_fwd(ids, W, scale): scale * W[ids], zeros where an id lies outside
    the vocabulary.  ids: int32 of any shape; W [vocab, d_model]; out ids.shape + (d_model,)."""
    V, d = W.shape
    dt, dev = W.dtype, W.device
    io, st = _io_of(W), _stream(dev)
    if not W.is_contiguous():
        raise ValueError("W must be contiguous")
    _req(ids, "ids", ids.shape, torch.int32, dev)
    out = torch.empty(tuple(ids.shape) + (d,), dtype=dt, device=dev)
    check(lib().naju_embed_fwd(ids.numel(), V, d, io, _p(ids), _p(W), float(scale), _p(out),
                               st))
    return out


@_on_its_device
def embed_bwd(ids, dout, vocab, scale=1.0, *, dW=None, ws=None):
    """dW = naju_embed_bwd(ids, dout, vocab, scale), fp32 [vocab, d_model].  With dW given the
    gradient is added to it (rows of tokens that do not occur are not touched).  Without ws
    every call takes scratch of its own from torch's allocator: token counts vary from batch to
    batch, and calls from several host threads must not sort in one another's lists."""
    d = dout.shape[-1]
    dt, dev = dout.dtype, dout.device
    io, st = _io_of(dout), _stream(dev)
    _req(ids, "ids", ids.shape, torch.int32, dev)
    _req(dout, "dout", tuple(ids.shape) + (d,), dt, dev)
    _opt(dW, "dW", (vocab, d), torch.float32, dev)
    accumulate = dW is not None
    if dW is None:
        dW = torch.empty((vocab, d), dtype=torch.float32, device=dev)
    T = ids.numel()
    if ws is None:
        nbytes = lib().naju_embed_bwd_workspace_bytes(T, vocab, d)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        nbytes, scratch = ws.nbytes, ws.tensor
    check(lib().naju_embed_bwd(T, vocab, d, io, _p(ids), _p(dout), float(scale),
                               int(accumulate), _p(dW), _p(scratch), nbytes, st))
    return dW


def _row_stride(t, name, R, V) -> int:
    """The distance of a matrix's contiguous rows."""
    rows, cols = t.stride()
    if (V > 1 and cols != 1) or (R > 1 and rows < V):
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return rows if R > 1 else V


def _req_rows(t, name, shape, dtype, device) -> int:
    """A matrix of contiguous rows, any distance apart; returns that distance."""
    if t is None:
        raise ValueError("%s is required" % name)
    if t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    return _row_stride(t, name, *shape)


def _distill_args(logits, t_ids, t_logits, temperature):
    if logits.dim() != 2 or t_ids.dim() != 2:
        raise ValueError("logits and t_ids must be matrices")
    R, V = logits.shape
    if V == 0:
        raise ValueError("logits: the vocabulary is empty")
    k = t_ids.shape[1]
    dt, dev = logits.dtype, logits.device
    io, st = _io_of(logits), _stream(dev)
    ld = _row_stride(logits, "logits", R, V)
    _req(t_ids, "t_ids", (R, k), torch.int32, dev)
    _req(t_logits, "t_logits", (R, k), torch.float32, dev)
    return R, dev, st, (R, V, k, io, _p(logits), ld, _p(t_ids), _p(t_logits), float(temperature))


def _distill_grad_out(logits, g, dlogits):
    R, V = logits.shape
    _req(g, "g", (R,), torch.float32, logits.device)
    if dlogits is None:
        dlogits = torch.empty((R, V), dtype=logits.dtype, device=logits.device)
    return dlogits, _req_rows(dlogits, "dlogits", (R, V), logits.dtype, logits.device)


@_on_its_device
def distill_fwd(logits, t_ids, t_logits, temperature=1.0):
    """loss, lse = naju_distill_fwd(...), fp32 [rows] each.  logits [rows, vocab] (contiguous
    rows, any row stride); t_ids int32 and t_logits fp32 [rows, k]: the teacher's top logits
    (index -1 or value -inf: no entry)."""
    R, dev, st, args = _distill_args(logits, t_ids, t_logits, temperature)
    loss = torch.empty(R, dtype=torch.float32, device=dev)
    lse = torch.empty(R, dtype=torch.float32, device=dev)
    check(lib().naju_distill_fwd(*args, _p(loss), _p(lse), st))
    return loss, lse


@_on_its_device
def distill_bwd(logits, t_ids, t_logits, lse, g, temperature=1.0, *, dlogits=None):
    """dlogits = naju_distill_bwd(...) for the upstream gradient g [rows] of the loss and the
    lse that distill_fwd returned; dlogits: a tensor to write (contiguous rows, any stride)."""
    R, dev, st, args = _distill_args(logits, t_ids, t_logits, temperature)
    _req(lse, "lse", (R,), torch.float32, dev)
    dlogits, ldd = _distill_grad_out(logits, g, dlogits)
    check(lib().naju_distill_bwd(*args, _p(lse), _p(g), _p(dlogits), ldd, st))
    return dlogits


@_on_its_device
def distill_fwd_bwd(logits, t_ids, t_logits, g, temperature=1.0, *, dlogits=None):
    """loss, dlogits = naju_distill_fwd_bwd(...): both in one pass over the logits, for row
    weights g that are known before the loss."""
    R, dev, st, args = _distill_args(logits, t_ids, t_logits, temperature)
    loss = torch.empty(R, dtype=torch.float32, device=dev)
    lse = torch.empty(R, dtype=torch.float32, device=dev)
    dlogits, ldd = _distill_grad_out(logits, g, dlogits)
    check(lib().naju_distill_fwd_bwd(*args, _p(g), _p(loss), _p(lse), _p(dlogits), ldd,
                                     st))
    return loss, dlogits


@_on_its_device
def logits_process(logits, history=None, lengths=None, repetition=None, presence=None,
                   frequency=None, bias_ids=None, bias=None, mask=None, *, ws=None):
    """out, best = naju_logits_process(...): penalties for the tokens of each row's history
    (int32 [rows, n], the first lengths[row] of it), biases (pairs bias_ids int32, bias fp32
    [rows, n]) and a grammar mask (int32 words [rows, ceil(vocab / 32)], bit set = allowed).
    out: fp32 [rows, vocab]; best: int32 [rows], -1 where nothing is allowed.  repetition,
    presence and frequency are fp32 [rows] or None."""
    if logits.dim() != 2:
        raise ValueError("logits must be a matrix")
    R, V = logits.shape
    if V == 0:
        raise ValueError("logits: the vocabulary is empty")
    dt, dev = logits.dtype, logits.device
    io, st = _io_of(logits), _stream(dev)
    ld = _row_stride(logits, "logits", R, V)
    H = nb = 0
    if history is not None:
        H = history.shape[-1]
        _req(history, "history", (R, H), torch.int32, dev)
    _opt(lengths, "lengths", (R,), torch.int32, dev)
    _opt(repetition, "repetition", (R,), torch.float32, dev)
    _opt(presence, "presence", (R,), torch.float32, dev)
    _opt(frequency, "frequency", (R,), torch.float32, dev)
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias_ids is not None:
        nb = bias_ids.shape[-1]
        _req(bias_ids, "bias_ids", (R, nb), torch.int32, dev)
        _req(bias, "bias", (R, nb), torch.float32, dev)
    _opt(mask, "mask", (R, (V + 31) // 32), torch.int32, dev)
    out = torch.empty((R, V), dtype=torch.float32, device=dev)
    best = torch.empty((R,), dtype=torch.int32, device=dev)
    ws = ws or _logits_records(R, dev, st)
    check(lib().naju_logits_process(R, V, io, _p(logits), ld, _p(history), H, _p(lengths),
                                    _p(repetition), _p(presence), _p(frequency), _p(bias_ids),
                                    _p(bias), nb, _p(mask), _p(out), _p(best), ws.tensor.data_ptr(),
                                    ws.nbytes, st))
    return out, best


@_on_its_device
def w4_quantize(W, group=64, *, zeros=False):
    """qweight, scales, zeros = naju_w4_quantize(W): weights W [d_in, d_out] (fp32 or bf16) as
    4-bit codes with one bf16 scale per `group` inputs of an output.  zeros=False: codes around
    8, and None is returned for the zeros."""
    K, N = W.shape
    dev = W.device
    io, st = _io_of(W), _stream(dev)
    _req(W, "W", (K, N), W.dtype, dev)
    ng = -(-K // group)
    qw = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, ng), dtype=torch.bfloat16, device=dev)
    z = torch.empty((N, ng), dtype=torch.uint8, device=dev) if zeros else None
    check(lib().naju_w4_quantize(K, N, group, io, _p(W), _p(qw), _p(scales), _p(z),
                                 st))
    return qw, scales, z


@_on_its_device
def w4_linear(x, qweight, scales, group, zeros=None, bias=None, res=None):
    """y = naju_w4_linear(x, ...), bf16 [rows, d_out]: x bf16 [rows, d_in], qweight uint8
    [d_out, d_in / 2], scales bf16 and zeros uint8 (None: 8) [d_out, ceil(d_in / group)], bias
    fp32 [d_out] or None, res bf16 [rows, d_out] or None."""
    R, K = x.shape
    N = qweight.shape[0]
    dev = x.device
    st = _stream(dev)
    ng = -(-K // group)
    if K % 2:
        raise ValueError("x: an odd number of inputs (two codes share a byte)")
    _req(x, "x", (R, K), torch.bfloat16, dev)
    _req(qweight, "qweight", (N, K // 2), torch.uint8, dev)
    _req(scales, "scales", (N, ng), torch.bfloat16, dev)
    _opt(zeros, "zeros", (N, ng), torch.uint8, dev)
    _opt(bias, "bias", (N,), torch.float32, dev)
    _opt(res, "res", (R, N), torch.bfloat16, dev)
    y = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
    check(lib().naju_w4_linear(R, K, N, group, _p(x), _p(qweight), _p(scales), _p(zeros),
                               _p(bias), _p(res), _p(y), st))
    return y
