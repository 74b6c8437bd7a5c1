"""ctypes binding of libnaju.so (include/naju.h, include/naju_testing.h).

Argument marshalling only: every function here (those of the vector-state scan,
the 4-bit product and the state cache through the compiled _naju_bind module)
checks tensor placement, dtype and contiguity, allocates outputs with torch on the inputs' device,
passes raw device pointers and the current CUDA stream to the C ABI, and
raises NajuError on a non-OK status.  All arithmetic runs in the library's
CUDA kernels; there is no host or PyTorch fallback.

With `stream` a call runs on that stream instead: what it allocates is that
stream's memory, and every tensor it takes or returns may be dropped at any
time after the call.  As ever, the given stream has to wait for the work that
fills the inputs, and a reader of the results for the given stream.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import inspect
import os
import re
import threading
from typing import Optional

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
HEADERS = [os.path.join(_ROOT, "include", "naju.h"), os.path.join(_ROOT, "include",
                                                                  "naju_testing.h")]

F32, BF16 = 0, 1
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "CUDA error",
           4: "inter-block wait timed out"}


class NajuError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_STATUS.get(status, status)} (status {status})")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("d_inner", ctypes.c_int64), ("d_state", ctypes.c_int64),
                ("conv_width", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib(build_if_missing: bool = True):
    """The loaded library.  Raises if it is not built (never falls back)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                if not build_if_missing:
                    raise RuntimeError(f"Naju CUDA library missing: {path}")
                _build.build()
            L = ctypes.CDLL(path)
            vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
            dp = ctypes.POINTER(Dims)
            L.naju_scan_workspace_bytes.argtypes = [dp]
            L.naju_scan_workspace_bytes.restype = sz
            L.naju_conv_silu_fwd.argtypes = [dp] + [vp] * 5
            L.naju_conv_silu_bwd.argtypes = [dp] + [vp] * 8
            L.naju_scan_fwd.argtypes = [dp] + [vp] * 13 + [sz, vp]
            L.naju_scan_bwd.argtypes = [dp] + [vp] * 23 + [sz, vp]
            L.naju_scan_step.argtypes = [i64, i64, i64, i32] + [vp] * 10
            L.naju_conv_silu_step.argtypes = [i64, i64, i32] + [vp] * 6
            L.naju_scan_step_conv.argtypes = [i64, i64, i64, i32] + [vp] * 13
            L.naju_last_device_status.argtypes = [vp, vp]
            L.naju_status_string.argtypes = [ctypes.c_int]
            L.naju_status_string.restype = ctypes.c_char_p
            L.naju_testing_set_wait_limit.argtypes = [i64]
            L.naju_testing_set_skip_publish.argtypes = [i32]
            L.naju_testing_set_fwd_groups.argtypes = [i32]
            L.naju_testing_fwd_groups.argtypes = [vp]
            L.naju_testing_fwd_groups.restype = i32
            L.naju_testing_set_bwd_groups.argtypes = [i32]
            L.naju_testing_set_fwd_impl.argtypes = [i32]
            L.naju_testing_fwd_impl.argtypes = [vp]
            L.naju_testing_fwd_impl.restype = i32
            L.naju_testing_set_bwd_impl.argtypes = [i32]
            L.naju_testing_bwd_impl.argtypes = [vp]
            L.naju_testing_bwd_impl.restype = i32
            L.naju_testing_bwd_groups.argtypes = [vp]
            L.naju_testing_bwd_groups.restype = i32
            L.naju_testing_set_bwd_pieces.argtypes = [i32]
            L.naju_testing_set_fwd_pieces.argtypes = [i32]
            L.naju_testing_fwd_pieces.argtypes = [vp]
            L.naju_testing_fwd_pieces.restype = i32
            L.naju_testing_bwd_pieces.argtypes = [vp]
            L.naju_testing_bwd_pieces.restype = i32
            L.naju_testing_set_vscan_cluster.argtypes = [i32]
            L.naju_testing_set_w4_impl.argtypes = [i32]
            L.naju_vscan_workspace_bytes.argtypes = [dp]
            L.naju_vscan_workspace_bytes.restype = sz
            L.naju_vscan_fwd.argtypes = [dp] + [vp] * 8 + [sz, vp]
            L.naju_vscan_bwd.argtypes = [dp] + [vp] * 12 + [sz, vp]
            L.naju_vscan_step.argtypes = [i64, i64, i32] + [vp] * 7
            L.naju_state_store.argtypes = [i64] * 4 + [vp] * 5
            L.naju_state_load.argtypes = [i64] * 4 + [vp] * 5
            L.naju_w4_quantize.argtypes = [i64] * 2 + [i32] * 2 + [vp] * 4
            L.naju_w4_linear.argtypes = [i64] * 3 + [i32] * 2 + [vp] * 7
            for name in ("naju_w4_quantize", "naju_w4_linear", "naju_state_store",
                         "naju_state_load", "naju_vscan_fwd", "naju_vscan_bwd",
                         "naju_vscan_step", "naju_conv_silu_fwd", "naju_conv_silu_bwd",
                         "naju_scan_fwd", "naju_scan_bwd", "naju_scan_step",
                         "naju_conv_silu_step", "naju_scan_step_conv",
                         "naju_last_device_status"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


_bind = None


def _load_bind():
    """The compiled marshalling module, bound to the loaded library.  Raises if
    it cannot be had (there is no other path for its functions)."""
    global _bind
    L = lib()
    with _lock:
        if _bind is None:
            path = _build.bind_path()
            if not os.path.exists(path):
                path = _build.build_bind()
            loader = importlib.machinery.ExtensionFileLoader("_naju_bind", path)
            spec = importlib.util.spec_from_file_location("_naju_bind", path, loader=loader)
            mod = importlib.util.module_from_spec(spec)
            loader.exec_module(mod)
            addr = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
            mod.bind(NajuError, addr(L.naju_vscan_workspace_bytes), addr(L.naju_vscan_fwd),
                     addr(L.naju_vscan_bwd), addr(L.naju_vscan_step), addr(L.naju_w4_linear),
                     addr(L.naju_state_store), addr(L.naju_state_load))
            _bind = mod
    return _bind


def declared_symbols() -> list[str]:
    """Function names declared in the public headers."""
    names = []
    for h in HEADERS:
        txt = open(h).read()
        txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
        names += re.findall(r"\b(naju_\w+)\s*\(", txt)
    return sorted(set(names))


# --------------------------------------------------------------- helpers
def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _torch_dt(code: int):
    return torch.float32 if code == F32 else torch.bfloat16


def _ptr(t: Optional[torch.Tensor], name: str = "", dtype=None, device=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(st: int, where: str):
    if st != 0:
        raise NajuError(st, where)


def make_dims(batch, seqlen, d_inner, d_state, dtype: int, out_dtype: Optional[int] = None,
              conv_width: int = 4) -> Dims:
    return Dims(batch, seqlen, d_inner, d_state, conv_width, dtype,
                dtype if out_dtype is None else out_dtype, 0)


def workspace_bytes(dims: Dims) -> int:
    return int(lib().naju_scan_workspace_bytes(ctypes.byref(dims)))


def alloc_workspace(dims: Dims, device) -> torch.Tensor:
    n = workspace_bytes(dims)
    if n == 0:
        raise NajuError(1, "naju_scan_workspace_bytes")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    ws.zero_()
    return ws


def _on_given_stream(fn):
    """fn with its `stream` argument, where one is given, as the current stream
    meanwhile, so that what fn allocates belongs to it; the allocator holds
    tensors that one stream owns and the other works on."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        flat = [] if stream is None else _tensors((args, kw))
        if not flat:
            return fn(*args, **kw)
        dev = flat[0].device
        caller = torch.cuda.current_stream(dev)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
        if stream.cuda_stream == caller.cuda_stream:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        for t in flat:
            t.record_stream(stream)
        for t in _tensors(out):
            t.record_stream(caller)
        return out

    return call


def _tensors(v) -> list:
    """The CUDA tensors in nested tuples and dicts."""
    if isinstance(v, torch.Tensor):
        return [v] if v.is_cuda else []
    if isinstance(v, dict):
        v = v.values()
    elif not isinstance(v, (tuple, list)):
        return []
    return [t for x in v for t in _tensors(x)]


# ------------------------------------------------------------- entry points
@_on_given_stream
def conv_silu_fwd(u, conv_w, conv_b=None, out_dtype=None, stream=None):
    Bt, L, d = u.shape
    dims = make_dims(Bt, L, d, 16, _dt(u), out_dtype, conv_w.shape[1])
    h = torch.empty(u.shape, dtype=_torch_dt(dims.out_dtype), device=u.device)
    _check(lib().naju_conv_silu_fwd(ctypes.byref(dims), _ptr(u, "u"),
                                    _ptr(conv_w, "conv_w", torch.float32),
                                    _ptr(conv_b, "conv_b", torch.float32), _ptr(h), _stream(stream)),
           "naju_conv_silu_fwd")
    return h


@_on_given_stream
def conv_silu_bwd(u, conv_w, conv_b, dh, stream=None):
    Bt, L, d = u.shape
    dims = make_dims(Bt, L, d, 16, _dt(u), None, conv_w.shape[1])
    du = torch.empty_like(u)
    dw = torch.empty_like(conv_w)
    db = torch.empty(d, dtype=torch.float32, device=u.device)
    _check(lib().naju_conv_silu_bwd(ctypes.byref(dims), _ptr(u, "u"),
                                    _ptr(conv_w, "conv_w", torch.float32),
                                    _ptr(conv_b, "conv_b", torch.float32),
                                    _ptr(dh, "dh", u.dtype), _ptr(du), _ptr(dw), _ptr(db),
                                    _stream(stream)), "naju_conv_silu_bwd")
    return du, dw, db


@_on_given_stream
def scan_fwd(hu, a, b, B, C, *, conv_w=None, conv_b=None, z=None, D=None, x0=None,
             out_dtype=None, workspace=None, want_final=True, y=None, x_final=None,
             stream=None):
    """Returns (y, x_final, workspace).  `hu` is u when conv_w is given."""
    Bt, L, d = hu.shape
    N = B.shape[-1]
    dt = _dt(hu)
    dims = make_dims(Bt, L, d, N, dt, out_dtype)
    dev = hu.device
    for name, t in (("a", a), ("b", b), ("B", B), ("C", C), ("z", z)):
        if t is not None and t.dtype != hu.dtype:
            raise TypeError(f"{name} must have the activation dtype {hu.dtype}")
    if workspace is None:
        workspace = alloc_workspace(dims, dev)
    if y is None:
        y = torch.empty((Bt, L, d), dtype=_torch_dt(dims.out_dtype), device=dev)
    if x_final is None and want_final:
        x_final = torch.empty((Bt, d, N), dtype=torch.float32, device=dev)
    _check(lib().naju_scan_fwd(
        ctypes.byref(dims), _ptr(hu, "hu"), _ptr(conv_w, "conv_w", torch.float32),
        _ptr(conv_b, "conv_b", torch.float32), _ptr(a, "a"), _ptr(b, "b"), _ptr(B, "B"),
        _ptr(C, "C"), _ptr(z, "z"), _ptr(D, "D", torch.float32), _ptr(x0, "x0", torch.float32),
        _ptr(y, "y"), _ptr(x_final, "x_final", torch.float32), _ptr(workspace, "workspace"),
        ctypes.c_size_t(workspace.numel()), _stream(stream)), "naju_scan_fwd")
    return y, x_final, workspace


@_on_given_stream
def scan_bwd(dy, hu, a, b, B, C, workspace, *, conv_w=None, conv_b=None, z=None, D=None,
             x0=None, dx_final=None, out_dtype=None, want_dx0=True, grads=None, stream=None):
    """Gradients of scan_fwd; `workspace` must hold that forward's checkpoints.
    Returns a dict: dhu, da, db, dB, dC, dz, dD, dconv_w, dconv_b, dx0."""
    Bt, L, d = hu.shape
    N = B.shape[-1]
    dims = make_dims(Bt, L, d, N, _dt(hu), out_dtype)
    dev = hu.device
    if grads is None:
        ot = _torch_dt(dims.out_dtype)
        grads = {
            "dhu": torch.empty((Bt, L, d), dtype=ot, device=dev),
            "da": torch.empty((Bt, L, d), dtype=ot, device=dev),
            "db": torch.empty((Bt, L, d), dtype=ot, device=dev) if b is not None else None,
            "dB": torch.empty((Bt, L, N), dtype=ot, device=dev),
            "dC": torch.empty((Bt, L, N), dtype=ot, device=dev),
            "dz": torch.empty((Bt, L, d), dtype=ot, device=dev) if z is not None else None,
            "dD": torch.empty(d, dtype=torch.float32, device=dev) if D is not None else None,
            "dconv_w": torch.empty_like(conv_w) if conv_w is not None else None,
            "dconv_b": torch.empty(d, dtype=torch.float32, device=dev)
            if conv_w is not None else None,
            "dx0": torch.empty((Bt, d, N), dtype=torch.float32, device=dev) if want_dx0 else None,
        }
    g = grads
    _check(lib().naju_scan_bwd(
        ctypes.byref(dims), _ptr(hu, "hu"), _ptr(conv_w, "conv_w", torch.float32),
        _ptr(conv_b, "conv_b", torch.float32), _ptr(a, "a"), _ptr(b, "b"), _ptr(B, "B"),
        _ptr(C, "C"), _ptr(z, "z"), _ptr(D, "D", torch.float32), _ptr(x0, "x0", torch.float32),
        _ptr(dy, "dy", hu.dtype), _ptr(dx_final, "dx_final", torch.float32), _ptr(g["dhu"]),
        _ptr(g["da"]), _ptr(g["db"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dz"]),
        _ptr(g["dD"]), _ptr(g["dconv_w"]), _ptr(g["dconv_b"]), _ptr(g["dx0"]),
        _ptr(workspace, "workspace"), ctypes.c_size_t(workspace.numel()), _stream(stream)),
        "naju_scan_bwd")
    return g


@_on_given_stream
def scan_step(state, h, a, b, B, C, z=None, D=None, y=None, stream=None):
    """One decode step; `state` [Bt, d, N] fp32 is updated in place.  Returns y."""
    Bt, d = h.shape
    N = B.shape[-1]
    if y is None:
        y = torch.empty_like(h)
    _check(lib().naju_scan_step(Bt, d, N, _dt(h), _ptr(h, "h"), _ptr(a, "a"), _ptr(b, "b"),
                                _ptr(B, "B"), _ptr(C, "C"), _ptr(z, "z"),
                                _ptr(D, "D", torch.float32), _ptr(state, "state", torch.float32),
                                _ptr(y, "y"), _stream(stream)), "naju_scan_step")
    return y


@_on_given_stream
def conv_silu_step(conv_state, u, conv_w, conv_b=None, h=None, stream=None):
    """Decode step of conv + SiLU; `conv_state` [Bt, d, 3] fp32 is updated in
    place (previous three inputs, oldest first).  Returns h."""
    Bt, d = u.shape
    if h is None:
        h = torch.empty_like(u)
    _check(lib().naju_conv_silu_step(Bt, d, _dt(u), _ptr(u, "u"),
                                     _ptr(conv_w, "conv_w", torch.float32),
                                     _ptr(conv_b, "conv_b", torch.float32),
                                     _ptr(conv_state, "conv_state", torch.float32),
                                     _ptr(h, "h"), _stream(stream)), "naju_conv_silu_step")
    return h


@_on_given_stream
def scan_step_conv(state, conv_state, u, a, b, B, C, conv_w, conv_b=None, z=None, D=None,
                   y=None, stream=None):
    """One decode step from the pre-conv input u (conv + SiLU fused); `state`
    and `conv_state` are updated in place.  Returns y."""
    Bt, d = u.shape
    N = B.shape[-1]
    if y is None:
        y = torch.empty_like(u)
    _check(lib().naju_scan_step_conv(Bt, d, N, _dt(u), _ptr(u, "u"),
                                     _ptr(conv_w, "conv_w", torch.float32),
                                     _ptr(conv_b, "conv_b", torch.float32),
                                     _ptr(conv_state, "conv_state", torch.float32),
                                     _ptr(a, "a"), _ptr(b, "b"), _ptr(B, "B"), _ptr(C, "C"),
                                     _ptr(z, "z"), _ptr(D, "D", torch.float32),
                                     _ptr(state, "state", torch.float32), _ptr(y, "y"),
                                     _stream(stream)), "naju_scan_step_conv")
    return y


# ------------------------------------------------------- vector-state scan
def vscan_workspace(dims: Dims, like: torch.Tensor) -> torch.Tensor:
    """A workspace of vscan_fwd and vscan_bwd on the device of `like`
    (contents undefined); dims as make_dims(batch, seqlen, d_inner, 1, ...)."""
    n = lib().naju_vscan_workspace_bytes(ctypes.byref(dims))
    if n == 0:
        raise NajuError(1, "naju_vscan_workspace_bytes")
    ws = like.new_empty(n + 256, dtype=torch.uint8)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def vscan_fwd(h, a, b=None, *, z=None, x0=None, out_dtype=None, workspace=None, want_final=True,
              y=None, x_final=None, stream=None):
    """Vector-state scan over [batch, seqlen, d_inner]: x_t = f x_{t-1} + i h,
    y = x SiLU(z).  b None: coupled gate; z None: no modulation.  Returns
    (y, x_final, workspace); the workspace is what vscan_bwd needs."""
    return (_bind or _load_bind()).vscan_fwd(h, a, b, z, x0, out_dtype, workspace, want_final, y,
                                             x_final, stream)


def vscan_bwd(dy, h, a, b, workspace, *, z=None, dx_final=None, out_dtype=None, want_dx0=True,
              grads=None, stream=None):
    """Gradients of vscan_fwd; `workspace` must hold that forward's
    checkpoints.  Returns a dict: dh, da, db (None without b), dz (None
    without z), dx0 (None unless wanted)."""
    return (_bind or _load_bind()).vscan_bwd(dy, h, a, b, workspace, z, dx_final, out_dtype,
                                             want_dx0, grads, stream)


def vscan_step(state, h, a, b=None, z=None, y=None, stream=None):
    """One decode step of the vector-state scan: h, a, b, z [batch, d_inner];
    `state` [batch, d_inner] fp32 is updated in place.  Returns y."""
    return (_bind or _load_bind()).vscan_step(state, h, a, b, z, y, stream)


# ------------------------------------------------------ 4-bit projections
@_on_given_stream
def w4_quantize(W, group=128, stream=None):
    """Quantises a projection W [n_out, n_in] to 4 bits a weight with one bf16
    scale per `group` (32, 64 or 128) inputs.  Returns (wq, scales): uint8
    [n_out, ceil(n_in / 128) * 64] in w4_linear's packed order, and bf16
    [n_out, ceil(n_in / group)]."""
    if W.dim() != 2:
        raise ValueError(f"W must be [n_out, n_in], got {tuple(W.shape)}")
    if group not in (32, 64, 128):
        raise NajuError(2, f"4-bit projection with groups of {group}")
    O, K = W.shape
    args = (O, K, group, _dt(W), _ptr(W, "W"))
    with torch.cuda.device(W.device):
        wq = torch.empty((O, -(-K // 128) * 64), dtype=torch.uint8, device=W.device)
        scales = torch.empty((O, -(-K // group)), dtype=torch.bfloat16, device=W.device)
        _check(lib().naju_w4_quantize(*args, _ptr(wq, "wq"), _ptr(scales, "scales"),
                                      _stream(stream)), "naju_w4_quantize")
    return wq, scales


def w4_linear(x, wq, scales, group=128, bias=None, residual=None, y=None, stream=None):
    """y = x W^T (+ bias) (+ residual) with the 4-bit W of w4_quantize:
    x [..., n_in] (its leading dimensions are rows), bias [n_out] fp32, residual
    and y [..., n_out] in x's dtype."""
    return (_bind or _load_bind()).w4_linear(x, wq, scales, group, bias, residual, y, stream)


# -------------------------------------------------------- 8-bit state cache
def state_pool(n_slots: int, d_inner: int, d_state: int, device):
    """An empty pool for parked decode states: (pool_q int8, pool_scale fp32);
    every slot reads back as a zero state."""
    return (torch.zeros((n_slots, d_inner, d_state), dtype=torch.int8, device=device),
            torch.zeros((n_slots, d_inner), dtype=torch.float32, device=device))


def state_store(state, slots, pool_q, pool_scale, stream=None):
    """Parks decode states: batch place i of `state` [n, d_inner, d_state] fp32
    into slot slots[i] (int32) of the pool, 8 bits a value with one scale per
    row.  Slots outside the pool store nothing; of places that name the same
    slot the last is stored."""
    (_bind or _load_bind()).state_store(state, slots, pool_q, pool_scale, stream)


def state_load(pool_q, pool_scale, slots, state=None, stream=None):
    """Resumes parked states: slot slots[i] into batch place i.  Slots outside
    the pool give a zero state.  Returns state [n, d_inner, d_state] fp32."""
    return (_bind or _load_bind()).state_load(pool_q, pool_scale, slots, state, stream)


def last_device_status(workspace, stream=None) -> int:
    return int(lib().naju_last_device_status(_ptr(workspace, "workspace"), _stream(stream)))


def testing_set_wait_limit(polls: int):
    lib().naju_testing_set_wait_limit(int(polls))


def testing_set_skip_publish(skip: bool):
    lib().naju_testing_set_skip_publish(1 if skip else 0)


def testing_set_fwd_groups(groups: int):
    lib().naju_testing_set_fwd_groups(int(groups))


def testing_fwd_groups(dims: Dims) -> int:
    return int(lib().naju_testing_fwd_groups(ctypes.byref(dims)))


def testing_set_fwd_impl(impl: int):
    lib().naju_testing_set_fwd_impl(int(impl))


def testing_fwd_impl(dims: Dims) -> int:
    return int(lib().naju_testing_fwd_impl(ctypes.byref(dims)))


def testing_set_bwd_impl(impl: int):
    lib().naju_testing_set_bwd_impl(int(impl))


def testing_bwd_impl(dims: Dims) -> int:
    return int(lib().naju_testing_bwd_impl(ctypes.byref(dims)))


def testing_set_bwd_groups(groups: int):
    lib().naju_testing_set_bwd_groups(int(groups))


def testing_bwd_groups(dims: Dims) -> int:
    return int(lib().naju_testing_bwd_groups(ctypes.byref(dims)))


def testing_set_bwd_pieces(pieces: int):
    lib().naju_testing_set_bwd_pieces(int(pieces))


def testing_bwd_pieces(dims: Dims) -> int:
    return int(lib().naju_testing_bwd_pieces(ctypes.byref(dims)))


def testing_set_fwd_pieces(pieces: int):
    lib().naju_testing_set_fwd_pieces(int(pieces))


def testing_fwd_pieces(dims: Dims) -> int:
    return int(lib().naju_testing_fwd_pieces(ctypes.byref(dims)))


def testing_set_vscan_cluster(blocks: int):
    lib().naju_testing_set_vscan_cluster(int(blocks))


def testing_set_w4_impl(impl: int):
    lib().naju_testing_set_w4_impl(int(impl))


def testing_set_sm_count(sms: int):
    lib().naju_testing_set_sm_count(int(sms))


def testing_sm_count() -> int:
    return int(lib().naju_testing_sm_count())
