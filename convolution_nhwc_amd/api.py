"""Thin ctypes binding of libcnhwc.so (C ABI in include/cnhwc.h).

The cnhwc_* functions mirror the C entry points one to one (argument
marshalling only: every step of the computation runs in the HIP library).
``fwd`` / ``dgrad`` / ``wgrad`` are conveniences over PyTorch device tensors: torch only
allocates the outputs and workspace and supplies the current stream.

A problem is a dict with keys n, h, w, c, k, r, s, stride, pad_h, pad_w,
groups and dtype ("f16" or "bf16").  Any non-zero status raises CnhwcError
with the library's reason text.  Loading fails loudly if the library has not
been built: there is no fallback.
"""
import contextlib
import ctypes
import functools
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcnhwc.so")

OK, INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, MISALIGNED, HIP_ERROR = range(6)
F16, BF16, F32, I8 = 0, 1, 2, 3
ACTS = {"silu": 0, "gelu": 1, "relu": 2, "sigmoid": 3}   # CNHWC_ACT_*
ACTS_OR_NONE = dict(ACTS, none=-1)
OP_FWD, OP_DGRAD, OP_WGRAD = 1, 2, 4
(VAR_AUTO, VAR_DGRAD_POINTWISE, VAR_DGRAD_IGEMM, VAR_DGRAD_DW_STREAM, VAR_DGRAD_DW_ROTATED,
 VAR_FWD_DIRECT, VAR_FWD_SPLITC, VAR_FWD_GROUPED, VAR_FWD_GENERIC, VAR_DGRAD_GENERIC,
 VAR_DGRAD_DW_TILED, VAR_FWD_DW_TILED, VAR_FWD_DW_ROTATED, VAR_DGRAD_GROUPED,
 VAR_WGRAD_GENERIC, VAR_WGRAD_POINTWISE, VAR_WGRAD_SPLITK, VAR_DGRAD_SPLITK, VAR_FWD_IGEMM) = range(19)

SYMBOLS = ("cnhwc_out_dims", "cnhwc_workspace_size", "cnhwc_plan", "cnhwc_chunk_plan",
           "cnhwc_fwd", "cnhwc_dgrad", "cnhwc_wgrad", "cnhwc_last_error", "cnhwc_set_override",
           "cnhwc_fwd_static_ws",
           "cnhwc_layernorm_fwd", "cnhwc_layernorm_bwd", "cnhwc_layernorm_workspace_size",
           "cnhwc_gated_fwd", "cnhwc_gated_bwd", "cnhwc_gated_workspace_size", "cnhwc_gated_plan",
           "cnhwc_dropout",
           "cnhwc_groupnorm_workspace_size", "cnhwc_groupnorm_fwd", "cnhwc_groupnorm_bwd",
           "cnhwc_adamw", "cnhwc_adamw_moments",
           "cnhwc_quantize_rows", "cnhwc_linear_i8", "cnhwc_linear_i8_workspace_size", "cnhwc_linear_i8_plan")
STATIC_WS_BYTES = 32 << 20   # CNHWC_STATIC_WS_BYTES


class CnhwcError(RuntimeError):
    def __init__(self, status, reason):
        super().__init__("cnhwc status %d: %s" % (status, reason))
        self.status = status
        self.reason = reason


class Problem(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("h", ctypes.c_int64), ("w", ctypes.c_int64),
                ("c", ctypes.c_int64), ("k", ctypes.c_int64), ("r", ctypes.c_int64),
                ("s", ctypes.c_int64), ("stride", ctypes.c_int32), ("pad_h", ctypes.c_int32),
                ("pad_w", ctypes.c_int32), ("groups", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Override(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("cpl", ctypes.c_int32), ("split_c", ctypes.c_int32),
                ("tune", ctypes.c_int32), ("chunk_limit_bytes", ctypes.c_int64)]


class LayernormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("eps", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GatedProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("f", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("act", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class DropoutProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("p", ctypes.c_double),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class GroupnormProblem(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("pixels", ctypes.c_int64), ("c", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("eps", ctypes.c_float),
                ("groups", ctypes.c_int32), ("act", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("weight_decay", ctypes.c_double), ("p_dtype", ctypes.c_int32),
                ("g_dtype", ctypes.c_int32), ("copy_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AdamwProblem(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("state_bits", ctypes.c_int32), ("count", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


class QuantizeProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class LinearI8Problem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("f", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("w_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("act", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        # One HIP runtime per process: when PyTorch is present its bundled
        # libamdhip64.so.7 must be the one our library binds to, so load torch
        # first (the dynamic loader then reuses the already-loaded soname).
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libcnhwc.so is not built (%s); run "
                               "`python -m convolution_nhwc_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(Problem)
        i64p = ctypes.POINTER(ctypes.c_int64)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        L.cnhwc_out_dims.argtypes = [P, i64p, i64p]
        L.cnhwc_workspace_size.argtypes = [P, ctypes.c_int, ctypes.POINTER(sz)]
        L.cnhwc_plan.argtypes = [P, ctypes.c_int, ctypes.c_char_p, sz, ctypes.POINTER(ctypes.c_int32)]
        L.cnhwc_chunk_plan.argtypes = [P, ctypes.c_int, i64p, ctypes.c_int64, i64p]
        L.cnhwc_fwd.argtypes = [P, vp, vp, vp, vp, sz, vp]
        L.cnhwc_dgrad.argtypes = [P, vp, vp, vp, vp, sz, vp]
        L.cnhwc_wgrad.argtypes = [P, vp, vp, vp, vp, sz, vp]
        L.cnhwc_fwd_static_ws.argtypes = [P, vp, vp, vp, vp]
        L.cnhwc_last_error.argtypes = []
        L.cnhwc_last_error.restype = ctypes.c_char_p
        L.cnhwc_set_override.argtypes = [ctypes.POINTER(Override)]
        LN, GP, DP = (ctypes.POINTER(t) for t in (LayernormProblem, GatedProblem, DropoutProblem))
        szp = ctypes.POINTER(sz)
        L.cnhwc_layernorm_fwd.argtypes = [LN, vp, vp, vp, vp, vp, vp, vp]
        L.cnhwc_layernorm_workspace_size.argtypes = [LN, szp]
        L.cnhwc_layernorm_bwd.argtypes = [LN, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cnhwc_gated_workspace_size.argtypes = [GP, ctypes.c_int, ctypes.c_int, szp]
        L.cnhwc_gated_plan.argtypes = [GP, ctypes.c_int, ctypes.c_char_p, sz]
        L.cnhwc_gated_fwd.argtypes = [GP, vp, vp, vp, vp, vp, sz, vp]
        L.cnhwc_gated_bwd.argtypes = [GP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cnhwc_dropout.argtypes = [DP, vp, vp, vp, vp, vp]
        GN = ctypes.POINTER(GroupnormProblem)
        L.cnhwc_groupnorm_workspace_size.argtypes = [GN, ctypes.c_int, szp]
        L.cnhwc_groupnorm_fwd.argtypes = [GN, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cnhwc_groupnorm_bwd.argtypes = [GN, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cnhwc_adamw.argtypes = [ctypes.POINTER(AdamwProblem), ctypes.POINTER(AdamwTensor), vp, vp, vp, vp]
        L.cnhwc_adamw_moments.argtypes = [ctypes.c_int64, vp, vp, vp, vp, vp, vp, vp]
        QP, LP = ctypes.POINTER(QuantizeProblem), ctypes.POINTER(LinearI8Problem)
        L.cnhwc_quantize_rows.argtypes = [QP, vp, vp, vp, vp]
        L.cnhwc_linear_i8_workspace_size.argtypes = [LP, ctypes.c_int, szp]
        L.cnhwc_linear_i8_plan.argtypes = [LP, ctypes.c_char_p, sz]
        L.cnhwc_linear_i8.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        for fn in SYMBOLS:
            if fn != "cnhwc_last_error":
                getattr(L, fn).restype = ctypes.c_int
        _lib = L
    return _lib


def _problem(p):
    if isinstance(p, Problem):
        return p
    dt = p.get("dtype", "f16")
    dt = {"f16": F16, "bf16": BF16, F16: F16, BF16: BF16}.get(dt, dt)
    return Problem(int(p["n"]), int(p["h"]), int(p["w"]), int(p["c"]), int(p["k"]), int(p["r"]),
                   int(p["s"]), int(p.get("stride", 1)), int(p.get("pad_h", 0)),
                   int(p.get("pad_w", 0)), int(p.get("groups", 1)), int(dt), 0)


def last_error():
    return lib().cnhwc_last_error().decode()


def _check(status):
    if status != OK:
        raise CnhwcError(status, last_error())


def cnhwc_out_dims(p):
    ho, wo = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().cnhwc_out_dims(ctypes.byref(_problem(p)), ctypes.byref(ho), ctypes.byref(wo)))
    return ho.value, wo.value


def cnhwc_workspace_size(p, op):
    b = ctypes.c_size_t()
    _check(lib().cnhwc_workspace_size(ctypes.byref(_problem(p)), op, ctypes.byref(b)))
    return b.value


def cnhwc_plan(p, op):
    buf = ctypes.create_string_buffer(256)
    v = ctypes.c_int32()
    _check(lib().cnhwc_plan(ctypes.byref(_problem(p)), op, buf, 256, ctypes.byref(v)))
    return buf.value.decode(), v.value


def cnhwc_chunk_plan(p, op, cap=4096):
    arr = (ctypes.c_int64 * cap)()
    n = ctypes.c_int64()
    _check(lib().cnhwc_chunk_plan(ctypes.byref(_problem(p)), op, arr, cap, ctypes.byref(n)))
    return [arr[i] for i in range(min(n.value, cap))]


def cnhwc_fwd(p, x, w, y, ws, ws_bytes, stream):
    """Raw entry point: pointers as ints (device addresses), stream as int."""
    _check(lib().cnhwc_fwd(ctypes.byref(_problem(p)), x, w, y, ws, ws_bytes, stream))


def cnhwc_fwd_static_ws(p, x, w, y, stream):
    """Forward pass with the library's static device workspace (no allocation)."""
    _check(lib().cnhwc_fwd_static_ws(ctypes.byref(_problem(p)), x, w, y, stream))


def cnhwc_dgrad(p, dy, w, dx, ws, ws_bytes, stream):
    _check(lib().cnhwc_dgrad(ctypes.byref(_problem(p)), dy, w, dx, ws, ws_bytes, stream))


def cnhwc_wgrad(p, x, dy, dw, ws, ws_bytes, stream):
    _check(lib().cnhwc_wgrad(ctypes.byref(_problem(p)), x, dy, dw, ws, ws_bytes, stream))


class _Forced(threading.local):
    key = None   # what of this thread's override decides the gated product's sizes


_forced = _Forced()


def cnhwc_set_override(variant=0, cpl=0, split_c=0, chunk_limit_bytes=0, tune=0):
    _check(lib().cnhwc_set_override(ctypes.byref(Override(variant, cpl, split_c, tune,
                                                          chunk_limit_bytes))))
    _forced.key = (split_c, tune)


def cnhwc_clear_override():
    _check(lib().cnhwc_set_override(None))
    _forced.key = None


@contextlib.contextmanager
def override(**kw):
    """Test-only: force dispatcher choices inside a with-block."""
    cnhwc_set_override(**kw)
    try:
        yield
    finally:
        cnhwc_clear_override()


# ---- PyTorch conveniences ----------------------------------------------------

def _stream_handle(torch, device):
    return torch.cuda.current_stream(device).cuda_stream


def _storage_dtype(torch, p):
    return torch.bfloat16 if p.get("dtype", "f16") in ("bf16", BF16) else torch.float16


def fwd(x, w, p, y=None, ws=None):
    """y = forward conv of device tensors x [N,H,W,C] and w [K,R,S,C/G] (16-bit)."""
    import torch
    ho, wo = cnhwc_out_dims(p)
    if y is None:
        y = torch.empty((p["n"], ho, wo, p["k"]), dtype=_storage_dtype(torch, p), device=x.device)
    need = cnhwc_workspace_size(p, OP_FWD)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    cnhwc_fwd(p, x.data_ptr(), w.data_ptr(), y.data_ptr(), ws.data_ptr() if ws is not None else None,
              ws.numel() * ws.element_size() if ws is not None else 0, _stream_handle(torch, x.device))
    return y


def dgrad(dy, w, p, dx=None, ws=None):
    """dx = backward-data conv of device tensors dy [N,Ho,Wo,K] and w [K,R,S,C/G]."""
    import torch
    if dx is None:
        dx = torch.empty((p["n"], p["h"], p["w"], p["c"]), dtype=_storage_dtype(torch, p),
                         device=dy.device)
    need = cnhwc_workspace_size(p, OP_DGRAD)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=dy.device)
    cnhwc_dgrad(p, dy.data_ptr(), w.data_ptr(), dx.data_ptr(),
                ws.data_ptr() if ws is not None else None,
                ws.numel() * ws.element_size() if ws is not None else 0,
                _stream_handle(torch, dy.device))
    return dx


def wgrad(x, dy, p, dw=None, ws=None):
    """dw = weight gradient of device tensors x [N,H,W,C] and dy [N,Ho,Wo,K]."""
    import torch
    if dw is None:
        dw = torch.empty((p["k"], p["r"], p["s"], p["c"] // p.get("groups", 1)),
                         dtype=_storage_dtype(torch, p), device=x.device)
    need = cnhwc_workspace_size(p, OP_WGRAD)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    cnhwc_wgrad(p, x.data_ptr(), dy.data_ptr(), dw.data_ptr(),
                ws.data_ptr() if ws is not None else None,
                ws.numel() * ws.element_size() if ws is not None else 0,
                _stream_handle(torch, x.device))
    return dw


# ---- channel mixing: layer norm, gated feed-forward, dropout -------------------
#
# x is a device tensor [..., c] whose last dimension is contiguous and whose
# leading dimensions step evenly (a dense tensor or a channel slice of one), so
# that it is rows of c channels with one row stride.  Outputs are new dense
# tensors of x's leading shape unless given.  Work goes to the current stream of
# x's device; a tensor written on another stream has to be waited for first, as
# in PyTorch.

_torch = None
_mix_types = {}


def _t():
    """PyTorch, imported on first use, and the element types by torch dtype."""
    global _torch
    if _torch is None:
        import torch
        _mix_types.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
        _torch = torch
    return _torch


def _rows(t, what, width=None):
    """(rows, width, row stride) of a tensor seen as rows of its last dimension."""
    shape = t.shape
    if not shape:
        raise ValueError("%s needs at least one dimension" % what)
    c = shape[-1]
    if width is not None and c != width:
        raise ValueError("%s has %d channels, expected %d" % (what, c, width))
    n = t.numel()
    if n and t.is_contiguous():
        return n // c, c, c
    rows = 1
    for s in shape[:-1]:
        rows *= s
    if not n:
        return rows, c, c
    if t.stride(-1) != 1 and c > 1:
        raise ValueError("%s: channels are not contiguous" % what)
    stride, inner = None, 1      # walk outwards; dimensions of size 1 have no step
    for size, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * inner:
            raise ValueError("%s: its leading dimensions do not step evenly (shape %s, strides %s)"
                             % (what, tuple(shape), tuple(t.stride())))
        inner *= size
    if stride is None:
        stride = c
    if stride < c:
        raise ValueError("%s: rows overlap (stride %d, %d channels)" % (what, stride, c))
    return rows, c, stride


def _same(t, ref, what, dtype=None):
    if t.device != ref.device:
        raise ValueError("%s is on %s, expected %s" % (what, t.device, ref.device))
    if t.dtype != (dtype or ref.dtype):
        raise ValueError("%s is %s, expected %s" % (what, t.dtype, dtype or ref.dtype))


def _operand(t, what, f32=True):
    """Element type of a GPU tensor."""
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor (got %s)" % (what, t.device))
    dt = _mix_types.get(t.dtype, -1)
    if dt < 0 or (dt == F32 and not f32):
        raise ValueError("%s must be float16, bfloat16%s (got %s)" % (what, " or float32" if f32 else "", t.dtype))
    return dt


def _out(t, what, rows, width, ref, stride, shape=None):
    """(output, its row stride): the caller's, or a new dense one of ref's shape
    (ref has the given row stride) or of another."""
    if t is None:
        # (like a dense ref: that takes 0.9 us, a shape 1.5)
        return _torch.empty_like(ref) if stride == width and shape is None else ref.new_empty(shape or ref.shape), width
    _same(t, ref, what)
    r, _, st = _rows(t, what, width)
    if r != rows:
        raise ValueError("%s has %d rows, expected %d" % (what, r, rows))
    return t, st


def _vector(t, n, what, ref):
    """Element type of a per-channel vector."""
    if t.device != ref.device:
        raise ValueError("%s is on %s, expected %s" % (what, t.device, ref.device))
    dt = _mix_types.get(t.dtype, -1)
    if dt < 0 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous [%d] tensor of float16, bfloat16 or float32 (got %s, %s)"
                         % (what, n, tuple(t.shape), t.dtype))
    return dt


def _ptr(t):
    return (t.data_ptr() or None) if t is not None else None


def _ws(ws, need, device):
    """(tensor to keep alive, pointer, bytes) of a workspace of `need` bytes."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = _torch.empty(need, dtype=_torch.uint8, device=device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on %s" % device)
    return ws, _ptr(ws), ws.numel() * ws.element_size()


def _enqueue(fn, device, *args):
    """fn(*args, current stream of device), with device current."""
    i = device.index
    if i == _torch.cuda.current_device():
        _check(fn(*args, _torch._C._cuda_getCurrentRawStream(i)))
    else:
        with _torch.cuda.device(device):
            _check(fn(*args, _torch._C._cuda_getCurrentRawStream(i)))


# Descriptors and workspace sizes by their fields (a model calls few shapes
# often), and by what of the thread's test override sizes depend on.

@functools.lru_cache(maxsize=1024)
def _ln_desc(*fields):
    """(descriptor reference, workspace bytes of the backward pass)"""
    prob = LayernormProblem(*fields, 0)
    b = ctypes.c_size_t()
    _check(lib().cnhwc_layernorm_workspace_size(ctypes.byref(prob), ctypes.byref(b)))
    return ctypes.byref(prob), b.value


@functools.lru_cache(maxsize=1024)
def _gated_desc(forced, op, unaligned, *fields):
    """(descriptor reference, workspace bytes)"""
    prob = GatedProblem(*fields, 0)
    b = ctypes.c_size_t()
    _check(lib().cnhwc_gated_workspace_size(ctypes.byref(prob), op, unaligned, ctypes.byref(b)))
    return ctypes.byref(prob), b.value


def _ln_params(dt, gamma, beta, c, ref):
    """param_dtype of gamma and beta (x's without either)."""
    pd = dt
    if gamma is not None:
        pd = _vector(gamma, c, "gamma", ref)
    if beta is not None:
        bd = _vector(beta, c, "beta", ref)
        if gamma is not None and bd != pd:
            raise ValueError("gamma is %s and beta is %s" % (gamma.dtype, beta.dtype))
        pd = bd
    return pd


def layernorm(x, gamma=None, beta=None, eps=1e-5, y=None):
    """(y, mean, rstd): layer norm of x [..., c] over its channels, and each
    row's fp32 statistics for layernorm_bwd."""
    torch = _t()
    dt = _operand(x, "x")
    rows, c, xs = _rows(x, "x")
    pd = _ln_params(dt, gamma, beta, c, x)
    y, ys = _out(y, "y", rows, c, x, xs)
    prob, _ = _ln_desc(rows, c, xs, ys, eps, dt, pd)
    dev = x.device
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    _enqueue(lib().cnhwc_layernorm_fwd, dev, prob, _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd))
    return y, mean, rstd


def layernorm_workspace(x, gamma=None):
    """Workspace bytes of layernorm_bwd for this x."""
    _t()
    dt = _operand(x, "x")
    rows, c, xs = _rows(x, "x")
    return _ln_desc(rows, c, xs, 0, 0.0, dt, _ln_params(dt, gamma, None, c, x))[1]


def layernorm_bwd(dy, x, mean, rstd, gamma=None, dx=None, param_dtype=None, ws=None):
    """(dx, dgamma, dbeta) of layernorm, from its x and statistics.  dgamma and
    dbeta have gamma's type (param_dtype, or x's, without a gamma).  dx has x's
    row stride."""
    torch = _t()
    dt = _operand(x, "x")
    rows, c, xs = _rows(x, "x")
    _same(dy, x, "dy")
    drows, _, ys = _rows(dy, "dy", c)
    if drows != rows:
        raise ValueError("dy has %d rows, x has %d" % (drows, rows))
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        _same(t, x, what, torch.float32)
        if t.numel() != rows or not t.is_contiguous():
            raise ValueError("%s must be a contiguous tensor of %d values" % (what, rows))
    ptype = gamma.dtype if gamma is not None else (param_dtype or x.dtype)
    if param_dtype is not None and param_dtype != ptype:
        raise ValueError("param_dtype is %s, gamma is %s" % (param_dtype, ptype))
    pd = _ln_params(dt, gamma, None, c, x) if gamma is not None else _mix_types.get(ptype, -1)
    if dx is None:
        dx = _new_rows(xs, c, x)
    else:
        _same(dx, x, "dx")
        if _rows(dx, "dx", c)[::2] != (rows, xs):
            raise ValueError("dx must have x's rows and row stride (%d)" % xs)
    dev = x.device
    dgamma = x.new_empty((c,), dtype=ptype)
    dbeta = torch.empty_like(dgamma)
    prob, need = _ln_desc(rows, c, xs, ys, 0.0, dt, pd)
    ws, wp, wb = _ws(ws, need, dev)
    _enqueue(lib().cnhwc_layernorm_bwd, dev, prob, _ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
             _ptr(dgamma), _ptr(dbeta), wp, wb)
    return dx, dgamma, dbeta


def _new_rows(stride, c, ref):
    """A new tensor of ref's shape with the given row stride, ref's own (the
    entry points give dx the row stride of x)."""
    if stride == c:
        return _torch.empty_like(ref)
    return ref.new_empty((*ref.shape[:-1], stride))[..., :c]


def _gated_operands(x, wg, wu, act):
    """(rows, c, f, row stride of x, act, dtype)"""
    dt = _operand(x, "x", f32=False)
    rows, c, xs = _rows(x, "x")
    a = ACTS.get(act, -1)
    if a < 0:
        raise ValueError("act must be one of %s (got %r)" % (", ".join(ACTS), act))
    f = wg.shape[0]
    for w, what in ((wg, "wg"), (wu, "wu")):
        _same(w, x, what)
        # [f, c], or the [f, 1, 1, c] filter of a pointwise convolution
        if w.dim() < 2 or w.shape[0] != f or w.shape[-1] != c or w.numel() != f * c or not w.is_contiguous():
            raise ValueError("%s must be a contiguous [%d, %d] tensor (got %s)" % (what, f, c, tuple(w.shape)))
    return rows, c, f, xs, a, dt


def _off16(*tensors):
    for t in tensors:
        if t.data_ptr() & 15:
            return 1
    return 0


def gated_workspace(x, wg, which="fwd", wu=None):
    """Workspace bytes of gated (which="fwd") or gated_bwd ("bwd") for operands
    like x, wg and wu.  Without wu it is taken to be aligned as wg is (the copies
    of weights off a 16-byte boundary lie in the workspace)."""
    _t()
    if which not in ("fwd", "bwd"):
        raise ValueError('which must be "fwd" or "bwd" (got %r)' % (which,))
    if wu is None:
        wu = wg
    rows, c, f, xs, a, dt = _gated_operands(x, wg, wu, "silu")
    op = OP_FWD if which == "fwd" else OP_DGRAD
    return _gated_desc(_forced.key, op, _off16(x, wg, wu), rows, c, f, xs, 0, a, dt)[1]


def gated_plan(x, wg, which="fwd"):
    """Names of the kernels the call runs on 16-byte-aligned operands."""
    _t()
    rows, c, f, xs, a, dt = _gated_operands(x, wg, wg, "silu")
    buf = ctypes.create_string_buffer(256)
    _check(lib().cnhwc_gated_plan(ctypes.byref(GatedProblem(rows, c, f, xs, 0, a, dt, 0)),
                                  OP_FWD if which == "fwd" else OP_DGRAD, buf, 256))
    return buf.value.decode()


def gated(x, wg, wu, act="silu", y=None, ws=None):
    """act(x wg^T) * (x wu^T) of x [..., c] and wg, wu [f, c] (or [f, 1, 1, c])."""
    _t()
    rows, c, f, xs, a, dt = _gated_operands(x, wg, wu, act)
    y, ys = _out(y, "y", rows, f, x, xs, (*x.shape[:-1], f))
    prob, need = _gated_desc(_forced.key, OP_FWD, _off16(x, wg, wu), rows, c, f, xs, ys, a, dt)
    ws, wp, wb = _ws(ws, need, x.device)
    _enqueue(lib().cnhwc_gated_fwd, x.device, prob, _ptr(x), _ptr(wg), _ptr(wu), _ptr(y), wp, wb)
    return y


def gated_bwd(dy, x, wg, wu, act="silu", need_dx=True, need_dw=True, ws=None):
    """(dx, dwg, dwu) of gated; None in the place of what is not needed.  dx
    has x's row stride."""
    torch = _t()
    rows, c, f, xs, a, dt = _gated_operands(x, wg, wu, act)
    _same(dy, x, "dy")
    drows, _, ys = _rows(dy, "dy", f)
    if drows != rows:
        raise ValueError("dy has %d rows, x has %d" % (drows, rows))
    dx = _new_rows(xs, c, x) if need_dx else None
    dwg = torch.empty_like(wg) if need_dw else None
    dwu = torch.empty_like(wu) if need_dw else None
    if rows or need_dw:          # an empty x has no dx to ask for
        prob, need = _gated_desc(_forced.key, OP_DGRAD, _off16(x, wg, wu), rows, c, f, xs, ys, a, dt)
        ws, wp, wb = _ws(ws, need, x.device)
        _enqueue(lib().cnhwc_gated_bwd, x.device, prob, _ptr(dy), _ptr(x), _ptr(wg), _ptr(wu), _ptr(dx), _ptr(dwg),
                 _ptr(dwu), wp, wb)
    return dx, dwg, dwu


def dropout(x, p, seed, offset=0, residual=None, y=None, device_offset=None):
    """residual + (keep ? x / (1 - p) : 0), the mask drawn by Philox4x32-10 from
    (seed, offset, element index).  device_offset: an int64 device tensor of one
    value that is added to offset when the kernel runs."""
    torch = _t()
    dt = _operand(x, "x")
    rows, c, xs = _rows(x, "x")
    rs = 0
    if residual is not None:
        _same(residual, x, "residual")
        rrows, _, rs = _rows(residual, "residual", c)
        if rrows != rows:
            raise ValueError("residual has %d rows, x has %d" % (rrows, rows))
    if device_offset is not None:
        _same(device_offset, x, "device_offset", torch.int64)
        if device_offset.numel() != 1:
            raise ValueError("device_offset must hold one value")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be in [0, 2^64) (got %d and %d)" % (seed, offset))
    y, ys = _out(y, "y", rows, c, x, xs)
    prob = DropoutProblem(rows, c, xs, rs, ys, p, seed, offset, dt, 0)
    _enqueue(lib().cnhwc_dropout, x.device, ctypes.byref(prob), _ptr(x), _ptr(residual), _ptr(y), _ptr(device_offset))
    return y


def dropout_bwd(dy, p, seed, offset=0, dx=None, device_offset=None):
    """The gradient of dropout in x (the residual's is dy itself): the same mask
    drawn again."""
    return dropout(dy, p, seed, offset, y=dx, device_offset=device_offset)


# ---- group norm -----------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _gn_desc(forced, op, *fields):
    """(descriptor reference, workspace bytes)"""
    prob = GroupnormProblem(*fields, 0)
    b = ctypes.c_size_t()
    _check(lib().cnhwc_groupnorm_workspace_size(ctypes.byref(prob), op, ctypes.byref(b)))
    return ctypes.byref(prob), b.value


def _act_or_none(act):
    a = ACTS_OR_NONE.get(act)
    if a is None:
        raise ValueError("act must be one of %s (got %r)" % (", ".join(ACTS_OR_NONE), act))
    return a


def _gn_operand(x, what="x"):
    """(samples, pixels, channels, row stride) of [n, ..., c]"""
    if x.dim() < 2:
        raise ValueError("%s needs a batch and a channel dimension (got shape %s)" % (what, tuple(x.shape)))
    rows, c, xs = _rows(x, what)
    n = x.shape[0]
    pixels = 1
    for s in x.shape[1:-1]:
        pixels *= s
    return n, pixels, c, xs


def group_norm(x, groups, gamma=None, beta=None, eps=1e-5, act="none", y=None, ws=None):
    """(y, mean, rstd): group norm of x [n, ..., c] over each sample's pixels and
    the c / groups channels of a group, then the activation; the fp32 statistics
    [n, groups] are for group_norm_bwd."""
    torch = _t()
    dt = _operand(x, "x")
    n, pixels, c, xs = _gn_operand(x)
    a = _act_or_none(act)
    pd = _ln_params(dt, gamma, beta, c, x)
    y, ys = _out(y, "y", n * pixels, c, x, xs)
    prob, need = _gn_desc(_forced.key, OP_FWD, n, pixels, c, xs, ys, eps, groups, a, dt, pd)
    mean = x.new_empty((n, groups), dtype=torch.float32)
    rstd = torch.empty_like(mean)
    ws, wp, wb = _ws(ws, need, x.device)
    _enqueue(lib().cnhwc_groupnorm_fwd, x.device, prob, _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
             wp, wb)
    return y, mean, rstd


def group_norm_workspace(x, groups, which="fwd"):
    """Workspace bytes of group_norm (which="fwd") or group_norm_bwd ("bwd") for this x."""
    _t()
    if which not in ("fwd", "bwd"):
        raise ValueError('which must be "fwd" or "bwd" (got %r)' % (which,))
    dt = _operand(x, "x")
    n, pixels, c, xs = _gn_operand(x)
    return _gn_desc(_forced.key, OP_FWD if which == "fwd" else OP_DGRAD, n, pixels, c, xs, 0, 0.0, groups, -1, dt, dt)[1]


def group_norm_bwd(dy, x, mean, rstd, groups, gamma=None, beta=None, act="none", dx=None, param_dtype=None, ws=None):
    """(dx, dgamma, dbeta) of group_norm, from its x and statistics.  dgamma and
    dbeta have gamma's type (param_dtype, or x's, without gamma and beta).  dx has
    x's row stride."""
    torch = _t()
    dt = _operand(x, "x")
    n, pixels, c, xs = _gn_operand(x)
    a = _act_or_none(act)
    _same(dy, x, "dy")
    drows, _, ys = _rows(dy, "dy", c)
    if drows != n * pixels:
        raise ValueError("dy has %d rows, x has %d" % (drows, n * pixels))
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        _same(t, x, what, torch.float32)
        if t.shape != (n, groups) or not t.is_contiguous():
            raise ValueError("%s must be a contiguous [%d, %d] tensor (got %s)" % (what, n, groups, tuple(t.shape)))
    given = gamma if gamma is not None else beta
    ptype = given.dtype if given is not None else (param_dtype or x.dtype)
    if param_dtype is not None and param_dtype != ptype:
        raise ValueError("param_dtype is %s, the weights are %s" % (param_dtype, ptype))
    pd = _ln_params(dt, gamma, beta, c, x) if given is not None else _mix_types.get(ptype, -1)
    if dx is None:
        dx = _new_rows(xs, c, x)
    else:
        _same(dx, x, "dx")
        if _rows(dx, "dx", c)[::2] != (n * pixels, xs):
            raise ValueError("dx must have x's rows and row stride (%d)" % xs)
    dgamma = x.new_empty((c,), dtype=ptype)
    dbeta = torch.empty_like(dgamma)
    prob, need = _gn_desc(_forced.key, OP_DGRAD, n, pixels, c, xs, ys, 0.0, groups, a, dt, pd)
    ws, wp, wb = _ws(ws, need, x.device)
    _enqueue(lib().cnhwc_groupnorm_bwd, x.device, prob, _ptr(dy), _ptr(x), _ptr(gamma), _ptr(beta), _ptr(mean), _ptr(rstd),
             _ptr(dx), _ptr(dgamma), _ptr(dbeta), wp, wb)
    return dx, dgamma, dbeta


# ---- AdamW ------------------------------------------------------------------------

ADAMW_BLOCK = 256   # CNHWC_ADAMW_BLOCK: elements that share a scale of 8-bit moments


class AdamW:
    """AdamW over a model's tensors, in place: one launch for up to 52 of them.

    params: contiguous GPU tensors of float32, float16 or bfloat16 on one
    device.  copies: for each a tensor of the same size that receives the
    updated values in its own type (the 16-bit weights of the next pass), or
    None.  bits: 32 (fp32 moments) or 8 (a byte each and a scale for every 256
    elements; see cnhwc_adamw for the codes).  weight_decay: one number, or one
    for each tensor.  seed: of the draws that round 8-bit moments (another than
    the dropout's, which draws the same words under the same seed).

    The moments of all tensors lie in flat tensors ``m`` and ``v`` (and
    ``scales`` [2, blocks] for 8 bits), tensor i's from ``offsets[i]`` on, a
    multiple of 256; ``state`` takes them as an earlier run left them, with its
    ``steps``, and so does assigning to ``m``, ``v`` and ``scales`` later.  What lies
    between the tensors stays as it is.

    A tensor whose memory is exchanged (``p.data = ...``, ``set_``) is followed to
    where it lies at the next step, if its size still fits; until then the
    optimizer holds the memory that it had.  (A captured step keeps the addresses
    that it was captured with.)"""

    def __init__(self, params, bits=32, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, copies=None, seed=0, state=None,
                 steps=0):
        torch = _t()
        self.params = tuple(params)
        if not self.params:
            raise ValueError("params is empty")
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32 (got %r)" % (bits,))
        if not 0 <= seed < 1 << 64:
            raise ValueError("seed must be in [0, 2^64) (got %d)" % seed)
        count = len(self.params)
        decays = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * count
        self.copies = tuple(copies) if copies is not None else (None,) * count
        for what, v in (("weight_decay", decays), ("copies", self.copies)):
            if len(v) != count:
                raise ValueError("%s has %d entries for %d tensors" % (what, len(v), count))
        self.device, self.bits, self.steps = self.params[0].device, bits, steps
        self.offsets, self._sizes, at = [], [p.numel() for p in self.params], 0
        self._list = (AdamwTensor * count)()
        for t, n, d in zip(self._list, self._sizes, decays):
            t.n, t.weight_decay = n, d
            self.offsets.append(at)
            at += -(-n // ADAMW_BLOCK) * ADAMW_BLOCK
        kind = torch.float32 if bits == 32 else torch.uint8
        self._shapes = [((at,), kind), ((at,), kind)] + [((2, at // ADAMW_BLOCK), torch.float32)] * (bits == 8)
        if state is None:
            state = [torch.zeros(shape, dtype=dtype, device=self.device) for shape, dtype in self._shapes]
        elif len(state) != len(self._shapes):
            raise ValueError("state must be (m, v%s)" % (", scales" if bits == 8 else ""))
        self._state = list(state)
        self.grads, self._fixed, self._watched = None, [], []
        self._look()
        self._prob = AdamwProblem(0.0, betas[0], betas[1], eps, 0, seed, bits, count)

    def _check(self, t, what, i, n):
        fits = t.device == self.device and t.numel() == n and t.is_contiguous()
        if fits and t.is_cuda and t.dtype in _mix_types:
            return _mix_types[t.dtype]
        what = "%s[%d]" % (what, i)     # (made where it is needed: it takes as long as the check)
        dt = _operand(t, what)
        if not fits:
            raise ValueError("%s must be a contiguous tensor of %d values on %s" % (what, n, self.device))
        return dt

    def _check_all(self, tensors, what):
        """The element types of a list with a tensor for each of params."""
        return [self._check(t, what, i, n) for i, (t, n) in enumerate(zip(tensors, self._sizes))]

    def _look(self):
        """Checks all tensors, then takes their addresses.  Their storages are held, so
        that nothing else can come to lie at an address that a step compares."""
        for t, (shape, dtype), what in zip(self._state, self._shapes, ("m", "v", "scales")):
            if t.device != self.device or t.shape != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError("state %s must be a contiguous %s tensor of %s on %s" % (what, list(shape), dtype, self.device))
        bound = self._watched[len(self._fixed):]
        types, grad_types = self._check_all(self.params, "params"), self._check_all(bound, "grads")
        copy_types = [c if c is None else self._check(c, "copies", i, n) for i, (c, n) in enumerate(zip(self.copies, self._sizes))]
        scales = self.scales if self.bits == 8 else ()
        for t, p, dt, copy, ct, n, o in zip(self._list, self.params, types, self.copies, copy_types, self._sizes, self.offsets):
            t.p, t.p_dtype = _ptr(p), dt
            if copy is not None:
                t.copy, t.copy_dtype = _ptr(copy), ct
            if n:
                t.m, t.v = (s.data_ptr() + o * s.element_size() for s in self._state[:2])
                if self.bits == 8:
                    t.m_scale, t.v_scale = (s.data_ptr() + o // ADAMW_BLOCK * 4 for s in scales)
        self._fixed = [*self.params, *(c for c in self.copies if c is not None), *self._state]
        self._at = [t.data_ptr() for t in self._fixed]
        self._held = [t.untyped_storage() for t in self._fixed]
        self._take(bound, grad_types, True)

    def _take(self, grads, types, bound):
        """Takes the addresses of checked gradients; bound: for more steps than the next."""
        for t, g, dt in zip(self._list, grads, types):
            t.g, t.g_dtype = _ptr(g), dt
        later, fixed = grads if bound else [], len(self._fixed)
        self._watched = self._fixed + later
        self._at[fixed:] = [g.data_ptr() for g in later]
        self._held[fixed:] = [g.untyped_storage() for g in later]

    def _follow(self, tensors, at):
        if list(map(_torch.Tensor.data_ptr, tensors)) != at:
            self._look()

    def _exchange(self, i, what, t):
        if i >= len(self._state) or not isinstance(t, _torch.Tensor):
            raise ValueError("%s cannot be %s" % (what, type(t).__name__))
        kept, self._state[i] = self._state[i], t
        try:
            self._look()
        except ValueError:
            self._state[i] = kept
            raise

    m = property(lambda self: self._state[0], lambda self, t: self._exchange(0, "m", t))
    v = property(lambda self: self._state[1], lambda self, t: self._exchange(1, "v", t))
    scales = property(lambda self: self._state[2] if self.bits == 8 else None, lambda self, t: self._exchange(2, "scales", t))

    def bind(self, grads):
        """The gradients of the steps to come: for each tensor one of its size,
        of any of the types.  A program whose gradients always lie in the same
        buffers binds them once."""
        self._gradients(grads, True)

    def _gradients(self, grads, bound):
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError("%d gradients for %d tensors" % (len(grads), len(self.params)))
        self._take(grads, self._check_all(grads, "grads"), bound)
        self.grads = grads

    def step(self, lr, grads=None, grad_scale=None, device_lr=None, device_step=None):
        """One step with these gradients (or those bound before).  For a captured
        graph, whose replays repeat a call: grad_scale and device_lr, float32
        device tensors of one value that multiply the gradients and lr, and
        device_step, an int64 one that is added to the step's number."""
        if grads is not None:
            self._gradients(grads, False)
        elif self.grads is None:
            raise ValueError("no gradients given or bound")
        elif len(self._watched) == len(self._fixed):
            self.bind(self.grads)     # an earlier step's
        for t, dtype, what in ((grad_scale, "float32", "grad_scale"), (device_lr, "float32", "device_lr"),
                               (device_step, "int64", "device_step")):
            if t is not None:
                _same(t, self.m, what, getattr(_torch, dtype))
                if t.numel() != 1:
                    raise ValueError("%s must hold one value" % what)
        self._follow(self._watched, self._at)
        q = self._prob
        q.lr, q.step = lr, self.steps + 1
        _enqueue(lib().cnhwc_adamw, self.device, ctypes.byref(q), self._list, _ptr(grad_scale), _ptr(device_lr),
                 _ptr(device_step))
        self.steps += 1

    def moments(self):
        """(m, v) as flat float32 tensors: what 8-bit moments stand for, or the
        fp32 moments themselves."""
        self._follow(self._state, self._at[len(self._fixed) - len(self._state):len(self._fixed)])
        if self.bits == 32:
            return self.m, self.v
        m = _torch.empty(self.m.shape, dtype=_torch.float32, device=self.device)
        v = _torch.empty_like(m)
        _enqueue(lib().cnhwc_adamw_moments, self.device, m.numel(), _ptr(self.m), _ptr(self.v), _ptr(self.scales[0]),
                 _ptr(self.scales[1]), _ptr(m), _ptr(v))
        return m, v


# ---- products in 8-bit integers ----------------------------------------------------

def quantize_rows(x, q=None):
    """(q, scale): the rows of x [..., c] in 8-bit integers, q = x / scale to the
    nearest, and their fp32 scales [...], max|x| / 127.  A new q has rows of a
    multiple of 16 bytes (zeros behind c): linear_i8 takes such weights as they
    are, and such an x too unless it has many rows of a c that is no multiple of
    16 itself (nothing tells it of the zeros, so it makes a copy that has them)."""
    torch = _t()
    dt = _operand(x, "x")
    rows, c, xs = _rows(x, "x")
    if q is None:
        pitch = -(-c // 16) * 16
        q = x.new_empty((*x.shape[:-1], pitch), dtype=torch.int8)[..., :c]
        qs = pitch
    else:
        _same(q, x, "q", torch.int8)
        qrows, _, qs = _rows(q, "q", c)
        if qrows != rows:
            raise ValueError("q has %d rows, x has %d" % (qrows, rows))
        if qs != c:
            raise ValueError("q must be dense (its rows are %d apart)" % qs)
    scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
    prob = QuantizeProblem(rows, c, xs, qs, dt, 0)
    _enqueue(lib().cnhwc_quantize_rows, x.device, ctypes.byref(prob), _ptr(x), _ptr(q), _ptr(scale))
    return q, scale


@functools.lru_cache(maxsize=1024)
def _linear_desc(forced, unaligned, *fields):
    """(descriptor reference, workspace bytes)"""
    prob = LinearI8Problem(*fields, 0)
    b = ctypes.c_size_t()
    _check(lib().cnhwc_linear_i8_workspace_size(ctypes.byref(prob), unaligned, ctypes.byref(b)))
    return ctypes.byref(prob), b.value


def _linear_operands(x, w):
    """(rows, c, f, row strides of x and w, x's type)"""
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor (got %s)" % x.device)
    dt = I8 if x.dtype == _torch.int8 else _operand(x, "x")
    rows, c, xs = _rows(x, "x")
    _same(w, x, "w", _torch.int8)
    f, _, ws = _rows(w, "w", c)
    return rows, c, f, xs, ws, dt


def linear_i8_workspace(x, w, act=None):
    """Workspace bytes of linear_i8 for operands like x and w and this act;
    without one, enough for every act (how a product is divided depends on it)."""
    _t()
    rows, c, f, xs, ws, dt = _linear_operands(x, w)
    acts = ACTS_OR_NONE.values() if act is None else (_act_or_none(act),)
    return max(_linear_desc(_forced.key, _off16(x, w), rows, c, f, xs, ws, 0, 0, a, dt, BF16)[1] for a in acts)


def linear_i8_plan(x, w, act="none", residual=None, y=None):
    """Names of the kernels the call runs on 16-byte-aligned operands."""
    _t()
    rows, c, f, xs, ws, dt = _linear_operands(x, w)
    rs, ys = (_rows(t, what, f)[2] if t is not None else 0 for t, what in ((residual, "residual"), (y, "y")))
    buf = ctypes.create_string_buffer(256)
    _check(lib().cnhwc_linear_i8_plan(ctypes.byref(LinearI8Problem(rows, c, f, xs, ws, rs, ys, _act_or_none(act), dt, BF16, 0)),
                                      buf, 256))
    return buf.value.decode()


def linear_i8(x, w, w_scale, x_scale=None, bias=None, residual=None, act="none", dtype=None, y=None, ws=None):
    """act((x w^T) * scales + bias) + residual in 8-bit integers: w [f, c] (or the
    [f, 1, 1, c] filter of a pointwise convolution) and w_scale [f] from
    quantize_rows; x [..., c] either 8-bit integers with their x_scale [...], or
    values, which are quantized row by row on the way.  bias [f] is fp32; y has
    the residual's type, x's (where it is a 16-bit one), or dtype."""
    torch = _t()
    rows, c, f, xs, wst, dt = _linear_operands(x, w)
    a = _act_or_none(act)
    for t, n, what in ((w_scale, f, "w_scale"), (bias, f, "bias"), (x_scale, rows, "x_scale")):
        if t is not None:
            _same(t, x, what, torch.float32)
            if t.numel() != n or not t.is_contiguous():
                raise ValueError("%s must be a contiguous tensor of %d values" % (what, n))
    if (dt == I8) != (x_scale is not None):
        raise ValueError("x_scale goes with an x of 8-bit integers, and only with one")
    for t in (y, residual):
        if t is not None:
            dtype = dtype or t.dtype
    if dtype is None and dt in (F16, BF16):
        dtype = x.dtype
    out = _mix_types.get(dtype, -1)
    if out not in (F16, BF16):
        raise ValueError("y must be float16 or bfloat16 (got %s)" % dtype)
    rs = 0
    if residual is not None:
        _same(residual, x, "residual", dtype)
        rrows, _, rs = _rows(residual, "residual", f)
        if rrows != rows:
            raise ValueError("residual has %d rows, x has %d" % (rrows, rows))
    if y is None:
        y, ys = x.new_empty((*x.shape[:-1], f), dtype=dtype), f
    else:
        _same(y, x, "y", dtype)
        yrows, _, ys = _rows(y, "y", f)
        if yrows != rows:
            raise ValueError("y has %d rows, expected %d" % (yrows, rows))
    prob, need = _linear_desc(_forced.key, _off16(x, w), rows, c, f, xs, wst, rs, ys, a, dt, out)
    ws, wp, wb = _ws(ws, need, x.device)
    _enqueue(lib().cnhwc_linear_i8, x.device, prob, _ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(bias),
             _ptr(residual), _ptr(y), wp, wb)
    return y
