"""Thin ctypes binding of libdora.so (include/dora.h), same names as the C ABI.

Argument marshalling only: tensors are passed as device pointers, outputs and
the workspace are allocated with torch (device memory plumbing), and every
step of the computation runs in the library's HIP kernels.  There is no CPU
or PyTorch fallback: if the library is missing or cannot be loaded, every
call raises.
"""
import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdora.so")

DORA_F32, DORA_BF16 = 0, 1
STATUS = {0: "DORA_OK", 1: "DORA_E_NULL", 2: "DORA_E_SHAPE", 3: "DORA_E_DTYPE",
          4: "DORA_E_ALIGN", 5: "DORA_E_WORKSPACE", 6: "DORA_E_ALIAS", 7: "DORA_E_HIP",
          8: "DORA_E_VALUE"}

# Every symbol include/dora.h declares.
EXPORTS = ("dora_strerror", "dora_last_error", "dora_norm_workspace", "dora_forward_workspace",
           "dora_backward_workspace", "dora_factored_norm", "dora_compose", "dora_forward",
           "dora_backward", "dora_linear_workspace", "dora_linear", "dora_merge_workspace",
           "dora_merge", "dora_backward_through_norm_workspace", "dora_backward_through_norm",
           "dora_factored_norm_grouped_workspace", "dora_factored_norm_grouped",
           "dora_forward_grouped_workspace", "dora_forward_grouped", "dora_forward_noalloc",
           "dora_rmsnorm", "dora_rmsnorm_backward_workspace", "dora_rmsnorm_backward",
           "dora_quantize_rows", "dora_dequantize_rows", "dora_linear_quantized_workspace",
           "dora_linear_quantized", "dora_backward_checkpoint_workspace",
           "dora_backward_checkpoint")

_lib = None


class DoraModule(ctypes.Structure):
    """struct dora_module of include/dora.h."""
    _fields_ = [("W", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("s", ctypes.c_float), ("d_out", ctypes.c_int64),
                ("d_in", ctypes.c_int64), ("r", ctypes.c_int64)]


class DoraError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


def lib():
    """Load libdora.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} not built; run python -m dora_adapter_amd.build first")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, sz, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        c_int = ctypes.c_int
        L.dora_strerror.restype = ctypes.c_char_p
        L.dora_strerror.argtypes = [c_int]
        L.dora_last_error.restype = ctypes.c_char_p
        L.dora_last_error.argtypes = []
        L.dora_norm_workspace.restype = sz
        L.dora_norm_workspace.argtypes = [i64, i64, i64, c_int]
        L.dora_forward_workspace.restype = sz
        L.dora_forward_workspace.argtypes = [i64, i64, i64, i64, c_int]
        L.dora_backward_workspace.restype = sz
        L.dora_backward_workspace.argtypes = [i64, i64, i64, i64, c_int]
        L.dora_factored_norm.restype = c_int
        L.dora_factored_norm.argtypes = [p, p, p, f, i64, i64, i64, c_int, p, p, p, p, p, p, sz,
                                         p]
        L.dora_compose.restype = c_int
        L.dora_compose.argtypes = [p, p, p, p, f, i64, i64, c_int, p, p]
        L.dora_forward.restype = c_int
        L.dora_forward.argtypes = [p, p, p, p, p, f, i64, i64, i64, i64, c_int, p, p, p, p, p,
                                   p, sz, p]
        L.dora_backward.restype = c_int
        L.dora_backward.argtypes = [p, p, p, p, p, p, p, f, p, p, i64, i64, i64, i64, c_int, p,
                                    p, p, p, p, sz, p]
        L.dora_backward_through_norm_workspace.restype = sz
        L.dora_backward_through_norm_workspace.argtypes = [i64, i64, i64, i64, c_int]
        L.dora_backward_through_norm.restype = c_int
        L.dora_backward_through_norm.argtypes = [p, p, p, p, p, p, p, f, p, p, p, i64, i64, i64,
                                                 i64, c_int, p, p, p, p, p, sz, p]
        mp = ctypes.POINTER(DoraModule)
        L.dora_factored_norm_grouped_workspace.restype = sz
        L.dora_factored_norm_grouped_workspace.argtypes = [mp, c_int, c_int]
        L.dora_factored_norm_grouped.restype = c_int
        L.dora_factored_norm_grouped.argtypes = [mp, c_int, c_int, p, p, sz, p]
        L.dora_forward_grouped_workspace.restype = sz
        L.dora_forward_grouped_workspace.argtypes = [mp, c_int, i64, c_int, p, p]
        L.dora_forward_grouped.restype = c_int
        L.dora_forward_grouped.argtypes = [p, i64, i64, mp, c_int, c_int, p, p, p, p, p, sz, p]
        L.dora_linear_workspace.restype = sz
        L.dora_linear_workspace.argtypes = [i64, i64, i64, c_int]
        L.dora_linear.restype = c_int
        L.dora_linear.argtypes = [p, p, i64, i64, i64, c_int, p, p, sz, p]
        L.dora_forward_noalloc.restype = c_int
        L.dora_forward_noalloc.argtypes = [p, p, p, p, p, f, i64, i64, i64, i64, c_int, p, p, p,
                                           p, p, p]
        L.dora_merge_workspace.restype = sz
        L.dora_merge_workspace.argtypes = [i64, i64, i64, c_int]
        L.dora_merge.restype = c_int
        L.dora_merge.argtypes = [p, p, p, p, f, i64, i64, i64, c_int, p, p, p, sz, p]
        L.dora_rmsnorm.restype = c_int
        L.dora_rmsnorm.argtypes = [p, p, p, f, i64, i64, c_int, i64, p, p, p, p, p, p]
        L.dora_rmsnorm_backward_workspace.restype = sz
        L.dora_rmsnorm_backward_workspace.argtypes = [i64, i64, c_int]
        L.dora_rmsnorm_backward.restype = c_int
        L.dora_rmsnorm_backward.argtypes = [p, p, p, p, p, i64, i64, c_int, p, p, p, sz, p]
        L.dora_quantize_rows.restype = c_int
        L.dora_quantize_rows.argtypes = [p, i64, i64, c_int, i64, p, p, p]
        L.dora_dequantize_rows.restype = c_int
        L.dora_dequantize_rows.argtypes = [p, p, i64, i64, c_int, i64, p, p]
        L.dora_linear_quantized_workspace.restype = sz
        L.dora_linear_quantized_workspace.argtypes = [i64, i64, i64, c_int]
        L.dora_linear_quantized.restype = c_int
        L.dora_linear_quantized.argtypes = [p, p, p, p, i64, i64, i64, c_int, p, p, sz, p]
        L.dora_backward_checkpoint_workspace.restype = sz
        L.dora_backward_checkpoint_workspace.argtypes = [i64, i64, i64, i64, c_int, c_int]
        L.dora_backward_checkpoint.restype = c_int
        L.dora_backward_checkpoint.argtypes = [p, p, p, p, p, p, p, p, f, p, p, p, i64, p, c_int,
                                               i64, i64, i64, i64, c_int, p, p, p, p, p, sz, p]
        _lib = L
    return _lib


def _dt(t):
    if t.dtype == torch.bfloat16:
        return DORA_BF16
    if t.dtype == torch.float32:
        return DORA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(rc):
    if rc != 0:
        raise DoraError(rc, lib().dora_last_error().decode())


def _dev(t):
    if not t.is_cuda:
        raise ValueError("libdora needs device tensors")
    return t.device


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def dora_norm_workspace(d_out, d_in, r, dtype):
    return lib().dora_norm_workspace(d_out, d_in, r, dtype)


def dora_forward_workspace(T, d_in, d_out, r, dtype):
    return lib().dora_forward_workspace(T, d_in, d_out, r, dtype)


def dora_backward_workspace(T, d_in, d_out, r, dtype):
    return lib().dora_backward_workspace(T, d_in, d_out, r, dtype)


def dora_backward_through_norm_workspace(T, d_in, d_out, r, dtype):
    return lib().dora_backward_through_norm_workspace(T, d_in, d_out, r, dtype)


def dora_backward_through_norm(dy, x, W, A, B, m, n, s, P, y, U=None, ws=None, out=None):
    """Backward with the gradient flowing through the row norm (U: the
    forward's kept V A^T = W A^T + s B A A^T, optional)."""
    return dora_backward(dy, x, W, A, B, m, n, s, P, y, ws=ws, out=out, through_norm=True, U=U)


def dora_factored_norm(W, A, B, s, terms=False, ws=None, n=None, U_out=None):
    """Row norms of W + s*B*A (fp32 [d_out]); with terms=True also returns
    (base, cross, gram).  U_out (fp32 [d_out, r]) receives
    V A^T = W A^T + s B A A^T."""
    dev = _dev(W)
    d_out, d_in = W.shape
    r = A.shape[0]
    dt = _dt(W)
    n = torch.empty(d_out, dtype=torch.float32, device=dev) if n is None else n
    extra = [torch.empty(d_out, dtype=torch.float32, device=dev) for _ in range(3)] if terms \
        else [None, None, None]
    need = lib().dora_norm_workspace(d_out, d_in, r, dt)
    ws = _ws(need, dev) if ws is None else ws
    _check(lib().dora_factored_norm(_ptr(W), _ptr(A), _ptr(B), float(s), d_out, d_in, r, dt,
                                    _ptr(n), *[_ptr(e) for e in extra], _ptr(U_out), _ptr(ws),
                                    ws.numel(), _stream(dev)))
    return (n, *extra) if terms else n


def dora_compose(base, lora, m, n, s, y=None):
    """y = (m/n) (.) (base + s*lora) in the stable single-pass form; y may be base."""
    dev = _dev(base)
    T, d_out = base.shape
    y = torch.empty_like(base) if y is None else y
    _check(lib().dora_compose(_ptr(base), _ptr(lora), _ptr(m), _ptr(n), float(s), T, d_out,
                              _dt(base), _ptr(y), _stream(dev)))
    return y


def dora_forward(x, W, A, B, m, s, n_in=None, want_P=True, ws=None, y=None, n_out=None,
                 P_out=None, U_out=None):
    """Module forward.  Returns (y, n, P) (P is None when want_P is False).
    U_out (fp32 [d_out, r]) receives the norm's V A^T = W A^T + s B A A^T for
    the backward through the norm."""
    dev = _dev(x)
    T, d_in = x.shape
    d_out = W.shape[0]
    r = A.shape[0]
    dt = _dt(x)
    y = torch.empty(T, d_out, dtype=x.dtype, device=dev) if y is None else y
    n_out = torch.empty(d_out, dtype=torch.float32, device=dev) if n_out is None else n_out
    if want_P and P_out is None:
        P_out = torch.empty(T, r, dtype=x.dtype, device=dev)
    need = lib().dora_forward_workspace(T, d_in, d_out, r, dt)
    ws = _ws(need, dev) if ws is None else ws
    _check(lib().dora_forward(_ptr(x), _ptr(W), _ptr(A), _ptr(B), _ptr(m), float(s), T, d_in,
                              d_out, r, dt, _ptr(y), _ptr(n_out), _ptr(P_out if want_P else None),
                              _ptr(n_in), _ptr(U_out), _ptr(ws), ws.numel(), _stream(dev)))
    return y, n_out, (P_out if want_P else None)


def dora_forward_noalloc(x, W, A, B, m, s, n_in=None, want_P=True, y=None, n_out=None,
                         P_out=None, U_out=None):
    """dora_forward on the library's fixed scratch (no workspace argument;
    the library allocates nothing).  Outputs as dora_forward."""
    dev = _dev(x)
    T, d_in = x.shape
    d_out = W.shape[0]
    r = A.shape[0]
    y = torch.empty(T, d_out, dtype=x.dtype, device=dev) if y is None else y
    n_out = torch.empty(d_out, dtype=torch.float32, device=dev) if n_out is None else n_out
    if want_P and P_out is None:
        P_out = torch.empty(T, r, dtype=x.dtype, device=dev)
    _check(lib().dora_forward_noalloc(_ptr(x), _ptr(W), _ptr(A), _ptr(B), _ptr(m), float(s), T,
                                      d_in, d_out, r, _dt(x), _ptr(y), _ptr(n_out),
                                      _ptr(P_out if want_P else None), _ptr(n_in), _ptr(U_out),
                                      _stream(dev)))
    return y, n_out, (P_out if want_P else None)


def dora_backward(dy, x, W, A, B, m, n, s, P, y, ws=None, out=None, through_norm=False, U=None):
    """Backward; returns dict(dx, dA, dB, dm).  The norm is detached unless
    through_norm is set (then dA and dB include the path through n)."""
    dev = _dev(W)
    T, d_in = x.shape
    d_out = W.shape[0]
    r = A.shape[0]
    dt = _dt(W)
    if out is None:
        out = {"dx": torch.empty(T, d_in, dtype=W.dtype, device=dev),
               "dA": torch.empty(r, d_in, dtype=W.dtype, device=dev),
               "dB": torch.empty(d_out, r, dtype=W.dtype, device=dev),
               "dm": torch.empty(d_out, dtype=torch.float32, device=dev)}
    L = lib()
    size, call = ((L.dora_backward_through_norm_workspace, L.dora_backward_through_norm)
                  if through_norm else (L.dora_backward_workspace, L.dora_backward))
    need = size(T, d_in, d_out, r, dt)
    ws = _ws(need, dev) if ws is None else ws
    extra = (_ptr(U),) if through_norm else ()
    if U is not None and not through_norm:
        raise ValueError("U is used by the backward through the norm only")
    _check(call(_ptr(dy), _ptr(x), _ptr(W), _ptr(A), _ptr(B), _ptr(m), _ptr(n), float(s),
                _ptr(P), _ptr(y), *extra, T, d_in, d_out, r, dt, _ptr(out["dx"]),
                _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dm"]), _ptr(ws), ws.numel(),
                _stream(dev)))
    return out


def dora_linear_workspace(T, d_in, d_out, dtype):
    return lib().dora_linear_workspace(T, d_in, d_out, dtype)


def dora_linear(x, W, y=None, ws=None):
    """y = x W^T on the forward's base-product kernel (merged-weight inference)."""
    dev = _dev(x)
    T, d_in = x.shape
    d_out = W.shape[0]
    dt = _dt(x)
    y = torch.empty(T, d_out, dtype=x.dtype, device=dev) if y is None else y
    need = lib().dora_linear_workspace(T, d_in, d_out, dt)
    if ws is None and need > 0:
        ws = _ws(need, dev)
    _check(lib().dora_linear(_ptr(x), _ptr(W), T, d_in, d_out, dt, _ptr(y), _ptr(ws),
                             0 if ws is None else ws.numel(), _stream(dev)))
    return y


def dora_merge_workspace(d_out, d_in, r, dtype):
    return lib().dora_merge_workspace(d_out, d_in, r, dtype)


def dora_merge(W, A, B, m, s, n_in=None, out=None, ws=None):
    """Merged weight W' = (m/n) (W + s B A) by rows (n factored unless n_in
    is given); out may be W itself."""
    dev = _dev(W)
    d_out, d_in = W.shape
    r = A.shape[0]
    dt = _dt(W)
    out = torch.empty_like(W) if out is None else out
    need = lib().dora_merge_workspace(d_out, d_in, r, dt)
    ws = _ws(need, dev) if ws is None else ws
    _check(lib().dora_merge(_ptr(W), _ptr(A), _ptr(B), _ptr(m), float(s), d_out, d_in, r, dt,
                            _ptr(n_in), _ptr(out), _ptr(ws), ws.numel(), _stream(dev)))
    return out


def _modules(mods):
    """(W, A, B, m, s) tuples -> a ctypes array of DoraModule."""
    arr = (DoraModule * max(len(mods), 1))()
    for k, (W, A, B, m, s) in enumerate(mods):
        arr[k] = DoraModule(W.data_ptr(), A.data_ptr(), B.data_ptr(),
                            None if m is None else m.data_ptr(), float(s), W.shape[0],
                            W.shape[1], A.shape[0])
    return arr


def _ptrs(ts):
    """Host array of device pointers (None entries stay NULL); None -> NULL."""
    if ts is None:
        return None
    arr = (ctypes.c_void_p * max(len(ts), 1))()
    for k, t in enumerate(ts):
        arr[k] = None if t is None else t.data_ptr()
    return arr


def dora_factored_norm_grouped_workspace(mods, dtype):
    return lib().dora_factored_norm_grouped_workspace(_modules(mods), len(mods), dtype)


def dora_forward_grouped_workspace(mods, T, dtype, n_in=None, P_out=None):
    return lib().dora_forward_grouped_workspace(_modules(mods), len(mods), T, dtype,
                                                _ptrs(n_in), _ptrs(P_out))


def dora_factored_norm_grouped(mods, ns=None, ws=None):
    """Row norms of W + sBA for every (W, A, B, m, s) in mods (m unused), in
    grouped launches.  Returns the list of fp32 norms."""
    if not mods:
        return []
    dev = _dev(mods[0][0])
    dt = _dt(mods[0][0])
    arr = _modules(mods)
    ns = [torch.empty(W.shape[0], dtype=torch.float32, device=dev) for W, *_ in mods] \
        if ns is None else ns
    need = lib().dora_factored_norm_grouped_workspace(arr, len(mods), dt)
    ws = _ws(need, dev) if ws is None else ws
    keep = _ptrs(ns)
    _check(lib().dora_factored_norm_grouped(arr, len(mods), dt, ctypes.cast(keep, ctypes.c_void_p),
                                            _ptr(ws), ws.numel(), _stream(dev)))
    return ns


def dora_forward_grouped(x, mods, n_in=None, want_P=True, ws=None, ys=None, ns=None, Ps=None):
    """dora_forward for sibling modules sharing x.  mods: (W, A, B, m, s)
    tuples; n_in: optional list of cached norms (entries may be None).
    Returns (ys, ns, Ps)."""
    if not mods:
        return [], [], []
    dev = _dev(x)
    T, d_in = x.shape
    dt = _dt(x)
    arr = _modules(mods)
    ys = [torch.empty(T, W.shape[0], dtype=x.dtype, device=dev) for W, *_ in mods] \
        if ys is None else ys
    ns = [torch.empty(W.shape[0], dtype=torch.float32, device=dev) for W, *_ in mods] \
        if ns is None else ns
    if want_P and Ps is None:
        Ps = [torch.empty(T, A.shape[0], dtype=x.dtype, device=dev) for _, A, *_ in mods]
    if not want_P:
        Ps = None
    py, pn, pP, pnin = _ptrs(ys), _ptrs(ns), _ptrs(Ps), _ptrs(n_in)
    vp = lambda a: None if a is None else ctypes.cast(a, ctypes.c_void_p)  # noqa: E731
    need = lib().dora_forward_grouped_workspace(arr, len(mods), T, dt, vp(pnin), vp(pP))
    ws = _ws(need, dev) if ws is None else ws
    _check(lib().dora_forward_grouped(_ptr(x), T, d_in, arr, len(mods), dt, vp(py), vp(pn),
                                      vp(pP), vp(pnin), _ptr(ws), ws.numel(), _stream(dev)))
    return ys, ns, Ps


# ------------------------------------------------ 8-bit rows and their users
# The calls below check what they are given: every tensor on one device,
# contiguous, of the type and shape the call documents (ValueError, TypeError
# otherwise), and they launch with that device current.

def _need(name, t, dev, dtype, *shape):
    """Refuse a tensor that is not what the library would read."""
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous():
        return t
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    raise ValueError(f"{name} is not contiguous")


def _at(t):
    return None if t is None else t.data_ptr()


def _rows(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} has {t.dim()} dimensions, not 2")
    return t.shape


def _groups(d, group):
    """Scales of a row of d values (one, or one for each `group` columns)."""
    if group == 0:
        return 1
    if group not in (32, 64, 128, 256, 512):
        raise ValueError(f"group {group} is neither 0 nor a power of two from 32 to 512")
    return -(-d // group)


def _need_ws(ws, dev):
    if ws is not None:
        if ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
            raise ValueError(f"ws is not a contiguous uint8 tensor on {dev}")
    return ws


# The handle of a device's current stream without a Stream object around it
# (1.7 us less a call, a fifth of a small call's host time), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev, call, *args):
    """The call on the current stream of `dev`, with `dev` current."""
    stream = _raw_stream(dev.index)
    if torch.cuda.current_device() == dev.index:
        rc = call(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, stream)
    if rc != 0:
        _check(rc)


def _norm_outputs(dtype, T, d, n):
    return {"y": (dtype, T, d), "h": (dtype, T, d), "rstd": (torch.float32, T),
            "q": (torch.int8, T, d), "scale": (torch.float32, T, n)}


def dora_rmsnorm(x, w, eps=1e-6, residual=None, want_y=True, want_h=None, want_rstd=False,
                 quantize=False, group=0, out=None):
    """h = x + residual (rounded to the element type) and y = w h / sqrt(mean(h^2) + eps) by
    rows of x [T, d].  Returns a dict of what was asked for: "y", "h" (want_h; by default with
    a residual), "rstd" (fp32 [T], for the backward), and with quantize "q" (int8 [T, d]) and
    "scale" (fp32 [T, groups]: one group, or one for each `group` columns) standing for y.
    out: a dict of preallocated outputs; then those are what is asked for.  out["h"] may be x
    or residual, out["y"] may be x."""
    dev = _dev(x)
    T, d = _rows("x", x)
    dt = _dt(x)
    n = _groups(d, group)
    _need("x", x, dev, x.dtype, T, d)
    _need("w", w, dev, x.dtype, d)
    if residual is not None:
        _need("residual", residual, dev, x.dtype, T, d)
    if out is None:
        kinds = _norm_outputs(x.dtype, T, d, n)
        want = {"y": want_y, "h": residual is not None if want_h is None else want_h,
                "rstd": want_rstd, "q": quantize, "scale": quantize}
        out = {k: torch.empty(*v[1:], dtype=v[0], device=dev) for k, v in kinds.items()
               if want[k]}
    else:
        for k, t in out.items():
            if k == "y" or k == "h":
                _need(k, t, dev, x.dtype, T, d)
            elif k == "q":
                _need(k, t, dev, torch.int8, T, d)
            elif k == "scale":
                _need(k, t, dev, torch.float32, T, n)
            elif k == "rstd":
                _need(k, t, dev, torch.float32, T)
            else:
                raise ValueError(f"out has no place for {k!r}")
        if ("q" in out) != ("scale" in out):
            raise ValueError("q and scale come together")
    if "y" not in out and "q" not in out:
        raise ValueError("neither y nor its 8-bit form is asked for")
    _launch(dev, lib().dora_rmsnorm, _at(x), _at(residual), _at(w), float(eps), T, d, dt, group,
            _at(out.get("y")), _at(out.get("h")), _at(out.get("rstd")), _at(out.get("q")),
            _at(out.get("scale")))
    return out


def dora_rmsnorm_backward_workspace(T, d, dtype):
    return lib().dora_rmsnorm_backward_workspace(T, d, dtype)


def dora_rmsnorm_backward(dy, h, w, rstd, dres=None, ws=None, out=None):
    """Gradients of dora_rmsnorm from the h and rstd it returned: dict(dx, dw), dx [T, d] the
    gradient of x (and of the residual), dw fp32 [d].  dres: the gradient that reaches h along
    the residual stream, added to dx (out["dx"] may be dres)."""
    dev = _dev(dy)
    T, d = _rows("dy", dy)
    dt = _dt(dy)
    _need("dy", dy, dev, dy.dtype, T, d)
    _need("h", h, dev, dy.dtype, T, d)
    _need("w", w, dev, dy.dtype, d)
    _need("rstd", rstd, dev, torch.float32, T)
    if dres is not None:
        _need("dres", dres, dev, dy.dtype, T, d)
    if out is None:
        out = {"dx": torch.empty_like(dy), "dw": torch.empty(d, dtype=torch.float32, device=dev)}
    else:
        _need("dx", out["dx"], dev, dy.dtype, T, d)
        _need("dw", out["dw"], dev, torch.float32, d)
    if _need_ws(ws, dev) is None:
        ws = _ws(dora_rmsnorm_backward_workspace(T, d, dt), dev)
    _launch(dev, lib().dora_rmsnorm_backward, _at(dy), _at(h), _at(w), _at(rstd), _at(dres),
            T, d, dt, _at(out["dx"]), _at(out["dw"]), _at(ws), ws.numel())
    return out


def dora_quantize_rows(x, group=0, q=None, scale=None):
    """Rows of x [T, d] as int8 values and fp32 scales [T, groups]: q = rint(x / scale), scale =
    max|x| / 127 over the row (group 0) or over each `group` columns.  Returns (q, scale)."""
    dev = _dev(x)
    T, d = _rows("x", x)
    dt = _dt(x)
    n = _groups(d, group)
    _need("x", x, dev, x.dtype, T, d)
    q = torch.empty(T, d, dtype=torch.int8, device=dev) if q is None \
        else _need("q", q, dev, torch.int8, T, d)
    scale = torch.empty(T, n, dtype=torch.float32, device=dev) if scale is None \
        else _need("scale", scale, dev, torch.float32, T, n)
    _launch(dev, lib().dora_quantize_rows, _at(x), T, d, dt, group, _at(q), _at(scale))
    return q, scale


def dora_dequantize_rows(q, scale, group=0, dtype=torch.bfloat16, out=None):
    """The values int8 rows stand for, q scale, in `dtype` (or in out's)."""
    dev = _dev(q)
    T, d = _rows("q", q)
    _need("q", q, dev, torch.int8, T, d)
    _need("scale", scale, dev, torch.float32, T, _groups(d, group))
    out = torch.empty(T, d, dtype=dtype, device=dev) if out is None \
        else _need("out", out, dev, out.dtype, T, d)
    _launch(dev, lib().dora_dequantize_rows, _at(q), _at(scale), T, d, _dt(out), group,
            _at(out))
    return out


def dora_linear_quantized_workspace(T, d_in, d_out, dtype):
    return lib().dora_linear_quantized_workspace(T, d_in, d_out, dtype)


def dora_linear_quantized(xq, xs, wq, wscale, dtype=torch.bfloat16, y=None, ws=None):
    """y = (xs xq) (wscale wq)^T: the linear layer of a merged weight in int8, one scale per
    token (xs [T, 1]) and one per output channel (wscale [d_out, 1]), as dora_rmsnorm and
    dora_quantize_rows give them with group 0.  int32 sums; y [T, d_out] in `dtype` (or y's)."""
    dev = _dev(xq)
    T, d_in = _rows("xq", xq)
    d_out = _rows("wq", wq)[0]
    _need("xq", xq, dev, torch.int8, T, d_in)
    _need("wq", wq, dev, torch.int8, d_out, d_in)
    _need("xs", xs, dev, torch.float32, T, 1)
    _need("wscale", wscale, dev, torch.float32, d_out, 1)
    y = torch.empty(T, d_out, dtype=dtype, device=dev) if y is None \
        else _need("y", y, dev, y.dtype, T, d_out)
    dt = _dt(y)
    if _need_ws(ws, dev) is None:
        need = dora_linear_quantized_workspace(T, d_in, d_out, dt)
        ws = _ws(need, dev) if need > 0 else None
    _launch(dev, lib().dora_linear_quantized, _at(xq), _at(xs), _at(wq), _at(wscale), T, d_in,
            d_out, dt, _at(y), _at(ws), 0 if ws is None else ws.numel())
    return y


def dora_backward_checkpoint_workspace(T, d_in, d_out, r, dtype, through_norm=False):
    return lib().dora_backward_checkpoint_workspace(T, d_in, d_out, r, dtype, int(through_norm))


def dora_backward_checkpoint(dy, xq, xs, W, A, B, m, n, s, P, yq, ys, group=0, through_norm=False,
                             U=None, ws=None, out=None):
    """dora_backward (or, with through_norm, dora_backward_through_norm) from x and y kept in 8
    bits by dora_quantize_rows (or dora_rmsnorm) with this `group`; returns
    dict(dx, dA, dB, dm)."""
    dev = _dev(dy)
    T, d_out = _rows("dy", dy)
    r, d_in = _rows("A", A)
    dt = _dt(dy)
    f32 = torch.float32
    for name, t, kind, shape in (
            ("dy", dy, dy.dtype, (T, d_out)), ("xq", xq, torch.int8, (T, d_in)),
            ("xs", xs, f32, (T, _groups(d_in, group))), ("W", W, dy.dtype, (d_out, d_in)),
            ("A", A, dy.dtype, (r, d_in)), ("B", B, dy.dtype, (d_out, r)), ("m", m, f32, (d_out,)),
            ("n", n, f32, (d_out,)), ("P", P, dy.dtype, (T, r)),
            ("yq", yq, torch.int8, (T, d_out)), ("ys", ys, f32, (T, _groups(d_out, group)))):
        _need(name, t, dev, kind, *shape)
    if U is not None:
        if not through_norm:
            raise ValueError("U is used by the backward through the norm only")
        _need("U", U, dev, f32, d_out, r)
    kinds = {"dx": (dy.dtype, T, d_in), "dA": (dy.dtype, r, d_in), "dB": (dy.dtype, d_out, r),
             "dm": (f32, d_out)}
    if out is None:
        out = {k: torch.empty(*v[1:], dtype=v[0], device=dev) for k, v in kinds.items()}
    else:
        for k, v in kinds.items():
            _need(k, out[k], dev, *v)
    if _need_ws(ws, dev) is None:
        ws = _ws(dora_backward_checkpoint_workspace(T, d_in, d_out, r, dt, through_norm), dev)
    _launch(dev, lib().dora_backward_checkpoint, _at(dy), _at(xq), _at(xs), _at(W), _at(A),
            _at(B), _at(m), _at(n), float(s), _at(P), _at(yq), _at(ys), group, _at(U),
            int(through_norm), T, d_in, d_out, r, dt, _at(out["dx"]), _at(out["dA"]),
            _at(out["dB"]), _at(out["dm"]), _at(ws), ws.numel())
    return out
