"""Thin ctypes binding of libdora.so (include/dora.h), same names as the C ABI.

Argument marshalling only: tensors are passed as device pointers, outputs and
the workspace are allocated with torch (device memory plumbing), and every
step of the computation runs in the library's HIP kernels.  There is no CPU
or PyTorch fallback: if the library is missing or cannot be loaded, every
call raises.
"""
import ctypes
import operator
import os
import struct

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
           "dora_backward_checkpoint", "dora_block_norm", "dora_block_norm_backward_workspace",
           "dora_block_norm_backward", "dora_quantize_fourbit", "dora_dequantize_fourbit",
           "dora_linear_fourbit_workspace", "dora_linear_fourbit", "dora_orthogonalize_workspace",
           "dora_orthogonalize", "dora_muon_workspace", "dora_muon")

_lib = None


class DoraModule(ctypes.Structure):
    """struct dora_module of include/dora.h."""
    _fields_ = [("W", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("s", ctypes.c_float), ("d_out", ctypes.c_int64),
                ("d_in", ctypes.c_int64), ("r", ctypes.c_int64)]


class DoraUpdate(ctypes.Structure):
    """struct dora_update of include/dora.h."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("momentum", ctypes.c_void_p), ("param_out", ctypes.c_void_p),
                ("momentum_out", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("lr", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("scale", ctypes.c_float)]


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
        L.dora_block_norm.restype = c_int
        L.dora_block_norm.argtypes = [p, p, p, p, i64, p, f, f, f, i64, i64, c_int, p, p, p, p, p]
        L.dora_block_norm_backward_workspace.restype = sz
        L.dora_block_norm_backward_workspace.argtypes = [i64, i64, i64, c_int]
        L.dora_block_norm_backward.restype = c_int
        L.dora_block_norm_backward.argtypes = [p, p, p, p, p, p, i64, p, p, p, f, f, i64, i64,
                                               c_int, p, p, p, p, p, p, sz, p]
        L.dora_quantize_fourbit.restype = c_int
        L.dora_quantize_fourbit.argtypes = [p, i64, i64, c_int, i64, p, p, p]
        L.dora_dequantize_fourbit.restype = c_int
        L.dora_dequantize_fourbit.argtypes = [p, p, i64, i64, c_int, i64, p, p]
        L.dora_linear_fourbit_workspace.restype = sz
        L.dora_linear_fourbit_workspace.argtypes = [i64, i64, i64, c_int]
        L.dora_linear_fourbit.restype = c_int
        L.dora_linear_fourbit.argtypes = [p, p, p, i64, i64, i64, i64, c_int, p, p, sz, p]
        up, fp = p, ctypes.POINTER(f)  # (structures, or their bytes)
        L.dora_orthogonalize_workspace.restype = sz
        L.dora_orthogonalize_workspace.argtypes = [i64, i64, c_int]
        L.dora_orthogonalize.restype = c_int
        L.dora_orthogonalize.argtypes = [p, i64, i64, c_int, c_int, fp, f, p, p, sz, p]
        L.dora_muon_workspace.restype = sz
        L.dora_muon_workspace.argtypes = [up, c_int, c_int]
        L.dora_muon.restype = c_int
        L.dora_muon.argtypes = [up, c_int, c_int, f, c_int, c_int, fp, f, p, sz, p]
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


# ------------------------------------------- norms on both sides of a residual
def _gate_rows(gate, T, d):
    """Tokens that share a row of the gate (0 without one): gate [d] or [G, d], G dividing T."""
    if gate is None:
        return 0
    if gate.dim() == 1:
        return max(T, 1)
    G = gate.shape[0] if gate.dim() == 2 else 0
    if T == 0 and G == 1:
        return 1
    if G < 1 or T < G or T % G:
        raise ValueError(f"gate of shape {tuple(gate.shape)} for {T} tokens: [d], or [G, d] with "
                         "G dividing them")
    return T // G


def _block_inputs(x, w_pre, w_post, gate):
    dev = _dev(x)
    T, d = _rows("x", x)
    rows = _gate_rows(gate, T, d)
    _need("x", x, dev, x.dtype, T, d)
    _need("w_pre", w_pre, dev, x.dtype, d)
    if w_post is not None:
        _need("w_post", w_post, dev, x.dtype, d)
    if gate is not None:
        _need("gate", gate, dev, x.dtype, *gate.shape[:-1], d)
    return dev, T, d, _dt(x), rows


def dora_block_norm(x, residual, w_pre, w_post=None, gate=None, residual_scale=1.0,
                    branch_scale=1.0, eps=1e-6, want_rstd=False, out=None):
    """The norms on both sides of a residual addition: u = w_post x / rms(x) (x without w_post),
    h = residual_scale residual + branch_scale gate u (rounded to the element type), y = w_pre h /
    rms(h).  gate: [d], or [G, d] for sequences of T / G tokens each (G = T: one a token).  Returns
    a dict of "h", "y" and, with want_rstd, "rstd_pre" and (with w_post) "rstd_post" (fp32 [T], for
    the backward).  out: a dict of preallocated outputs, h and y at least; then those are what is
    asked for.  out["h"] may be residual, out["y"] may be x."""
    dev, T, d, dt, rows = _block_inputs(x, w_pre, w_post, gate)
    _need("residual", residual, dev, x.dtype, T, d)
    if out is None:
        out = {"h": torch.empty_like(x), "y": torch.empty_like(x)}
        if want_rstd:
            out["rstd_pre"] = torch.empty(T, dtype=torch.float32, device=dev)
            if w_post is not None:
                out["rstd_post"] = torch.empty(T, dtype=torch.float32, device=dev)
    else:
        if "h" not in out or "y" not in out:
            raise ValueError("out needs h and y")
        for k, t in out.items():
            if k in ("h", "y"):
                _need(k, t, dev, x.dtype, T, d)
            elif k in ("rstd_pre", "rstd_post"):
                _need(k, t, dev, torch.float32, T)
            else:
                raise ValueError(f"out has no place for {k!r}")
    _launch(dev, lib().dora_block_norm, _at(x), _at(residual), _at(w_post), _at(gate), rows,
            _at(w_pre), float(residual_scale), float(branch_scale), float(eps), T, d, dt,
            _at(out["h"]), _at(out["y"]), _at(out.get("rstd_post")), _at(out.get("rstd_pre")))
    return out


def dora_block_norm_backward_workspace(T, d, gate_rows, dtype):
    return lib().dora_block_norm_backward_workspace(T, d, gate_rows, dtype)


def dora_block_norm_backward(dy, x, h, w_pre, rstd_pre, w_post=None, rstd_post=None, gate=None,
                             dh=None, residual_scale=1.0, branch_scale=1.0, ws=None, out=None):
    """Gradients of dora_block_norm from its x, h and factors.  dh: the gradient that reaches h
    along the residual stream.  Returns dict(dx, dresidual, dw_pre) with "dw_post" and "dgate"
    where there is a w_post and a gate; dw are fp32, dgate has the gate's shape and type.  out: a
    dict of preallocated outputs, dx and dresidual at least (out["dresidual"] may be dh)."""
    dev, T, d, dt, rows = _block_inputs(x, w_pre, w_post, gate)
    f32 = torch.float32
    _need("dy", dy, dev, x.dtype, T, d)
    _need("h", h, dev, x.dtype, T, d)
    _need("rstd_pre", rstd_pre, dev, f32, T)
    if w_post is not None:
        if rstd_post is None:
            raise ValueError("w_post comes with rstd_post")
        _need("rstd_post", rstd_post, dev, f32, T)
    if dh is not None:
        _need("dh", dh, dev, x.dtype, T, d)
    kinds = {"dx": (x.dtype, T, d), "dresidual": (x.dtype, T, d), "dw_pre": (f32, d)}
    if w_post is not None:
        kinds["dw_post"] = (f32, d)
    if gate is not None:
        kinds["dgate"] = (x.dtype, *gate.shape)
    if out is None:
        out = {k: torch.empty(*v[1:], dtype=v[0], device=dev) for k, v in kinds.items()}
    else:
        if "dx" not in out or "dresidual" not in out:
            raise ValueError("out needs dx and dresidual")
        for k, t in out.items():
            if k not in kinds:
                raise ValueError(f"out has no place for {k!r}")
            _need(k, t, dev, *kinds[k])
    if _need_ws(ws, dev) is None:
        need = dora_block_norm_backward_workspace(T, d, rows, dt)
        ws = _ws(need, dev) if need > 0 else None
    _launch(dev, lib().dora_block_norm_backward, _at(dy), _at(dh), _at(x), _at(h), _at(w_post),
            _at(gate), rows, _at(w_pre), _at(rstd_post) if w_post is not None else None,
            _at(rstd_pre), float(residual_scale), float(branch_scale), T, d, dt, _at(out["dx"]),
            _at(out["dresidual"]), _at(out.get("dgate")), _at(out.get("dw_post")),
            _at(out.get("dw_pre")), _at(ws), 0 if ws is None else ws.numel())
    return out


# ------------------------------------------------------------- 4-bit weights
def _fourbit_groups(d, group):
    if group not in (32, 64, 128, 256, 512):
        raise ValueError(f"group {group} is not a power of two from 32 to 512")
    return -(-d // group)


def dora_quantize_fourbit(x, group=128, codes=None, scale=None):
    """Rows of x [T, d] as e2m1 codes (uint8 [T, groups * group / 2], two a byte) and bf16 scales
    [T, groups], one for each `group` columns: max|x| / 6 at six significant bits, so that every
    restored value is a bf16 number.  Returns (codes, scale)."""
    dev = _dev(x)
    T, d = _rows("x", x)
    dt = _dt(x)
    n = _fourbit_groups(d, group)
    _need("x", x, dev, x.dtype, T, d)
    codes = torch.empty(T, n * group // 2, dtype=torch.uint8, device=dev) if codes is None \
        else _need("codes", codes, dev, torch.uint8, T, n * group // 2)
    scale = torch.empty(T, n, dtype=torch.bfloat16, device=dev) if scale is None \
        else _need("scale", scale, dev, torch.bfloat16, T, n)
    _launch(dev, lib().dora_quantize_fourbit, _at(x), T, d, dt, group, _at(codes), _at(scale))
    return codes, scale


def dora_dequantize_fourbit(codes, scale, d, group=128, dtype=torch.bfloat16, out=None):
    """The values [T, d] that 4-bit rows stand for, in `dtype` (or in out's)."""
    dev = _dev(codes)
    T = _rows("codes", codes)[0]
    n = _fourbit_groups(d, group)
    _need("codes", codes, dev, torch.uint8, T, n * group // 2)
    _need("scale", scale, dev, torch.bfloat16, T, n)
    out = torch.empty(T, d, dtype=dtype, device=dev) if out is None \
        else _need("out", out, dev, out.dtype, T, d)
    _launch(dev, lib().dora_dequantize_fourbit, _at(codes), _at(scale), T, d, _dt(out), group,
            _at(out))
    return out


def dora_linear_fourbit_workspace(T, d_in, d_out, dtype):
    return lib().dora_linear_fourbit_workspace(T, d_in, d_out, dtype)


def dora_linear_fourbit(x, codes, scale, group=128, y=None, ws=None):
    """y = x W^T for a weight W [d_out, d_in] held as dora_quantize_fourbit gives it (codes, scale,
    with this group); x [T, d_in], y [T, d_out] in x's type."""
    dev = _dev(x)
    T, d_in = _rows("x", x)
    d_out = _rows("codes", codes)[0]
    dt = _dt(x)
    n = _fourbit_groups(d_in, group)
    _need("x", x, dev, x.dtype, T, d_in)
    _need("codes", codes, dev, torch.uint8, d_out, n * group // 2)
    _need("scale", scale, dev, torch.bfloat16, d_out, n)
    y = torch.empty(T, d_out, dtype=x.dtype, device=dev) if y is None \
        else _need("y", y, dev, x.dtype, T, d_out)
    if _need_ws(ws, dev) is None:
        need = dora_linear_fourbit_workspace(T, d_in, d_out, dt)
        ws = _ws(need, dev) if need > 0 else None
    _launch(dev, lib().dora_linear_fourbit, _at(x), _at(codes), _at(scale), group, T, d_in, d_out,
            dt, _at(y), _at(ws), 0 if ws is None else ws.numel())
    return y


# ------------------------------------------------- orthogonalised updates
QUINTIC = (3.4445, -4.7750, 2.0315)


def _coefficients(c):
    a, b, d = (float(v) for v in c)
    return (ctypes.c_float * 3)(a, b, d)


def dora_orthogonalize_workspace(rows, cols, dtype):
    return lib().dora_orthogonalize_workspace(rows, cols, dtype)


def dora_orthogonalize(U, steps=5, coefficients=QUINTIC, eps=1e-7, out=None, ws=None):
    """Newton-Schulz steps X <- a X + b (X X^T) X + c (X X^T)^2 X from X = U / (|U| + eps), U
    [rows, cols]: the orthogonal matrix near U, its singular values brought close to one.  out
    may be U."""
    dev = _dev(U)
    rows, cols = _rows("U", U)
    dt = _dt(U)
    _need("U", U, dev, U.dtype, rows, cols)
    out = torch.empty_like(U) if out is None else _need("out", out, dev, U.dtype, rows, cols)
    if _need_ws(ws, dev) is None:
        ws = _ws(dora_orthogonalize_workspace(rows, cols, dt), dev)
    _launch(dev, lib().dora_orthogonalize, _at(U), rows, cols, dt, int(steps),
            _coefficients(coefficients), float(eps), _at(out), _at(ws), ws.numel())
    return out


# DoraUpdate's fields (a fifth of the time that ctypes takes to fill the structures).
_UPDATE = struct.Struct("5Q2q3f4x")
assert _UPDATE.size == ctypes.sizeof(DoraUpdate)
_shape_of, _dtype_of = operator.attrgetter("shape"), operator.attrgetter("dtype")


def dora_muon_workspace(params):
    """Bytes for dora_muon on these parameters (their shapes and type)."""
    if not params:
        return 0
    arr = b"".join([_UPDATE.pack(0, 0, 0, 0, 0, *_rows("a parameter", q), 0, 0, 0) for q in params])
    return lib().dora_muon_workspace(arr, len(params), _dt(params[0]))


def dora_muon(params, grads, momenta, lr, mu=0.95, weight_decay=0.0, scales=None, nesterov=True,
              steps=5, coefficients=QUINTIC, eps=1e-7, params_out=None, momenta_out=None, ws=None):
    """One step of the Muon optimiser on a list of matrices (for instance every adapter's A and
    B with the gradients of dora_backward), in few launches: momentum M <- mu M + grad (fp32),
    param <- param - lr (weight_decay param + scale O) with O the orthogonalised grad + mu M
    (nesterov; else M).  scales: one number a matrix (default 1).  In place unless params_out /
    momenta_out are given; returns (params_out, momenta_out)."""
    params_out = params if params_out is None else params_out
    momenta_out = momenta if momenta_out is None else momenta_out
    n = len(params)
    scales = [1.0] * n if scales is None else scales
    for name, ts in (("grads", grads), ("momenta", momenta), ("scales", scales),
                     ("params_out", params_out), ("momenta_out", momenta_out)):
        if len(ts) != n:
            raise ValueError(f"{name} has {len(ts)} entries for {n} params")
    if n == 0:
        return params_out, momenta_out
    dev = _dev(params[0])
    kind, dt = params[0].dtype, _dt(params[0])
    lists = {"params": (params, kind), "grads": (grads, kind), "momenta": (momenta, torch.float32)}
    if params_out is not params:
        lists["params_out"] = params_out, kind
    if momenta_out is not momenta:
        lists["momenta_out"] = momenta_out, torch.float32
    shapes = list(map(_shape_of, params))
    if set(map(len, shapes)) != {2}:
        raise ValueError("a parameter is not a matrix")
    at = {}
    for name, (ts, t) in lists.items():
        # (whole lists at a time: half of a step's host time are these checks)
        if not (list(map(_shape_of, ts)) == shapes and set(map(_dtype_of, ts)) == {t}
                and set(map(torch.Tensor.get_device, ts)) == {dev.index}
                and all(map(torch.Tensor.is_contiguous, ts))):
            for k, (x, shape) in enumerate(zip(ts, shapes)):
                _need(f"{name}[{k}]", x, dev, t, *shape)
        at[name] = list(map(torch.Tensor.data_ptr, ts))
    lr, weight_decay = float(lr), float(weight_decay)
    arr = b"".join([
        _UPDATE.pack(p, g, m, po, mo, rows, cols, lr, weight_decay, float(scale))
        for p, g, m, po, mo, (rows, cols), scale
        in zip(at["params"], at["grads"], at["momenta"], at.get("params_out", at["params"]),
               at.get("momenta_out", at["momenta"]), shapes, scales)])
    if _need_ws(ws, dev) is None:
        ws = _ws(lib().dora_muon_workspace(arr, n, dt), dev)
    _launch(dev, lib().dora_muon, arr, n, dt, float(mu), int(bool(nesterov)), int(steps),
            _coefficients(coefficients), float(eps), _at(ws), ws.numel())
    return params_out, momenta_out
