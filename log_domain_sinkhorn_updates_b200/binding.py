"""ctypes binding of the C ABI declared in ``include/flashsinkhorn.h``.

Argument marshalling only: every step of the computation runs in the CUDA
library.  Device arrays are torch CUDA tensors (their data pointers are
passed through); host arrays are numpy arrays.  If the shared library is
missing the import fails loudly -- there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libflashsinkhorn.so")

FS_OK, FS_ERR_INVALID_ARG, FS_ERR_CUDA, FS_ERR_UNSUPPORTED, FS_ERR_NONFINITE, FS_ERR_TIMEOUT, FS_ERR_OOM = range(7)
FS_F32, FS_BF16 = 0, 1
PRECISIONS = {"auto": 0, "bf16": 1, "tf32": 2, "3xtf32": 3, "3xf16": 4, "f32_simt": 5}
PRECISION_NAMES = {v: k for k, v in PRECISIONS.items()}
SCHEDULES = {"alternating": 0, "symmetric": 1}
COSTS = {"sqeuclidean": 0, "cosine": 1}
STATUS_NAMES = {0: "FS_OK", 1: "FS_ERR_INVALID_ARG", 2: "FS_ERR_CUDA", 3: "FS_ERR_UNSUPPORTED",
                4: "FS_ERR_NONFINITE", 5: "FS_ERR_TIMEOUT", 6: "FS_ERR_OOM"}

EXPORTS = ["fs_create", "fs_update_f", "fs_update_g", "fs_solve", "fs_marginal_err", "fs_ot_cost",
           "fs_sync", "fs_get_info", "fs_destroy", "fs_last_error", "fs_solve_host", "fs_kernel_launches",
           "fs_update_f_noalloc", "fs_transport_apply", "fs_barycentric_map", "fs_grad_x",
           "fs_transport_apply_t", "fs_grad_y", "fs_hvp_x", "fs_selftest_wait", "fs_cross_attn", "fs_cross_attn_grad",
           "fs_cross_attn_workspace", "fs_cross_entropy", "fs_cross_entropy_grad", "fs_cross_entropy_workspace",
           "fs_check", "fs_selftest_check"]


class FsDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n", ctypes.c_int), ("m", ctypes.c_int), ("d", ctypes.c_int),
                ("dtype", ctypes.c_int), ("prec", ctypes.c_int), ("eps", ctypes.c_float), ("cost", ctypes.c_int)]


class FsInfo(ctypes.Structure):
    _fields_ = [("prec", ctypes.c_int), ("d_pad", ctypes.c_int), ("row_bytes", ctypes.c_int),
                ("swizzle_bytes", ctypes.c_int), ("stages", ctypes.c_int), ("block_rows", ctypes.c_int),
                ("block_cols", ctypes.c_int), ("splits_f", ctypes.c_int), ("splits_g", ctypes.c_int),
                ("launches_update", ctypes.c_int), ("launches_solve_iter", ctypes.c_int),
                ("device_bytes", ctypes.c_size_t), ("cta_pair", ctypes.c_int), ("last_apply_path", ctypes.c_int),
                ("last_solve_graph", ctypes.c_int), ("last_measure_fused", ctypes.c_int),
                ("last_hvp_fused", ctypes.c_int), ("last_apply_parts", ctypes.c_int)]

    def as_dict(self):
        d = {k: getattr(self, k) for k, _ in self._fields_}
        d["prec"] = PRECISION_NAMES.get(d["prec"], d["prec"])
        d["last_apply_path"] = {0: None, 1: "tc", 2: "simt", 3: "tc_pair", 4: "tc_q2", 5: "lse_vec", 6: "tc_2s"}.get(d["last_apply_path"],
                                                                               d["last_apply_path"])
        d["last_solve_graph"] = {0: None, 1: "graph", 2: "direct"}.get(d["last_solve_graph"], d["last_solve_graph"])
        return d


class FsView(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_longlong), ("token", ctypes.c_longlong), ("head", ctypes.c_longlong)]


class FsAttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n", ctypes.c_int), ("m", ctypes.c_int), ("heads", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("d", ctypes.c_int), ("dv", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("q", FsView), ("k", FsView), ("v", FsView), ("out", FsView),
                ("dout", FsView), ("dq", FsView), ("dk", FsView), ("dvw", FsView)]


class FsXentDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("v", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("ldx", ctypes.c_longlong), ("ldw", ctypes.c_longlong),
                ("lddx", ctypes.c_longlong), ("lddw", ctypes.c_longlong), ("ignore_index", ctypes.c_longlong)]


class FsError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_lib = None
_torch = None  # the torch module, bound when an operator without a handle is first called


def lib():
    """The loaded C library (ctypes.CDLL); raises ImportError if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"CUDA extension missing: {LIB_PATH} (run log_domain_sinkhorn_updates_b200/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        vp, dp, fp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_double), ctypes.c_void_p
        L.fs_create.argtypes = [ctypes.POINTER(FsDesc), vp, vp, vp, vp, vp, ctypes.POINTER(ctypes.c_void_p)]
        L.fs_update_f.argtypes = [vp, fp, fp]
        L.fs_update_g.argtypes = [vp, fp, fp]
        L.fs_solve.argtypes = [vp, fp, fp, ctypes.c_int, ctypes.c_int]
        L.fs_marginal_err.argtypes = [vp, fp, fp, dp, dp]
        L.fs_ot_cost.argtypes = [vp, fp, fp, dp, dp]
        L.fs_sync.argtypes = [vp]
        L.fs_get_info.argtypes = [vp, ctypes.POINTER(FsInfo)]
        L.fs_destroy.argtypes = [vp]
        L.fs_last_error.argtypes = [vp]
        L.fs_last_error.restype = ctypes.c_char_p
        L.fs_solve_host.argtypes = [ctypes.POINTER(FsDesc), vp, vp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                    dp, dp, dp, dp, vp]
        L.fs_update_f_noalloc.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float, vp, vp, vp, vp,
                                          vp, vp]
        L.fs_transport_apply.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp]
        L.fs_barycentric_map.argtypes = [vp, vp, vp, vp, vp]
        L.fs_grad_x.argtypes = [vp, vp, vp, vp, vp, vp]
        L.fs_transport_apply_t.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp]
        L.fs_grad_y.argtypes = [vp, vp, vp, vp, vp, vp]
        L.fs_hvp_x.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_double, vp]
        L.fs_selftest_wait.argtypes = [vp, ctypes.c_int]
        L.fs_kernel_launches.argtypes = []
        L.fs_kernel_launches.restype = ctypes.c_ulonglong
        szt, ad, xd = ctypes.c_size_t, ctypes.POINTER(FsAttnDesc), ctypes.POINTER(FsXentDesc)
        L.fs_cross_attn_workspace.argtypes = [ad, ctypes.c_int]
        L.fs_cross_attn.argtypes = [ad] + [vp] * 8 + [szt, vp]
        L.fs_cross_attn_grad.argtypes = [ad] + [vp] * 12 + [szt, vp]
        L.fs_cross_entropy_workspace.argtypes = [xd, vp, vp, ctypes.c_int]
        L.fs_cross_entropy.argtypes = [xd] + [vp] * 6 + [szt, vp]
        L.fs_cross_entropy_grad.argtypes = [xd] + [vp] * 9 + [szt, vp]
        L.fs_check.argtypes = [vp]
        L.fs_selftest_check.argtypes = [ctypes.c_int, vp]
        L.fs_cross_attn_workspace.restype = L.fs_cross_entropy_workspace.restype = szt
        for name in EXPORTS:
            if name not in ("fs_last_error", "fs_kernel_launches", "fs_cross_attn_workspace",
                            "fs_cross_entropy_workspace"):
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status, handle=None):
    if status != FS_OK:
        msg = lib().fs_last_error(handle)
        raise FsError(status, msg.decode() if msg else "")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _f32(t):
    import torch
    if t is not None and t.dtype != torch.float32:
        raise ValueError("potentials and weights must be float32")
    return _ptr(t)


def _stream_ptr(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class Handle:
    """Owns an ``fs_handle*``; freed by ``fs_destroy`` (or when collected)."""

    def __init__(self, ptr, desc, stream):
        self.ptr = ptr
        self.desc = desc
        self.stream = stream

    @property
    def batch(self):
        return self.desc.batch

    @property
    def n(self):
        return self.desc.n

    @property
    def m(self):
        return self.desc.m

    def __del__(self):
        try:
            fs_destroy(self)
        except Exception:
            pass


def fs_create(X, Y, a=None, b=None, eps=0.1, prec="auto", stream=None, cost="sqeuclidean") -> Handle:
    """X [batch, n, d] / [n, d], Y likewise (CUDA float32 or bfloat16), a [batch, n], b [batch, m] or None.
    cost: "sqeuclidean" (C = |x - y|^2) or "cosine" (C = 1 - cos(x, y))."""
    import torch
    if X.dim() == 2:
        X, Y = X.unsqueeze(0), Y.unsqueeze(0)
        a = None if a is None else a.reshape(1, -1)
        b = None if b is None else b.reshape(1, -1)
    if X.dtype != Y.dtype:
        raise ValueError("X and Y must share a dtype")
    dtype = {torch.float32: FS_F32, torch.bfloat16: FS_BF16}.get(X.dtype)
    if dtype is None:
        raise ValueError("X, Y must be float32 or bfloat16")
    B, n, d = X.shape
    m = Y.shape[1]
    if Y.shape[0] != B or Y.shape[2] != d:
        raise ValueError("X and Y shapes disagree")
    desc = FsDesc(B, n, m, d, dtype, PRECISIONS[prec] if isinstance(prec, str) else int(prec), float(eps),
                  COSTS[cost])
    out = ctypes.c_void_p()
    st = lib().fs_create(ctypes.byref(desc), _ptr(X), _ptr(Y), _f32(a), _f32(b), _stream_ptr(stream),
                         ctypes.byref(out))
    _check(st)
    return Handle(out, desc, stream)


def fs_update_f(h: Handle, g, f):
    _check(lib().fs_update_f(h.ptr, _f32(g), _f32(f)), h.ptr)


def fs_update_g(h: Handle, f, g):
    _check(lib().fs_update_g(h.ptr, _f32(f), _f32(g)), h.ptr)


def fs_solve(h: Handle, f, g, iters, schedule="alternating"):
    _check(lib().fs_solve(h.ptr, _f32(f), _f32(g), int(iters), SCHEDULES[schedule]), h.ptr)


def fs_marginal_err(h: Handle, f, g, row=True, col=True):
    er = np.zeros(h.batch)
    ec = np.zeros(h.batch)
    dp = ctypes.POINTER(ctypes.c_double)
    _check(lib().fs_marginal_err(h.ptr, _f32(f), _f32(g), er.ctypes.data_as(dp) if row else None,
                                 ec.ctypes.data_as(dp) if col else None), h.ptr)
    return (er if row else None), (ec if col else None)


def fs_ot_cost(h: Handle, f, g):
    dual = np.zeros(h.batch)
    primal = np.zeros(h.batch)
    dp = ctypes.POINTER(ctypes.c_double)
    _check(lib().fs_ot_cost(h.ptr, _f32(f), _f32(g), dual.ctypes.data_as(dp), primal.ctypes.data_as(dp)), h.ptr)
    return dual, primal


def fs_sync(h: Handle):
    _check(lib().fs_sync(h.ptr), h.ptr)


def fs_get_info(h: Handle) -> dict:
    info = FsInfo()
    _check(lib().fs_get_info(h.ptr, ctypes.byref(info)), h.ptr)
    return info.as_dict()


def fs_destroy(h: Handle):
    if h is not None and h.ptr:
        p, h.ptr = h.ptr, None
        lib().fs_destroy(p)


def fs_last_error(h: Handle = None) -> str:
    msg = lib().fs_last_error(h.ptr if h is not None else None)
    return msg.decode() if msg else ""


def fs_update_f_noalloc(X, Y, b, g, f, eps, stream=None):
    """One f-update through the allocation-free entry point: X [n, d], Y [m, d] float32 CUDA
    tensors, b [m] or None (uniform), g [m], output f [n].  Asynchronous on the stream."""
    if X.dim() != 2 or Y.dim() != 2 or X.shape[1] != Y.shape[1]:
        raise ValueError("X [n, d] and Y [m, d] expected")
    n, d = X.shape
    m = Y.shape[0]
    _check(lib().fs_update_f_noalloc(n, m, d, float(eps), _f32(X), _f32(Y), _f32(b), _f32(g), _f32(f),
                                     _stream_ptr(stream)))


def fs_kernel_launches() -> int:
    """Kernels the library has launched in this process (host-side count)."""
    return int(lib().fs_kernel_launches())


def fs_solve_host(X, Y, a, b, g0, eps, iters, dtype="f32", prec="auto", schedule="alternating", stream=None,
                  measure=True, out=None, cost="sqeuclidean"):
    """End-to-end solve from host (numpy) arrays through ``fs_solve_host``.

    X, Y: [batch, n|m, d] float32 (or uint16 bfloat16 bits with dtype="bf16"),
    a, b: float32 or None (uniform), g0: [batch, m] float32 initial g.
    Returns (f, g, err_row, err_col, dual, primal) as numpy arrays.
    """
    X = np.ascontiguousarray(X)
    Y = np.ascontiguousarray(Y)
    if X.ndim == 2:
        X, Y = X[None], Y[None]
    B, n, d = X.shape
    m = Y.shape[1]
    desc = FsDesc(B, n, m, d, FS_BF16 if dtype == "bf16" else FS_F32, PRECISIONS[prec], float(eps), COSTS[cost])
    if out is None:
        f = np.empty((B, n), np.float32)
        g = np.array(g0, dtype=np.float32).reshape(B, m)
    else:
        f, g = out
        g[...] = np.asarray(g0, dtype=np.float32).reshape(B, m)
    res = [np.zeros(B) for _ in range(4)]
    dp = ctypes.POINTER(ctypes.c_double)
    vp = lambda arr: None if arr is None else ctypes.c_void_p(arr.ctypes.data)  # noqa: E731
    rp = [r.ctypes.data_as(dp) if measure else None for r in res]
    st = lib().fs_solve_host(ctypes.byref(desc), vp(X), vp(Y),
                             vp(None if a is None else np.ascontiguousarray(a, np.float32)),
                             vp(None if b is None else np.ascontiguousarray(b, np.float32)),
                             vp(f), vp(g), int(iters), SCHEDULES[schedule], *rp,
                             None if stream is None else ctypes.c_void_p(stream.cuda_stream))
    _check(st)
    return (f, g, *res)


def fs_transport_apply(h: Handle, f, g, V, out, r=None):
    """out[k, i, :] = sum_j P_ij V[k, j, :] (V float32 [batch, m, dv]); r[k, i] = sum_j P_ij if given."""
    import torch
    if V.dtype != torch.float32 or out.dtype != torch.float32:
        raise ValueError("V and out must be float32")
    dv = V.shape[-1]
    _check(lib().fs_transport_apply(h.ptr, _f32(f), _f32(g), _ptr(V), int(dv), _ptr(out), _f32(r)), h.ptr)


def fs_barycentric_map(h: Handle, f, g, Y, out):
    """out[k, i, :] = sum_j P_ij y_j / sum_j P_ij (Y in the handle's dtype, [batch, m, d])."""
    _check(lib().fs_barycentric_map(h.ptr, _f32(f), _f32(g), _ptr(Y), _f32(out)), h.ptr)


def fs_grad_x(h: Handle, f, g, X, Y, grad):
    """grad[k, i, :] = 2 (r_i x_i - sum_j P_ij y_j) (squared Euclidean cost)."""
    _check(lib().fs_grad_x(h.ptr, _f32(f), _f32(g), _ptr(X), _ptr(Y), _f32(grad)), h.ptr)


def fs_transport_apply_t(h: Handle, f, g, U, out, c=None):
    """out[k, j, :] = sum_i P_ij U[k, i, :] (U float32 [batch, n, du]); c[k, j] = sum_i P_ij if given."""
    import torch
    if U.dtype != torch.float32 or out.dtype != torch.float32:
        raise ValueError("U and out must be float32")
    _check(lib().fs_transport_apply_t(h.ptr, _f32(f), _f32(g), _ptr(U), int(U.shape[-1]), _ptr(out), _f32(c)),
           h.ptr)


def fs_grad_y(h: Handle, f, g, X, Y, grad):
    """grad[k, j, :] = 2 (c_j y_j - sum_i P_ij x_i) (squared Euclidean cost)."""
    _check(lib().fs_grad_y(h.ptr, _f32(f), _f32(g), _ptr(X), _ptr(Y), _f32(grad)), h.ptr)


def fs_hvp_x(h: Handle, f, g, X, Y, V, out, max_cg_iters=200, cg_rtol=1e-6) -> int:
    """out = H V, the Hessian of the entropic OT cost with respect to X times V (float32 [n, d]) at
    optimal potentials; returns the conjugate-gradient steps taken."""
    it = ctypes.c_int(0)
    _check(lib().fs_hvp_x(h.ptr, _f32(f), _f32(g), _ptr(X), _ptr(Y), _f32(V), _f32(out), int(max_cg_iters),
                          float(cg_rtol), ctypes.byref(it)), h.ptr)
    return it.value


def fs_selftest_wait(h: Handle, timeout_ms=50) -> int:
    """Run the failure-path self test; returns the library status (FS_ERR_TIMEOUT = 5 expected)."""
    return int(lib().fs_selftest_wait(h.ptr, int(timeout_ms)))


# ---- row-softmax operators without a handle ----
# A call's descriptor and workspace size follow from the tensors' shapes, strides, types and
# device (and the alignment they start on) alone, so they are checked and built once for each
# such combination and kept (at most _PLAN_LIMIT of them; no data, address or tensor is kept).
_plans = {}
_PLAN_LIMIT = 4096
_OP_DTYPES = {"torch.float32": FS_F32, "torch.bfloat16": FS_BF16}


def _same(what, cond):
    if not cond:
        raise ValueError(what)


def _op_dtype(first, *others):
    """The operators' dtype code; every tensor must share it and the device."""
    dt = _OP_DTYPES.get(str(first.dtype))
    if dt is None:
        raise ValueError("tensors must be float32 or bfloat16")
    if not first.is_cuda:
        raise ValueError("expected a CUDA tensor")
    for t in others:
        if t.dtype != first.dtype:
            raise ValueError("tensors must share a dtype")
        if t.device != first.device:
            raise ValueError("tensors must be on one device")
    return dt


def _side(t, dtype, shape, device, what):
    """Address of a contiguous side array (lengths, bias, statistics, targets).  The caller holds t itself until its work
    is enqueued: a temporary's last reference is the call's, and the workspace could take the memory of one let go."""
    if t is None:
        raise ValueError(f"{what} is needed")
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {shape} on the tensors' device")
    return t.data_ptr()


def _view(t, what):
    if t.dim() != 4:
        raise ValueError(f"{what} must be [batch, token, head, width]")
    s, w = t.stride(), t.shape[3]
    if w > 1 and s[3] != 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    return FsView(s[0], s[1], s[2])


def _size(answer):
    """A workspace query's answer; an error where the device could not be asked."""
    if answer == ctypes.c_size_t(-1).value:
        raise FsError(FS_ERR_CUDA, lib().fs_last_error(None).decode())
    return int(answer)


def _plan(key, build, query):
    """(descriptor, reference to it, workspace bytes) of `key`, built on its first use."""
    plan = _plans.get(key)
    if plan is None:
        torch = _torch
        desc, device = build()
        with torch.cuda.device(device):
            plan = (desc, ctypes.byref(desc), _size(query(ctypes.byref(desc))))
        if len(_plans) >= _PLAN_LIMIT:
            _plans.clear()
        _plans[key] = plan
    return plan


def _ready():
    """(library, torch), both loaded."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return lib(), _torch


def _raw_stream(torch, device, stream):
    """The given stream's address, or that of the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
    return stream.cuda_stream


def _scratch(torch, device, need, stream, workspace):
    """(workspace, its bytes): the given one, or one from torch's allocator in the stream's order (under
    graph capture, of the capture's own pool).  The caller holds it until its work is enqueued."""
    if workspace is None:
        if not need:
            return None, 0
        if stream is None:
            return torch.empty(need, dtype=torch.uint8, device=device), need
        with torch.cuda.stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=device), need
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the tensors' device")
    return workspace, workspace.numel() * workspace.element_size()


def _fits(**sizes):
    """Sizes as the descriptors' C ints hold them (ctypes would cut them off without a word)."""
    for name, value in sizes.items():
        if not 0 <= value < 1 << 31:
            raise ValueError(f"{name} is {value}, over what the call takes")


def _ignore_index(value):
    value = int(value)
    if not -(1 << 63) <= value < 1 << 63:
        raise ValueError("ignore_index is not a 64-bit integer")
    return value


def _attn_desc(q, k, v, out, scale):
    dt = _op_dtype(q, k, v, out)
    views = [_view(t, w) for t, w in ((q, "q"), (k, "k"), (v, "v"), (out, "out"))]
    B, n, H, d = q.shape
    m, Hk, dv = k.shape[1], k.shape[2], v.shape[3]
    _same("k must be [batch, m, kv_heads, d]", k.shape[0] == B and k.shape[3] == d)
    _same("v must be [batch, m, kv_heads, dv]", tuple(v.shape[:3]) == (B, m, Hk))
    _same("out must be [batch, n, heads, dv]", tuple(out.shape) == (B, n, H, dv))
    _fits(batch=B, n=n, m=m, heads=H, kv_heads=Hk, d=d, dv=dv)
    return FsAttnDesc(B, n, m, H, Hk, d, dv, dt, float(max(d, 1) ** -0.5 if scale is None else scale), *views)


def _attn_grad_desc(q, k, v, out, dout, dq, dk, dv, scale):
    desc = _attn_desc(q, k, v, out, scale)
    _op_dtype(q, dout, dq, dk, dv)
    for t, like, what in ((dout, out, "dout"), (dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        _same(f"{what} has the wrong shape", t.shape == like.shape)
    desc.dout, desc.dq, desc.dk, desc.dvw = (_view(t, w) for t, w in ((dout, "dout"), (dq, "dq"), (dk, "dk"),
                                                                     (dv, "dv")))
    return desc


def fs_cross_attn(q, k, v, out, lse=None, k_len=None, bias=None, scale=None, stream=None, workspace=None):
    """Cross attention: out[b, i, h] = sum_j softmax_j(scale q_i.k_j + bias_j) v_j.

    q [batch, n, heads, d], k [batch, m, kv_heads, d], v [batch, m, kv_heads, dv], out [batch, n,
    heads, dv]: CUDA float32 or bfloat16 with any strides whose last one is 1 (slices of a fused
    projection, inputs expanded over the batch); bfloat16 widths that are not multiples of 8 up to 128,
    or rows off 16 bytes, leave the tensor cores.  heads is a multiple of kv_heads.  lse (written
    if given): float32 [batch, heads, n].  k_len: int32 [batch] valid keys, or None for all; bias:
    float32 [batch, m] added to the scores, -1e30 or less masking the key.  Masked keys may hold
    anything; a row without a key gives 0 and lse -inf.  scale: 1/sqrt(d) if None.  stream: the
    device's current one if None (tensors used on another stream must be kept alive by the
    caller).  workspace: uint8 tensor of fs_cross_attn_workspace bytes; allocated if None."""
    L, torch = _ready()
    dev = q.get_device()
    scale = None if scale is None else float(scale)  # plans are kept by its value
    desc, ref, need = _plan(
        (scale, dev, q.dtype, k.dtype, v.dtype, out.dtype, k.get_device(), v.get_device(), out.get_device(), q.shape,
         k.shape, v.shape, out.shape, q.stride(), k.stride(), v.stride(), out.stride()),
        lambda: (_attn_desc(q, k, v, out, scale), q.device), lambda d: L.fs_cross_attn_workspace(d, 0))
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return fs_cross_attn(q, k, v, out, lse, k_len, bias, scale, stream, workspace)
    lenp = _side(k_len, torch.int32, (desc.batch,), dev, "k_len") if k_len is not None else None
    biasp = _side(bias, torch.float32, (desc.batch, desc.m), dev, "bias") if bias is not None else None
    lsep = _side(lse, torch.float32, (desc.batch, desc.heads, desc.n), dev, "lse") if lse is not None else None
    raw = _raw_stream(torch, dev, stream)
    ws, size = _scratch(torch, dev, need, stream, workspace)
    status = L.fs_cross_attn(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), lenp, biasp, out.data_ptr(), lsep,
                             ws.data_ptr() if size else None, size, raw)
    if status:
        _check(status)


def fs_cross_attn_grad(q, k, v, out, lse, dout, dq, dk, dv, k_len=None, bias=None, scale=None, stream=None,
                       workspace=None):
    """Gradients dq, dk, dv of fs_cross_attn from its out and lse and the gradient dout of out
    (shapes of q, k, v and out; the other arguments as in the forward)."""
    L, torch = _ready()
    dev = q.get_device()
    scale = None if scale is None else float(scale)  # plans are kept by its value
    tensors = (q, k, v, out, dout, dq, dk, dv)
    desc, ref, need = _plan(
        (scale, dev, *[x for t in tensors for x in (t.shape, t.stride(), t.dtype, t.get_device())]),
        lambda: (_attn_grad_desc(q, k, v, out, dout, dq, dk, dv, scale), q.device),
        lambda d: L.fs_cross_attn_workspace(d, 1))
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return fs_cross_attn_grad(q, k, v, out, lse, dout, dq, dk, dv, k_len, bias, scale, stream, workspace)
    lsep = _side(lse, torch.float32, (desc.batch, desc.heads, desc.n), dev, "lse")
    lenp = _side(k_len, torch.int32, (desc.batch,), dev, "k_len") if k_len is not None else None
    biasp = _side(bias, torch.float32, (desc.batch, desc.m), dev, "bias") if bias is not None else None
    raw = _raw_stream(torch, dev, stream)
    ws, size = _scratch(torch, dev, need, stream, workspace)
    status = L.fs_cross_attn_grad(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), lenp, biasp, out.data_ptr(), lsep,
                                  dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                  ws.data_ptr() if size else None, size, raw)
    if status:
        _check(status)


def fs_cross_attn_workspace(q, k, v, out, dout=None, dq=None, dk=None, dv=None) -> int:
    """Workspace bytes of fs_cross_attn, or (with dout, dq, dk and dv) of fs_cross_attn_grad."""
    import torch
    grad = dout is not None
    desc = _attn_grad_desc(q, k, v, out, dout, dq, dk, dv, None) if grad else _attn_desc(q, k, v, out, None)
    with torch.cuda.device(q.device):
        return _size(lib().fs_cross_attn_workspace(ctypes.byref(desc), int(grad)))


def _rows(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    return t.stride(0)


def _xent_desc(x, w, scale, ignore_index):
    dt = _op_dtype(x, w)
    ldx, ldw = _rows(x, "x"), _rows(w, "w")
    _same("x [n, d] and w [v, d] must share d", x.shape[1] == w.shape[1])
    _fits(rows=x.shape[0], classes=w.shape[0], width=x.shape[1])
    return FsXentDesc(x.shape[0], w.shape[0], x.shape[1], dt, float(scale), ldx, ldw, 0, 0, ignore_index)


def _xent_grad_desc(x, w, dx, dw, scale, ignore_index):
    desc = _xent_desc(x, w, scale, ignore_index)
    _op_dtype(x, dx, dw)
    _same("dx and dw have the shapes of x and w", dx.shape == x.shape and dw.shape == w.shape)
    desc.lddx, desc.lddw = _rows(dx, "dx"), _rows(dw, "dw")
    return desc


def fs_cross_entropy(x, w, target, loss, lse, scale=1.0, ignore_index=-100, stream=None, workspace=None):
    """Softmax cross entropy of logits scale x w^T without storing them: x [n, d], w [v, d] (CUDA
    float32 or bfloat16, rows contiguous, any row stride), target int64 [n]; writes loss and lse,
    float32 [n].  loss_i = lse_i - z_{i, target_i}, 0 where the target is ignore_index, NaN where it
    is anything else outside the classes.  stream, workspace: as in fs_cross_attn."""
    L, torch = _ready()
    dev, xp, wp = x.get_device(), x.data_ptr(), w.data_ptr()
    scale, ignore_index = float(scale), _ignore_index(ignore_index)  # plans are kept by their values
    desc, ref, need = _plan(
        (scale, ignore_index, xp & 127, wp & 15, dev, w.get_device(), x.dtype, w.dtype, x.shape, w.shape, x.stride(),
         w.stride()),
        lambda: (_xent_desc(x, w, scale, ignore_index), x.device),
        lambda d: L.fs_cross_entropy_workspace(d, xp, wp, 0))
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return fs_cross_entropy(x, w, target, loss, lse, scale, ignore_index, stream, workspace)
    shape = (desc.n,)
    tp = _side(target, torch.int64, shape, dev, "target")
    lossp, lsep = _side(loss, torch.float32, shape, dev, "loss"), _side(lse, torch.float32, shape, dev, "lse")
    raw = _raw_stream(torch, dev, stream)
    ws, size = _scratch(torch, dev, need, stream, workspace)
    status = L.fs_cross_entropy(ref, xp, wp, tp, lossp, lsep, ws.data_ptr() if size else None, size, raw)
    if status:
        _check(status)


def fs_cross_entropy_grad(x, w, target, lse, dloss, dx, dw, dlse=None, scale=1.0, ignore_index=-100, stream=None,
                          workspace=None):
    """Gradients dx and dw (shapes of x and w) from the forward's lse and the gradients dloss and
    dlse (float32 [n]; dlse None for 0) of its outputs.  Other arguments as in the forward."""
    L, torch = _ready()
    dev, xp, wp = x.get_device(), x.data_ptr(), w.data_ptr()
    scale, ignore_index = float(scale), _ignore_index(ignore_index)  # plans are kept by their values
    desc, ref, need = _plan(
        (scale, ignore_index, xp & 127, wp & 15, dev,
         *[y for t in (x, w, dx, dw) for y in (t.shape, t.stride(), t.dtype, t.get_device())]),
        lambda: (_xent_grad_desc(x, w, dx, dw, scale, ignore_index), x.device),
        lambda d: L.fs_cross_entropy_workspace(d, xp, wp, 1))
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return fs_cross_entropy_grad(x, w, target, lse, dloss, dx, dw, dlse, scale, ignore_index, stream, workspace)
    shape = (desc.n,)
    tp = _side(target, torch.int64, shape, dev, "target")
    lsep, dlossp = _side(lse, torch.float32, shape, dev, "lse"), _side(dloss, torch.float32, shape, dev, "dloss")
    dlsep = _side(dlse, torch.float32, shape, dev, "dlse") if dlse is not None else None
    raw = _raw_stream(torch, dev, stream)
    ws, size = _scratch(torch, dev, need, stream, workspace)
    status = L.fs_cross_entropy_grad(ref, xp, wp, tp, lsep, dlossp, dlsep, dx.data_ptr(), dw.data_ptr(),
                                     ws.data_ptr() if size else None, size, raw)
    if status:
        _check(status)


def fs_cross_entropy_workspace(x, w, dx=None, dw=None) -> int:
    """Workspace bytes of fs_cross_entropy, or (with dx and dw) of fs_cross_entropy_grad."""
    import torch
    grad = dx is not None
    desc = _xent_grad_desc(x, w, dx, dw, 1.0, -100) if grad else _xent_desc(x, w, 1.0, -100)
    with torch.cuda.device(x.device):
        return _size(lib().fs_cross_entropy_workspace(ctypes.byref(desc), x.data_ptr(), w.data_ptr(), int(grad)))


def fs_check(stream=None):
    """Wait for the stream and raise FsError if a handle-less call on its device reported a
    bounded wait that ran out since the last check."""
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _check(lib().fs_check(ctypes.c_void_p(s.cuda_stream)))


def fs_selftest_check(timeout_ms=50, stream=None):
    """Enqueue a bounded wait that runs out after timeout_ms: the next fs_check raises FsError (FS_ERR_TIMEOUT)."""
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _check(lib().fs_selftest_check(int(timeout_ms), ctypes.c_void_p(s.cuda_stream)))
