"""ctypes binding of libpmx.so (the C ABI declared in include/pmx.h).

Argument marshalling only: torch tensors provide device memory and the
current HIP stream; every step of the computation runs in libpmx's kernels.
Importing this module raises if the built library is missing, so no caller
can silently fall back to another implementation.
"""
import collections
import ctypes
import math
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# PMX_LIBRARY selects another build of the same library (the host-sanitized
# libpmx_san.so of build.py's --sanitize); there is no other implementation
LIB_PATH = os.environ.get("PMX_LIBRARY") or os.path.join(_HERE, "libpmx.so")

OK, ERR_INVALID_VALUE, ERR_NOT_SUPPORTED, ERR_WORKSPACE, ERR_ALIAS, ERR_HIP = range(6)
RUNNING, CONVERGED, MAXITER, STAGNATED, NONFINITE, DIVERGED = -1, 0, 1, 2, 3, 4
F32, BF16 = 0, 1
I32, I64 = 0, 1
MAX_GROUPS, MAX_TOP, MAX_VOCAB, MAX_TOKENS = 1000, 1023, (1 << 22) - 1, 1 << 30
MAX_NORM_COLS, MAX_ROUTE_TOP, MAX_ROUTE_ROWS = 16384, 16, 1 << 25
OP_STATS, OP_INV_ROOT, OP_POLAR, OP_APPLY, OP_POLAR_VARBATCH = range(5)
VARBATCH_MAX_DIM = 64
VARBATCH_MAX_SIDE = 8192
OPTS_VERSION = 4
METHOD_NEWTON_SCHULZ, METHOD_INVERSE_NEWTON = 0, 1
SCALE_FROBENIUS, SCALE_POWER = 0, 1
TRACE_LEN = 64
MAX_SKETCH = 16
STATUS_NAMES = {RUNNING: "RUNNING", CONVERGED: "CONVERGED", MAXITER: "MAXITER",
                STAGNATED: "STAGNATED", NONFINITE: "NONFINITE", DIVERGED: "DIVERGED"}

EXPORTS = [
    "pmx_create", "pmx_destroy", "pmx_status_string", "pmx_version",
    "pmx_matfn_opts_default", "pmx_workspace_size",
    "pmx_shampoo_stats_update", "pmx_shampoo_stats_update_batched",
    "pmx_matfn_inv_root", "pmx_matfn_inv_root_batched",
    "pmx_matfn_polar", "pmx_matfn_polar_batched", "pmx_matfn_polar_varbatch",
    "pmx_precond_apply", "pmx_precond_apply_batched",
    "pmx_trace_enable", "pmx_trace_collect", "pmx_set_host_poll",
    "pmx_shampoo_config_default", "pmx_shampoo_plan_create", "pmx_shampoo_plan_destroy",
    "pmx_shampoo_plan_sizes", "pmx_shampoo_plan_init", "pmx_shampoo_plan_step",
    "pmx_sketch_gaussian", "pmx_precond_apply_noalloc", "pmx_polar_varbatch_workspace_size",
    "pmx_grouped_product", "pmx_grouped_product_workspace_size",
    "pmx_grouped_outer", "pmx_grouped_outer_workspace_size",
    "pmx_embedding", "pmx_embedding_grad", "pmx_embedding_grad_workspace_size",
    "pmx_distill_loss", "pmx_distill_grad", "pmx_distill_workspace_size",
    "pmx_layer_norm", "pmx_layer_norm_grad", "pmx_layer_norm_grad_workspace_size",
    "pmx_route", "pmx_route_grad", "pmx_route_workspace_size",
    "pmx_fp8_store", "pmx_fp8_load", "pmx_fp8_store_weight",
    "pmx_silu_checkpoint", "pmx_silu_checkpoint_grad",
    "pmx_fp8_product",
]

# kernel classes of the launch trace (pmx_kernel_class)
KERNEL_CLASSES = ["gemm_power", "gemm_update", "gemm_resid", "gemm_stats", "gemm_apply",
                  "skinny", "skinny_alpha", "other"]


class Opts(ctypes.Structure):
    _fields_ = [("struct_version", ctypes.c_int32), ("degree", ctypes.c_int32),
                ("sketch_p", ctypes.c_int32), ("max_iter", ctypes.c_int32),
                ("accelerate", ctypes.c_int32), ("alpha_lo", ctypes.c_float),
                ("alpha_hi", ctypes.c_float), ("tol", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("fp64_iters", ctypes.c_int32),
                ("degree_max", ctypes.c_int32), ("adapt_ratio", ctypes.c_float),
                ("method", ctypes.c_int32), ("scale_mode", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ShampooConfig(ctypes.Structure):
    _fields_ = [("struct_version", ctypes.c_int32), ("block", ctypes.c_int32),
                ("root_every", ctypes.c_int32), ("adaptive_lr", ctypes.c_int32),
                ("beta", ctypes.c_float), ("eps", ctypes.c_float), ("lr", ctypes.c_float),
                ("momentum", ctypes.c_float), ("root_opts", Opts)]


class Layer(ctypes.Structure):
    _fields_ = [("dims", ctypes.c_int32), ("shape", ctypes.c_int32 * 4)]


class PolarBlock(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("u", ctypes.c_void_p), ("m", ctypes.c_int32),
                ("n", ctypes.c_int32), ("ldg", ctypes.c_int32), ("ldu", ctypes.c_int32)]


class DistillProblem(ctypes.Structure):
    _fields_ = [("struct_version", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int32), ("top", ctypes.c_int32),
                ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
                ("teacher_ids", ctypes.c_void_p), ("ld_ids", ctypes.c_int64),
                ("teacher", ctypes.c_void_p), ("ld_teacher", ctypes.c_int64),
                ("labels", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("ids_type", ctypes.c_int32), ("labels_type", ctypes.c_int32),
                ("teacher_dtype", ctypes.c_int32), ("tau", ctypes.c_float),
                ("mix", ctypes.c_float), ("reserved", ctypes.c_int32)]


class RouteProblem(ctypes.Structure):
    _fields_ = [("struct_version", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("experts", ctypes.c_int32), ("top", ctypes.c_int32),
                ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64), ("live", ctypes.c_void_p),
                ("balance", ctypes.c_float), ("zloss", ctypes.c_float),
                ("normalize", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Info(ctypes.Structure):
    _fields_ = [("status", ctypes.c_int32), ("iters", ctypes.c_int32 * 2),
                ("gemms", ctypes.c_int32), ("sketch_products", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("scale", ctypes.c_float),
                ("residual", ctypes.c_float * 2),
                ("alpha", (ctypes.c_float * TRACE_LEN) * 2),
                ("rtrace", (ctypes.c_float * TRACE_LEN) * 2)]


INFO_DTYPE = np.dtype([("status", "<i4"), ("iters", "<i4", (2,)), ("gemms", "<i4"),
                       ("sketch_products", "<i4"), ("stages", "<i4"), ("scale", "<f4"),
                       ("residual", "<f4", (2,)), ("alpha", "<f4", (2, TRACE_LEN)),
                       ("rtrace", "<f4", (2, TRACE_LEN))])
assert INFO_DTYPE.itemsize == ctypes.sizeof(Info)

_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libpmx.so is not built (%s); run "
                          "`python -m preconditioned_optimizer_matrix_amd.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "pmx_create": (_i32, [ctypes.POINTER(_vp), _i32]),
        "pmx_destroy": (_i32, [_vp]),
        "pmx_status_string": (ctypes.c_char_p, [_i32]),
        "pmx_version": (_i32, []),
        "pmx_matfn_opts_default": (_i32, [ctypes.POINTER(Opts)]),
        "pmx_workspace_size": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(Opts),
                                      ctypes.POINTER(_sz)]),
        "pmx_shampoo_stats_update": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp,
                                            _i32, _f32, _f32, _vp, _sz, _vp]),
        "pmx_shampoo_stats_update_batched": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _i64, _vp,
                                                    _i32, _i64, _vp, _i32, _i64, _f32, _f32,
                                                    _i32, _vp, _sz, _vp]),
        "pmx_matfn_inv_root": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _i32,
                                      ctypes.POINTER(Opts), _vp, _vp, _sz, _vp]),
        "pmx_matfn_inv_root_batched": (_i32, [_vp, _vp, _i32, _i32, _i64, _i32, _vp, _i32, _i64,
                                              _vp, _i32, _i64, _i32, ctypes.POINTER(Opts), _vp,
                                              _vp, _sz, _vp]),
        "pmx_matfn_polar": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32,
                                   ctypes.POINTER(Opts), _vp, _vp, _sz, _vp]),
        "pmx_matfn_polar_batched": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _i64, _vp, _i32,
                                           _i64, _i32, ctypes.POINTER(Opts), _vp, _vp, _sz,
                                           _vp]),
        "pmx_matfn_polar_varbatch": (_i32, [_vp, ctypes.POINTER(PolarBlock), _i32, _i32,
                                            ctypes.POINTER(Opts), _vp, _vp, _sz, _vp]),
        "pmx_precond_apply": (_i32, [_vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp, _i32,
                                     _vp, _i32, _vp, _sz, _vp]),
        "pmx_precond_apply_batched": (_i32, [_vp, _vp, _i32, _i64, _vp, _i32, _i32, _i32, _i32,
                                             _i64, _vp, _i32, _i64, _vp, _i32, _i64, _i32, _vp,
                                             _sz, _vp]),
        "pmx_polar_varbatch_workspace_size": (_i32, [ctypes.POINTER(PolarBlock), _i32, _i32,
                                                     ctypes.POINTER(Opts),
                                                     ctypes.POINTER(_sz)]),
        "pmx_precond_apply_noalloc": (_i32, [_vp, _vp, _i32, _i64, _vp, _i32, _i32, _i32, _i32,
                                             _i64, _vp, _i32, _i64, _vp, _i32, _i64, _i32,
                                             _vp]),
        "pmx_trace_enable": (_i32, [_vp, _i32]),
        "pmx_set_host_poll": (_i32, [_vp, _i32]),
        "pmx_shampoo_config_default": (_i32, [ctypes.POINTER(ShampooConfig)]),
        "pmx_shampoo_plan_create": (_i32, [_vp, ctypes.POINTER(ShampooConfig),
                                           ctypes.POINTER(Layer), _i32,
                                           ctypes.POINTER(ctypes.c_void_p)]),
        "pmx_shampoo_plan_destroy": (_i32, [_vp]),
        "pmx_shampoo_plan_sizes": (_i32, [_vp, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]),
        "pmx_shampoo_plan_init": (_i32, [_vp, _vp, _sz, _vp]),
        "pmx_shampoo_plan_step": (_i32, [_vp, ctypes.POINTER(ctypes.c_void_p),
                                         ctypes.POINTER(ctypes.c_void_p), _i64, _vp, _sz, _vp,
                                         _sz, _vp]),
        "pmx_sketch_gaussian": (_i32, [_vp, ctypes.c_uint64, _i32, _i32, _i32, _i32, _i32, _vp,
                                       _i32, _vp, _vp]),
        "pmx_trace_collect": (_i32, [_vp, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_int64)]),
        "pmx_grouped_product_workspace_size": (_i32, [_i64, _i32, _i32, _i32, _i32,
                                                      ctypes.POINTER(_sz)]),
        "pmx_grouped_product": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _vp, _i32, _i64, _i64,
                                       _i32, _vp, _i32, _i32, _vp, _i32, _i64, _vp, _sz, _vp]),
        "pmx_grouped_outer_workspace_size": (_i32, [_i64, _i32, _i32, _i32, _i32,
                                                    ctypes.POINTER(_sz)]),
        "pmx_grouped_outer": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _vp, _i32, _i64, _vp, _i32,
                                     _i32, _vp, _i32, _i64, _i64, _i32, _vp, _sz, _vp]),
        "pmx_embedding": (_i32, [_vp, _vp, _i32, _i32, _i32, _i64, _vp, _i32, _i64, _f32, _vp,
                                 _i64, _vp]),
        "pmx_embedding_grad_workspace_size": (_i32, [_i64, _i32, _i32, ctypes.POINTER(_sz)]),
        "pmx_embedding_grad": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _vp, _i32, _i32, _f32,
                                      _i64, _vp, _i32, _i64, _i32, _vp, _sz, _vp]),
        "pmx_distill_workspace_size": (_i32, [ctypes.POINTER(DistillProblem),
                                              ctypes.POINTER(_sz)]),
        "pmx_distill_loss": (_i32, [_vp, ctypes.POINTER(DistillProblem), _vp, _vp, _vp, _vp, _i64,
                                    _vp, _sz, _vp]),
        "pmx_distill_grad": (_i32, [_vp, ctypes.POINTER(DistillProblem), _vp, _vp, _vp, _i64,
                                    _vp]),
        "pmx_layer_norm": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _vp, _vp, _i32, _f32, _vp,
                                  _i64, _vp, _vp]),
        "pmx_layer_norm_grad_workspace_size": (_i32, [_i64, _i32, _i32, ctypes.POINTER(_sz)]),
        "pmx_layer_norm_grad": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _vp, _i64, _vp, _vp,
                                       _i32, _vp, _i64, _vp, _vp, _i32, _vp, _sz, _vp]),
        "pmx_route_workspace_size": (_i32, [ctypes.POINTER(RouteProblem), ctypes.POINTER(_sz)]),
        "pmx_route": (_i32, [_vp, ctypes.POINTER(RouteProblem), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                             _vp, _sz, _vp]),
        "pmx_route_grad": (_i32, [_vp, ctypes.POINTER(RouteProblem), _vp, _vp, _vp, _vp, _vp, _vp,
                                  _i64, _vp]),
        "pmx_fp8_store": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _vp, _i64, _vp, _i64, _vp]),
        "pmx_fp8_load": (_i32, [_vp, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _i32, _i64, _vp]),
        "pmx_fp8_store_weight": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _i64, _i64, _i32, _vp,
                                        _i64, _i64, _vp, _i64, _i64, _vp]),
        "pmx_silu_checkpoint": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _i32, _vp, _i64, _vp,
                                       _i64, _vp, _i64, _vp]),
        "pmx_silu_checkpoint_grad": (_i32, [_vp, _vp, _i32, _i64, _i32, _i64, _vp, _i64, _vp,
                                            _i64, _i32, _vp, _i64, _vp, _i64, _vp]),
        "pmx_fp8_product": (_i32, [_vp, _vp, _i64, _i32, _i64, _vp, _i64, _vp, _i32, _i64, _i64,
                                   _vp, _i64, _i64, _vp, _i32, _i32, _vp, _i32, _i64, _vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


class PmxError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        msg = lib.pmx_status_string(code).decode()
        super().__init__("%s: %s" % (where, msg))


def check(code, where=""):
    if code != OK:
        raise PmxError(code, where)


def default_opts(**kw):
    """pmx_matfn_opts with the library defaults, fields overridden by kw."""
    o = Opts()
    check(lib.pmx_matfn_opts_default(ctypes.byref(o)), "opts_default")
    for k, v in kw.items():
        if not hasattr(o, k):
            raise KeyError(k)
        setattr(o, k, v)
    return o


# ---------------------------------------------------------------- torch glue
def _torch():
    import torch
    return torch


_handles = {}


def handle(device=None):
    torch = _torch()
    dev = torch.cuda.current_device() if device is None else int(device)
    h = _handles.get(dev)
    if h is None:
        hv = _vp()
        check(lib.pmx_create(ctypes.byref(hv), dev), "pmx_create")
        h = _handles[dev] = hv
    return h


def _stream(t):
    torch = _torch()
    return _vp(torch.cuda.current_stream(t.device).cuda_stream)


def _stream_of(device):
    torch = _torch()
    return _vp(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("unsupported dtype %s" % t.dtype)


def _mat(t):
    """(rows, cols, ld, batch_stride, batch) of a 2-D or 3-D row-major tensor."""
    if t.dim() == 2:
        if t.stride(1) != 1:
            raise ValueError("matrices must have unit column stride")
        return t.shape[0], t.shape[1], t.stride(0), 0, 1
    if t.dim() == 3:
        if t.stride(2) != 1:
            raise ValueError("matrices must have unit column stride")
        return t.shape[1], t.shape[2], t.stride(1), t.stride(0), t.shape[0]
    raise ValueError("expected a 2-D matrix or a 3-D batch")


def _ptr(t):
    return _vp(t.data_ptr()) if t is not None else _vp(0)


def workspace_bytes(op, m, n, batch=1, dtype=F32, opts=None):
    sz = _sz()
    check(lib.pmx_workspace_size(None, op, m, n, batch, dtype,
                                 ctypes.byref(opts) if opts is not None else None,
                                 ctypes.byref(sz)), "workspace_size")
    return sz.value


def workspace(nbytes, device):
    """Workspace tensor (256-byte aligned: torch's caching allocator aligns to 512 B)."""
    torch = _torch()
    t = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)
    assert t.data_ptr() % 256 == 0
    return t


def new_info(batch, device):
    torch = _torch()
    return torch.zeros(batch * INFO_DTYPE.itemsize, dtype=torch.uint8, device=device)


def parse_info(info_tensor):
    """Device info buffer -> numpy structured array (synchronises via .cpu())."""
    raw = info_tensor.detach().cpu().numpy().tobytes()
    return np.frombuffer(raw, dtype=INFO_DTYPE)


def shampoo_stats_update(G, L, R, beta, eps, ws=None):
    """In place: L <- beta L + (1-beta) G G^T + eps I, R <- beta R + (1-beta) G^T G + eps I."""
    m, n, ldg, sg, batch = _mat(G)
    if L is not None and L.dim() == 3:
        batch = L.shape[0]
    elif R is not None and R.dim() == 3:
        batch = R.shape[0]
    if L is not None:
        _, _, ldl, sl, _ = _mat(L)
    else:
        ldl, sl = m, 0
    if R is not None:
        _, _, ldr, sr, _ = _mat(R)
    else:
        ldr, sr = n, 0
    dt = _dtype_code(G)
    need = workspace_bytes(OP_STATS, m, n, batch, dt, None)
    if need and (ws is None or ws.numel() < need):
        ws = workspace(need, G.device)
    check(lib.pmx_shampoo_stats_update_batched(
        handle(G.device.index), _ptr(G), dt, m, n, ldg, sg, _ptr(L), ldl, sl,
        _ptr(R), ldr, sr, float(beta), float(eps), batch, _ptr(ws) if need else None,
        ws.numel() if need else 0, _stream(G)), "shampoo_stats_update")
    return L, R


def inv_root(A, p, opts=None, aux=True, out=None, out_aux=None, info=None, ws=None):
    """A^{-1/p} (and A^{1/p} if aux) of an SPD matrix or a batch of them.
    Returns (X, X_aux or None, info_tensor)."""
    torch = _torch()
    n, n2, lda, sa, batch = _mat(A)
    if n != n2:
        raise ValueError("A must be square")
    if opts is None:
        opts = default_opts()
    X = out if out is not None else torch.empty_like(A, memory_format=torch.contiguous_format)
    XA = None
    if aux:
        XA = out_aux if out_aux is not None else torch.empty_like(X)
    _, _, ldx, sx, _ = _mat(X)
    ldaux, saux = (n, 0)
    if XA is not None:
        _, _, ldaux, saux, _ = _mat(XA)
    if info is None:
        info = new_info(batch, A.device)
    need = workspace_bytes(OP_INV_ROOT, n, n, batch, F32, opts)
    if ws is None or ws.numel() < need:
        ws = workspace(need, A.device)
    check(lib.pmx_matfn_inv_root_batched(
        handle(A.device.index), _ptr(A), n, lda, sa, int(p), _ptr(X), ldx, sx, _ptr(XA),
        ldaux, saux, batch, ctypes.byref(opts), _ptr(info), _ptr(ws), ws.numel(),
        _stream(A)), "matfn_inv_root")
    return X, XA, info


def polar(G, opts=None, out=None, info=None, ws=None):
    """Polar factor of G (m x n) or a batch; returns (U, info_tensor)."""
    torch = _torch()
    m, n, ldg, sg, batch = _mat(G)
    if opts is None:
        opts = default_opts()
    U = out if out is not None else torch.empty_like(G, memory_format=torch.contiguous_format)
    _, _, ldu, su, _ = _mat(U)
    if info is None:
        info = new_info(batch, G.device)
    dt = _dtype_code(G)
    need = workspace_bytes(OP_POLAR, m, n, batch, dt, opts)
    if ws is None or ws.numel() < need:
        ws = workspace(need, G.device)
    check(lib.pmx_matfn_polar_batched(
        handle(G.device.index), _ptr(G), dt, m, n, ldg, sg, _ptr(U), ldu, su, batch,
        ctypes.byref(opts), _ptr(info), _ptr(ws), ws.numel(), _stream(G)), "matfn_polar")
    return U, info


class VarBlocks:
    """The descriptor table of a variable-size polar call: the addresses,
    shapes and row strides of the blocks Gs (2-D, unit column stride, one
    dtype) and of their outputs Us (allocated when not given).  Built once and
    passed to polar_varbatch(blocks=...) on every call over the same tensors,
    so a call marshals nothing per block; valid while those tensors live."""

    def __init__(self, Gs, Us=None):
        torch = _torch()
        self.Gs = list(Gs)
        if not self.Gs:
            raise ValueError("no blocks")
        self.Us = (list(Us) if Us is not None else
                   [torch.empty_like(g, memory_format=torch.contiguous_format) for g in self.Gs])
        if len(self.Us) != len(self.Gs):
            raise ValueError("one output per block")
        self.count = len(self.Gs)
        self.arr = (PolarBlock * self.count)()
        for i, (g, u) in enumerate(zip(self.Gs, self.Us)):
            if g.dim() != 2 or u.dim() != 2:
                raise ValueError("blocks are 2-D matrices")
            m, n, ldg, _, _ = _mat(g)
            _, _, ldu, _, _ = _mat(u)
            self.arr[i] = PolarBlock(_ptr(g), _ptr(u), m, n, ldg, ldu)
        self.dtype = _dtype_code(self.Gs[0])
        self.device = self.Gs[0].device


def polar_varbatch(Gs=None, opts=None, outs=None, info=None, ws=None, blocks=None):
    """Polar factors of a list of 2-D blocks of different shapes (sides up to
    VARBATCH_MAX_SIDE, one dtype) in one call: blocks of sides up to
    VARBATCH_MAX_DIM in one fused launch, larger ones grouped by shape;
    returns (list of U, info_tensor).  `blocks` (a VarBlocks) replaces Gs and
    outs with a descriptor table built beforehand."""
    if opts is None:
        opts = default_opts()
    if blocks is None:
        blocks = VarBlocks(Gs, outs)
    count, dev = blocks.count, blocks.device
    if info is None:
        info = new_info(count, dev)
    sz = _sz()
    check(lib.pmx_polar_varbatch_workspace_size(blocks.arr, count, blocks.dtype,
                                                ctypes.byref(opts), ctypes.byref(sz)),
          "polar_varbatch_workspace_size")
    need = sz.value
    if ws is None or ws.numel() < need:
        ws = workspace(need, dev)
    check(lib.pmx_matfn_polar_varbatch(handle(dev.index), blocks.arr, count, blocks.dtype,
                                       ctypes.byref(opts), _ptr(info), _ptr(ws), ws.numel(),
                                       _stream(blocks.Gs[0])), "matfn_polar_varbatch")
    return blocks.Us, info


def shampoo_config(root_opts=None, **kw):
    """pmx_shampoo_config with the library defaults, fields overridden by kw."""
    c = ShampooConfig()
    check(lib.pmx_shampoo_config_default(ctypes.byref(c)), "shampoo_config_default")
    for k, v in kw.items():
        if not hasattr(c, k):
            raise KeyError(k)
        setattr(c, k, v)
    if root_opts is not None:
        c.root_opts = root_opts
    return c


def _layer(shape):
    ly = Layer()
    ly.dims = len(shape)
    if ly.dims not in (2, 4):
        # passed on: the library rejects it (PMX_ERR_INVALID_VALUE)
        return ly
    for i, v in enumerate(shape[:4]):
        ly.shape[i] = int(v)
    return ly


class ShampooPlan:
    """A whole Shampoo step over a list of layer shapes (2-D or 4-D), with its
    device state and workspace (torch tensors on `device`)."""

    def __init__(self, shapes, device, config=None):
        torch = _torch()
        self.device = torch.device(device)
        self.config = config if config is not None else shampoo_config()
        arr = (Layer * len(shapes))(*[_layer(s) for s in shapes])
        self.nlayers = len(shapes)
        plan = ctypes.c_void_p()
        check(lib.pmx_shampoo_plan_create(handle(self.device.index), ctypes.byref(self.config),
                                          arr, len(shapes), ctypes.byref(plan)),
              "shampoo_plan_create")
        self.plan = plan
        sb, wb = _sz(), _sz()
        check(lib.pmx_shampoo_plan_sizes(plan, ctypes.byref(sb), ctypes.byref(wb)),
              "shampoo_plan_sizes")
        self.state = workspace(sb.value, self.device)
        self.ws = workspace(wb.value, self.device)
        check(lib.pmx_shampoo_plan_init(plan, _ptr(self.state), self.state.numel(),
                                        _stream_of(self.device)), "shampoo_plan_init")

    def step(self, Ws, Gs, t):
        if len(Ws) != self.nlayers or len(Gs) != self.nlayers:
            raise ValueError("one weight and one gradient per layer")
        for w, g in zip(Ws, Gs):
            if w.dtype != _torch().float32 or g.dtype != _torch().float32:
                raise TypeError("fp32 weights and gradients")
            if not (w.is_contiguous() and g.is_contiguous()):
                raise ValueError("contiguous weights and gradients")
        wp = (ctypes.c_void_p * self.nlayers)(*[w.data_ptr() for w in Ws])
        gp = (ctypes.c_void_p * self.nlayers)(*[g.data_ptr() for g in Gs])
        check(lib.pmx_shampoo_plan_step(self.plan, wp, gp, int(t), _ptr(self.state),
                                        self.state.numel(), _ptr(self.ws), self.ws.numel(),
                                        _stream_of(self.device)), "shampoo_plan_step")

    def __del__(self):
        if getattr(self, "plan", None) is not None and lib is not None:
            lib.pmx_shampoo_plan_destroy(self.plan)
            self.plan = None


def precond_apply(Linv, G, Rinv, out=None, ws=None):
    """P = Linv G Rinv (single or batched)."""
    torch = _torch()
    m, n, ldg, sg, batch = _mat(G)
    _, _, ldl, sl, _ = _mat(Linv)
    _, _, ldr, sr, _ = _mat(Rinv)
    P = out if out is not None else torch.empty_like(G, memory_format=torch.contiguous_format)
    _, _, ldp, sp, _ = _mat(P)
    dt = _dtype_code(G)
    need = workspace_bytes(OP_APPLY, m, n, batch, dt, None)
    if ws is None or ws.numel() < need:
        ws = workspace(need, G.device)
    check(lib.pmx_precond_apply_batched(
        handle(G.device.index), _ptr(Linv), ldl, sl, _ptr(G), dt, m, n, ldg, sg, _ptr(Rinv),
        ldr, sr, _ptr(P), ldp, sp, batch, _ptr(ws), ws.numel(), _stream(G)),
        "precond_apply")
    return P


def sketch_gaussian(seed, matrix, stage, k, n, p, device=None, words=True):
    """The iterations' Gaussian sketch S_k (n x p fp32) of (matrix, stage, k)
    and, if words, the raw Philox words behind it (n x p int32 tensor holding
    the uint32 bits); returns (S, words or None)."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else int(device))
    S = torch.empty((n, p), dtype=torch.float32, device=dev)
    Wd = torch.empty((n, p), dtype=torch.int32, device=dev) if words else None
    check(lib.pmx_sketch_gaussian(handle(dev.index), ctypes.c_uint64(int(seed)), int(matrix),
                                  int(stage), int(k), int(n), int(p), _ptr(S), int(p), _ptr(Wd),
                                  _stream_of(dev)), "sketch_gaussian")
    return S, Wd


NOALLOC_SCRATCH_BYTES = 32 << 20


def precond_apply_noalloc(Linv, G, Rinv, out=None):
    """P = Linv G Rinv through the allocation-free entry point (the library's
    scratch holds the intermediate; no workspace)."""
    torch = _torch()
    m, n, ldg, sg, batch = _mat(G)
    _, _, ldl, sl, _ = _mat(Linv)
    _, _, ldr, sr, _ = _mat(Rinv)
    P = out if out is not None else torch.empty_like(G, memory_format=torch.contiguous_format)
    _, _, ldp, sp, _ = _mat(P)
    check(lib.pmx_precond_apply_noalloc(
        handle(G.device.index), _ptr(Linv), ldl, sl, _ptr(G), _dtype_code(G), m, n, ldg, sg,
        _ptr(Rinv), ldr, sr, _ptr(P), ldp, sp, batch, _stream(G)), "precond_apply_noalloc")
    return P


def set_host_poll(chunk, device=None):
    """Host-polled convergence for this device's handle: after every `chunk`
    updates the iteration loops publish whether any matrix still iterates and
    stop enqueuing once none does (0 turns it off: all max_iter updates are
    enqueued and the surplus ones exit on the device).  Same results either
    way; the calling thread waits on the published points."""
    check(lib.pmx_set_host_poll(handle(device), int(chunk)), "set_host_poll")


def trace_enable(enable=True, device=None):
    """Bracket every launch of this device's handle with HIP events."""
    check(lib.pmx_trace_enable(handle(device), 1 if enable else 0), "trace_enable")


def trace_collect(device=None):
    """{kernel class: (total ms, launches)} of the launches since trace_enable
    or the previous collect (waits for the recorded events)."""
    n = len(KERNEL_CLASSES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    check(lib.pmx_trace_collect(handle(device), ms, cnt), "trace_collect")
    return {KERNEL_CLASSES[i]: (ms[i], cnt[i]) for i in range(n)}


# ---------------------------------------------------------------- training step
# Products grouped by expert, the token embedding, the distillation loss.
# Arguments that describe one call are checked here only as far as the tensors
# themselves go (device, type, shape agreement, unit column stride); sizes,
# strides, alignment and overlap are checked by the library.

_codes = {}


def _fill_codes():
    torch = _torch()
    _codes.update({torch.float32: F32, torch.bfloat16: BF16, torch.int32: I32, torch.int64: I64})
    _codes["stream"] = torch._C._cuda_getCurrentRawStream
    _codes["empty"] = torch.empty
    _codes["f32"] = torch.float32
    _codes["e4m3"], _codes["byte"], _codes["i32"] = torch.float8_e4m3fn, torch.uint8, torch.int32
    _codes["bool"] = torch.bool


def _elem_code(t):
    c = _codes.get(t.dtype)
    if c is None or not t.is_floating_point():
        raise TypeError("unsupported dtype %s" % t.dtype)
    return c


def _index_code(t):
    c = _codes.get(t.dtype)
    if c is None or t.is_floating_point():
        raise TypeError("index tensors are int32 or int64, not %s" % t.dtype)
    return c


def _on(first, *rest):
    """The GPU all the tensors live on."""
    if not _codes:
        _fill_codes()
    d = first.get_device()
    if d < 0:
        raise ValueError("tensors live on the GPU")
    for t in rest:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors on different devices")
    return d


def _call(d):
    """Handle and current stream of GPU d."""
    h = _handles.get(d)
    return (h if h is not None else handle(d)), _codes["stream"](d)


def _rows_of(t, what):
    """(rows, columns, row distance) of a 2-D tensor with unit column stride."""
    s = t.shape
    if len(s) != 2:
        raise ValueError("%s must be 2-D" % what)
    r, c = s
    ld, one = t.stride()
    if one != 1 and c > 1:
        raise ValueError("%s must have unit column stride" % what)
    return r, c, (ld if r > 1 else max(c, 1))


def _vector(t, what):
    if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector" % what)
    return t.numel()


def _matrices_of(t, what):
    """(batch, rows, columns, row distance, matrix distance) of a 3-D tensor."""
    s = t.shape
    if len(s) != 3:
        raise ValueError("%s must be 3-D" % what)
    b, r, c = s
    sb, ld, one = t.stride()
    if one != 1 and c > 1:
        raise ValueError("%s must have unit column stride" % what)
    if r <= 1:
        ld = max(c, 1)
    return b, r, c, ld, (sb if b > 1 else r * ld)


_sizes = {}


def _need(query, *args):
    """Workspace bytes of a call's sizes (host arithmetic only, remembered)."""
    key = (query,) + args
    n = _sizes.get(key)
    if n is None:
        sz = _sz()
        check(getattr(lib, query)(*args, ctypes.byref(sz)), query)
        n = _keep_size(key, sz.value)
    return n


def _keep_size(key, n):
    if len(_sizes) >= 4096:
        _sizes.clear()
    _sizes[key] = n
    return n


def _ws_for(need, ws, device):
    # numel elements from data_ptr on are the workspace's only when contiguous
    if ws is not None and (ws.device != device or not ws.is_contiguous()):
        raise ValueError("ws must be contiguous, on the other tensors' device")
    if not need:
        return None, 0
    if ws is None or ws.numel() < need:
        ws = workspace(need, device)
    return ws.data_ptr(), ws.numel() * ws.element_size()


def grouped_product(A, B, offsets, trans_b=False, out=None, out_dtype=None, ws=None):
    """C[t] = A[t] B[e] (trans_b: A[t] B[e]^T) for the rows offsets[e] <= t <
    offsets[e + 1] of group e; rows in no group are zeros.  A (rows x k), B
    (groups x k x n, or groups x n x k with trans_b) bf16 or fp32, offsets
    (groups + 1) int32 or int64 on the device; C in A's type or fp32."""
    d = _on(A, B, offsets, out)
    rows, k, lda = _rows_of(A, "A")
    groups, br, bc, ldb, sb = _matrices_of(B, "B")
    n = br if trans_b else bc
    if (bc if trans_b else br) != k:
        raise ValueError("A and B disagree about k")
    if B.dtype != A.dtype:
        raise TypeError("A and B have different types")
    if _vector(offsets, "offsets") != groups + 1:
        raise ValueError("one offset per group and one more")
    if out is None:
        out = _codes["empty"]((rows, n), dtype=out_dtype or A.dtype, device=A.device)
    elif tuple(out.shape) != (rows, n) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has another shape or type")
    _, _, ldc = _rows_of(out, "out")
    dt = _elem_code(A)
    need = _need("pmx_grouped_product_workspace_size", rows, k, n, groups, dt)
    wp, wn = _ws_for(need, ws, A.device)
    h, st = _call(d)
    check(lib.pmx_grouped_product(
        h, A.data_ptr(), dt, rows, k, lda, B.data_ptr(), n, ldb, sb,
        1 if trans_b else 0, offsets.data_ptr(), _index_code(offsets), groups, out.data_ptr(),
        _elem_code(out), ldc, wp, wn, st), "grouped_product")
    return out


def grouped_outer(A, B, offsets, out=None, out_dtype=None, accumulate=False, ws=None):
    """C[e] = A_e^T B_e over the rows of group e (accumulate: C[e] += ...):
    with A = dY and B = X the gradient of out x in weights.  A (rows x m), B
    (rows x n); C (groups x m x n) in A's type or fp32."""
    d = _on(A, B, offsets, out)
    rows, m, lda = _rows_of(A, "A")
    rb, n, ldb = _rows_of(B, "B")
    if rb != rows:
        raise ValueError("A and B have different numbers of rows")
    if B.dtype != A.dtype:
        raise TypeError("A and B have different types")
    groups = _vector(offsets, "offsets") - 1
    if groups < 1:
        raise ValueError("one offset per group and one more")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _codes["empty"]((groups, m, n), dtype=out_dtype or A.dtype, device=A.device)
    elif tuple(out.shape) != (groups, m, n) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has another shape or type")
    _, _, _, ldc, sc = _matrices_of(out, "out")
    dt = _elem_code(A)
    need = _need("pmx_grouped_outer_workspace_size", rows, m, n, groups, dt)
    wp, wn = _ws_for(need, ws, A.device)
    h, st = _call(d)
    check(lib.pmx_grouped_outer(
        h, A.data_ptr(), dt, rows, m, lda, B.data_ptr(), n, ldb,
        offsets.data_ptr(), _index_code(offsets), groups, out.data_ptr(), _elem_code(out), ldc, sc,
        1 if accumulate else 0, wp, wn, st), "grouped_outer")
    return out


def embedding(W, ids, scale=1.0, out=None):
    """scale W[ids] for a table W (vocab x dim) and ids of any shape; an id
    outside the table gives zeros."""
    d = _on(W, ids, out)
    vocab, dim, ldt = _rows_of(W, "W")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    shape = tuple(ids.shape) + (dim,)
    if out is None:
        out = _codes["empty"](shape, dtype=W.dtype, device=W.device)
        ldy = dim
    else:
        if tuple(out.shape) != shape or out.dtype != W.dtype:
            raise ValueError("out has another shape or type")
        if out.dim() == 2:
            ldy = _rows_of(out, "out")[2]
        elif out.is_contiguous():
            ldy = dim
        else:
            raise ValueError("out must be contiguous")
    h, st = _call(d)
    check(lib.pmx_embedding(h, W.data_ptr(), _elem_code(W), vocab, dim, ldt,
                            ids.data_ptr(), _index_code(ids), ids.numel(), scale, out.data_ptr(),
                            ldy, st), "embedding")
    return out


def embedding_grad(dY, ids, vocab, scale=1.0, padding_idx=-1, out=None, out_dtype=None,
                   accumulate=False, ws=None):
    """Gradient of embedding's table: dW[v] = scale sum of dY over the tokens
    of id v, zeros elsewhere (accumulate: added to out instead).  Tokens of
    padding_idx, or of ids outside the table, are left out.  dY is tokens x dim
    (or ids' shape x dim, contiguous); dW in dY's type or out_dtype."""
    d = _on(dY, ids, out)
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    if tuple(dY.shape[:-1]) != tuple(ids.shape):
        raise ValueError("one row of dY per id")
    if dY.dim() != 2:
        if not dY.is_contiguous():
            raise ValueError("dY must be contiguous")
        dY = dY.view(-1, dY.shape[-1])
    tokens, dim, lddy = _rows_of(dY, "dY")
    vocab = int(vocab)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _codes["empty"]((vocab, dim), dtype=out_dtype or dY.dtype, device=dY.device)
    elif tuple(out.shape) != (vocab, dim) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has another shape or type")
    _, _, lddw = _rows_of(out, "out")
    need = _need("pmx_embedding_grad_workspace_size", tokens, vocab, dim)
    wp, wn = _ws_for(need, ws, dY.device)
    h, st = _call(d)
    check(lib.pmx_embedding_grad(
        h, dY.data_ptr(), _elem_code(dY), tokens, dim, lddy, ids.data_ptr(),
        _index_code(ids), vocab, scale, padding_idx, out.data_ptr(), _elem_code(out), lddw,
        1 if accumulate else 0, wp, wn, st), "embedding_grad")
    return out


def _distill_problem(Z, teacher_ids, teacher, tau, mix, labels, weights):
    _on(Z, teacher_ids, teacher, labels, weights)
    rows, vocab, ldz = _rows_of(Z, "Z")
    top = ids = ld_ids = te = ld_te = it = td = 0
    if teacher_ids is not None:
        ri, top, ld_ids = _rows_of(teacher_ids, "teacher_ids")
        rt, tt, ld_te = _rows_of(teacher, "teacher")
        if ri != rows or rt != rows or tt != top:
            raise ValueError("teacher_ids and teacher are rows x top")
        ids, te = teacher_ids.data_ptr(), teacher.data_ptr()
        it, td = _index_code(teacher_ids), _elem_code(teacher)
    lab = lt = wp = None
    if labels is not None:
        if _vector(labels, "labels") != rows:
            raise ValueError("one label per row")
        lab, lt = labels.data_ptr(), _index_code(labels)
    if weights is not None:
        if _vector(weights, "weights") != rows:
            raise ValueError("one weight per row")
        if weights.dtype != _codes["f32"]:
            raise TypeError("weights are fp32")
        wp = weights.data_ptr()
    return DistillProblem(1, _elem_code(Z), rows, vocab, top, Z.data_ptr(), ldz, ids, ld_ids, te, ld_te,
                          lab, wp, it, lt or 0, td, tau, mix, 0)


def _dz_of(Z, out):
    if out is None:
        out = _codes["empty"](Z.shape, dtype=Z.dtype, device=Z.device)
    elif out.shape != Z.shape or out.dtype != Z.dtype or out.device != Z.device:
        raise ValueError("out has another shape, type or device")
    return out, _rows_of(out, "out")[2]


def distill_loss(Z, teacher_ids, teacher, tau=1.0, mix=1.0, labels=None, weights=None, grad=False,
                 out=None, ws=None):
    """Distillation of the student's logits Z (rows x vocab) from a teacher's
    top logits: teacher_ids and teacher (rows x top), mixed with the cross
    entropy of the labels; weights (rows, fp32; zero: the row is ignored)
    default to 1 / rows.  Returns (total, rows, stats, dZ): the weighted sum,
    every row's loss, what distill_grad needs, and with grad (or out, which
    may be Z itself) the gradient of total."""
    q = _distill_problem(Z, teacher_ids, teacher, tau, mix, labels, weights)
    empty, dev, n = _codes["empty"], Z.device, q.rows
    f32 = _codes["f32"]
    total, rows = empty((), dtype=f32, device=dev), empty((n,), dtype=f32, device=dev)
    if grad or out is not None:
        dz, lddz = _dz_of(Z, out)
        stats, sp, zp = None, None, dz.data_ptr()
    else:
        stats = empty((n, 3), dtype=f32, device=dev)
        dz, lddz, sp, zp = None, 0, stats.data_ptr(), None
    ref = ctypes.byref(q)
    key = ("distill", n, q.vocab, q.top, q.dtype)
    need = _sizes.get(key)
    if need is None:
        sz = _sz()
        check(lib.pmx_distill_workspace_size(ref, ctypes.byref(sz)), "distill_workspace_size")
        need = _keep_size(key, sz.value)
    wp, wn = _ws_for(need, ws, dev)
    h, st = _call(Z.get_device())
    check(lib.pmx_distill_loss(h, ref, rows.data_ptr(), total.data_ptr(), sp, zp, lddz, wp, wn, st),
          "distill_loss")
    return total, rows, stats, dz


def distill_grad(Z, teacher_ids, teacher, stats, upstream=None, tau=1.0, mix=1.0, labels=None,
                 weights=None, out=None):
    """Gradient of distill_loss's total times `upstream` (a device fp32 scalar,
    default 1), from the stats of a distill_loss call of the same problem.  out
    may be Z itself."""
    torch = _torch()
    q = _distill_problem(Z, teacher_ids, teacher, tau, mix, labels, weights)
    _on(Z, stats, upstream)
    if tuple(stats.shape) != (q.rows, 3) or stats.dtype != torch.float32 or not stats.is_contiguous():
        raise ValueError("stats are those distill_loss returned")
    if upstream is not None and (upstream.numel() != 1 or upstream.dtype != torch.float32):
        raise ValueError("upstream is one fp32 value")
    dz, lddz = _dz_of(Z, out)
    h, st = _call(Z.get_device())
    check(lib.pmx_distill_grad(
        h, ctypes.byref(q), stats.data_ptr(),
        upstream.data_ptr() if upstream is not None else None, dz.data_ptr(), lddz,
        st), "distill_grad")
    return dz


# ---------------------------------------------------------------- expert layer
# Layer norm, the router with its balance loss, activations kept in 8 bits, and
# products of 8-bit values.

def _out_like(out, shape, dtype, device, what="out"):
    """`out`, or a new tensor; its row distance."""
    if out is None:
        return _codes["empty"](shape, dtype=dtype, device=device), max(shape[-1], 1)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError("%s has another shape or type" % what)
    return out, _rows_of(out, what)[2]


def _param(t, cols, what):
    if t is None:
        return None
    if _vector(t, what) != cols:
        raise ValueError("one value of %s per column" % what)
    return t.data_ptr()


def layer_norm(X, weight=None, bias=None, eps=1e-5, out=None, stats=None):
    """Layer norm of the rows of X (rows x cols, bf16 or fp32): returns (Y,
    stats), stats (rows x 2 fp32, mean and 1 / sqrt(variance + eps)) being what
    layer_norm_grad needs.  weight and bias (cols; both of one type, X's or
    fp32) default to ones and zeros."""
    d = _on(X, weight, bias, out, stats)
    rows, cols, ldx = _rows_of(X, "X")
    wp, bp = _param(weight, cols, "weight"), _param(bias, cols, "bias")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias have different types")
    param = weight if weight is not None else bias
    dt = _elem_code(X)
    out, ldy = _out_like(out, (rows, cols), X.dtype, X.device)
    if stats is None:
        stats = _codes["empty"]((rows, 2), dtype=_codes["f32"], device=X.device)
    elif tuple(stats.shape) != (rows, 2) or stats.dtype != _codes["f32"] or not stats.is_contiguous():
        raise ValueError("stats is rows x 2, fp32, contiguous")
    h, st = _call(d)
    check(lib.pmx_layer_norm(h, X.data_ptr(), dt, rows, cols, ldx, wp, bp,
                             dt if param is None else _elem_code(param), eps, out.data_ptr(), ldy,
                             stats.data_ptr(), st), "layer_norm")
    return out, stats


def layer_norm_grad(dY, X, stats, weight=None, params=True, out=None, dweight=None, dbias=None,
                    accumulate=False, ws=None):
    """Gradients of layer_norm: (dX, dweight, dbias), dX in X's type (out may
    be dY itself), dweight and dbias fp32 (accumulate: added to those given).
    params=False leaves the last two out (None)."""
    d = _on(dY, X, stats, weight, out, dweight, dbias)
    rows, cols, lddy = _rows_of(dY, "dY")
    rx, cx, ldx = _rows_of(X, "X")
    if (rx, cx) != (rows, cols):
        raise ValueError("dY and X have different shapes")
    if X.dtype != dY.dtype:
        raise TypeError("dY and X have different types")
    f32 = _codes["f32"]
    if tuple(stats.shape) != (rows, 2) or stats.dtype != f32 or not stats.is_contiguous():
        raise ValueError("stats are those layer_norm returned")
    wp = _param(weight, cols, "weight")
    dt = _elem_code(dY)
    out, lddx = _out_like(out, (rows, cols), X.dtype, X.device)
    need = 0
    if params:
        if accumulate and (dweight is None or dbias is None):
            raise ValueError("accumulate needs dweight and dbias")
        if dweight is None or dbias is None:
            both = _codes["empty"](2 * cols, dtype=f32, device=X.device).split_with_sizes((cols, cols))
            dweight, dbias = both[0] if dweight is None else dweight, both[1] if dbias is None else dbias
        for t in (dweight, dbias):
            if t.dtype != f32 or _vector(t, "dweight and dbias") != cols:
                raise ValueError("dweight and dbias are fp32, one value per column")
        need = _need("pmx_layer_norm_grad_workspace_size", rows, cols, dt)
    elif accumulate or dweight is not None or dbias is not None:
        raise ValueError("params=False has no dweight, dbias or accumulate")
    wsp, wn = _ws_for(need, ws, X.device)
    h, st = _call(d)
    check(lib.pmx_layer_norm_grad(
        h, dY.data_ptr(), dt, rows, cols, lddy, X.data_ptr(), ldx, stats.data_ptr(), wp,
        dt if weight is None else _elem_code(weight), out.data_ptr(), lddx,
        dweight.data_ptr() if params else None, dbias.data_ptr() if params else None,
        1 if accumulate else 0, wsp, wn, st), "layer_norm_grad")
    return out, dweight, dbias


# ids, gates, slots: rows x top; counts: experts; offsets: experts + 1; tokens:
# rows * top; loss: one value.  tally holds the counts and, last, the number of
# live tokens: what processes that balance together sum before route_grad.
Routes = collections.namedtuple("Routes", "ids gates counts offsets slots tokens loss tally")


def _route_problem(Z, top, live, balance, zloss, normalize):
    rows, experts, ldz = _rows_of(Z, "Z")
    lp = None
    if live is not None:
        if _vector(live, "live") != rows:
            raise ValueError("one live flag per row")
        if live.dtype not in (_codes["bool"], _codes["byte"]):
            raise TypeError("live is bool or uint8")
        lp = live.data_ptr()
    return RouteProblem(1, _elem_code(Z), rows, experts, top, Z.data_ptr(), ldz, lp, balance, zloss,
                        1 if normalize else 0, 0)


def route(Z, top, live=None, balance=0.0, zloss=0.0, normalize=True, order=True, ws=None):
    """Routes each row of the logits Z (rows x experts, bf16 or fp32) to its
    `top` experts: returns Routes.  ids (largest logit first, the lowest index
    among equals) and gates (softmax there, with normalize divided by their
    sum); counts and offsets of the experts; slots, the row of each pair among
    the pairs sorted by expert, and tokens, the token of each such row (-1
    behind the last): embedding(X, tokens) and offsets are what grouped_product
    takes (order=False leaves both out); loss, the balance loss plus the
    z-loss.  Rows whose live flag is 0 are not routed: ids and slots -1."""
    d = _on(Z, live)
    top = int(top)
    q = _route_problem(Z, top, live, balance, zloss, normalize)
    empty, dev = _codes["empty"], Z.device
    rows, experts = q.rows, q.experts
    if top < 0 or top >> 31:
        raise ValueError("top is out of range")
    ref = ctypes.byref(q)
    key = ("route", rows, experts, top)
    need = _sizes.get(key)
    if need is None:  # refuses sizes beyond the limits before anything of them is allocated
        sz = _sz()
        check(lib.pmx_route_workspace_size(ref, ctypes.byref(sz)), "route_workspace_size")
        need = _keep_size(key, sz.value)
    # one buffer of each type, cut up: an allocation costs the host as much as two views
    n, e1 = rows * top, experts + 1
    cuts = (n, e1, e1, n, n) if order else (n, e1, e1)
    parts = empty(sum(cuts), dtype=_codes["i32"], device=dev).split_with_sizes(cuts)
    ids, tally, offsets = parts[0].view(rows, top), parts[1], parts[2]
    slots, tokens = (parts[3].view(rows, top), parts[4]) if order else (None, None)
    gates, loss = empty(n + 1, dtype=_codes["f32"], device=dev).split_with_sizes((n, 1))
    gates, loss = gates.view(rows, top), loss.view(())
    wp, wn = _ws_for(need, ws, dev)
    h, st = _call(d)
    check(lib.pmx_route(h, ref, ids.data_ptr(), gates.data_ptr(), tally.data_ptr(), offsets.data_ptr(),
                        slots.data_ptr() if order else None, tokens.data_ptr() if order else None,
                        loss.data_ptr(), wp, wn, st), "route")
    return Routes(ids, gates, tally[:experts], offsets, slots, tokens, loss, tally)


def route_grad(Z, routes, dgates=None, upstream=None, live=None, balance=0.0, zloss=0.0, normalize=True,
               out=None):
    """Gradient of the logits from that of the gates (dgates, rows x top fp32)
    and of the loss (upstream, a device fp32 scalar, default 1), with the
    arguments of the route call.  out may be Z itself."""
    ids, gates, tally = routes.ids, routes.gates, routes.tally
    d = _on(Z, live, ids, gates, tally, dgates, upstream, out)
    shape = tuple(ids.shape)
    if len(shape) != 2 or tuple(gates.shape) != shape or shape[0] != Z.shape[0] or tally.numel() != Z.shape[1] + 1:
        raise ValueError("routes are those of a route call of the same logits")
    q = _route_problem(Z, shape[1], live, balance, zloss, normalize)
    i32, f32 = _codes["i32"], _codes["f32"]
    for t, want in ((ids, i32), (gates, f32), (tally, i32)):
        if t.dtype != want or not t.is_contiguous():
            raise ValueError("routes are those of a route call")
    if dgates is not None and (tuple(dgates.shape) != shape or dgates.dtype != f32 or not dgates.is_contiguous()):
        raise ValueError("dgates is rows x top, fp32, contiguous")
    if upstream is not None and (upstream.numel() != 1 or upstream.dtype != f32):
        raise ValueError("upstream is one fp32 value")
    dz, lddz = _dz_of(Z, out)
    h, st = _call(d)
    check(lib.pmx_route_grad(h, ctypes.byref(q), ids.data_ptr(), gates.data_ptr(), tally.data_ptr(),
                             dgates.data_ptr() if dgates is not None else None,
                             upstream.data_ptr() if upstream is not None else None, dz.data_ptr(), lddz, st),
          "route_grad")
    return dz


def _up128(n):
    return (n + 127) // 128 * 128


def _fp8_of(values, scales, halves=1):
    """(rows, padded columns, row distances) of stored rows."""
    if values.dtype != _codes["e4m3"] or scales.dtype != _codes["byte"]:
        raise TypeError("values are float8_e4m3fn and scales uint8")
    rows, wide, ldv = _rows_of(values, "values")
    rs, blocks, lds = _rows_of(scales, "scales")
    if wide % (128 * halves) or rs != rows or blocks * 128 != wide:
        raise ValueError("values are rows x a multiple of 128, scales one for each 128 of them")
    return rows, wide, ldv, lds


def _fp8_out(values, scales, rows, wide, device):
    values, ldv = _out_like(values, (rows, wide), _codes["e4m3"], device, "values")
    scales, lds = _out_like(scales, (rows, wide // 128), _codes["byte"], device, "scales")
    return values, ldv, scales, lds


def fp8_store(X, values=None, scales=None):
    """The rows of X (bf16 or fp32) in 8 bits: (values, scales), float8_e4m3fn
    of rows x cols padded with zeros to a multiple of 128, and one power of two
    for each 128 of a row as uint8, exponent + 127."""
    d = _on(X, values, scales)
    rows, cols, ldx = _rows_of(X, "X")
    dt = _elem_code(X)
    values, ldv, scales, lds = _fp8_out(values, scales, rows, _up128(cols), X.device)
    h, st = _call(d)
    check(lib.pmx_fp8_store(h, X.data_ptr(), dt, rows, cols, ldx, values.data_ptr(), ldv, scales.data_ptr(),
                            lds, st), "fp8_store")
    return values, scales


def fp8_load(values, scales, cols=None, dtype=None, out=None):
    """What fp8_store's values stand for, exactly, in bf16 (the default) or
    fp32; cols: of the stored rows (default: the padded ones)."""
    d = _on(values, scales, out)
    rows, wide, ldv, lds = _fp8_of(values, scales)
    cols = wide if cols is None else int(cols)
    if _up128(cols) != wide:
        raise ValueError("values hold another number of columns")
    if dtype is None:
        dtype = out.dtype if out is not None else _torch().bfloat16
    out, ldy = _out_like(out, (rows, cols), dtype, values.device)
    h, st = _call(d)
    check(lib.pmx_fp8_load(h, values.data_ptr(), ldv, scales.data_ptr(), lds, rows, cols, out.data_ptr(),
                           _elem_code(out), ldy, st), "fp8_load")
    return out


def _blocks_out(t, shape, dtype, device, what):
    if t is None:
        t = _codes["empty"](shape, dtype=dtype, device=device)
    elif tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError("%s has another shape or type" % what)
    return (t,) + _matrices_of(t, what)[3:]


def fp8_store_weight(W, transposed=False, values=None, scales=None):
    """Weights W (groups x n x k, or one n x k) in 8 bits with one power of two
    for each 128 x 128 tile: values groups x n x k (k padded to a multiple of
    128) and scales, or transposed, groups x k x n (n padded): the same values
    and powers, what the input gradient's fp8_product takes."""
    d = _on(W, values, scales)
    if W.dim() == 2:
        W = W.unsqueeze(0)
    groups, n, k, ldw, sw = _matrices_of(W, "W")
    dt = _elem_code(W)
    r, c = (k, n) if transposed else (n, k)
    wide = _up128(c)
    values, ldv, sv = _blocks_out(values, (groups, r, wide), _codes["e4m3"], W.device, "values")
    scales, lds, ss = _blocks_out(scales, (groups, _up128(r) // 128, wide // 128), _codes["byte"], W.device,
                                  "scales")
    h, st = _call(d)
    check(lib.pmx_fp8_store_weight(h, W.data_ptr(), dt, groups, n, k, ldw, sw, 1 if transposed else 0,
                                   values.data_ptr(), ldv, sv, scales.data_ptr(), lds, ss, st),
          "fp8_store_weight")
    return values, scales


def silu_checkpoint(H, gated=False, out=None, values=None, scales=None):
    """A = silu(H), or with gated silu of H's first half times its second, and H
    in 8 bits for the backward pass, in one go: (A, values, scales).  gated:
    each half padded to a multiple of 128 by itself."""
    d = _on(H, out, values, scales)
    rows, cols, ldh = _rows_of(H, "H")
    dt = _elem_code(H)
    halves = 2 if gated else 1
    if cols % halves:
        raise ValueError("gated needs an even number of columns")
    cols //= halves
    out, lda = _out_like(out, (rows, cols), H.dtype, H.device)
    values, ldv, scales, lds = _fp8_out(values, scales, rows, halves * _up128(cols), H.device)
    h, st = _call(d)
    check(lib.pmx_silu_checkpoint(h, H.data_ptr(), dt, rows, cols, ldh, halves - 1, out.data_ptr(), lda,
                                  values.data_ptr(), ldv, scales.data_ptr(), lds, st), "silu_checkpoint")
    return out, values, scales


def silu_checkpoint_grad(dA, values, scales, gated=False, again=True, out=None, act=None):
    """(dH, A) from the upstream dA (rows x cols) and the stored H: the gradient
    of silu_checkpoint there, and the activation once more, which is what the
    next weight's gradient takes (again=False: None)."""
    d = _on(dA, values, scales, out, act)
    rows, cols, ldda = _rows_of(dA, "dA")
    dt = _elem_code(dA)
    halves = 2 if gated else 1
    rv, wide, ldv, lds = _fp8_of(values, scales, halves)
    if rv != rows or wide != halves * _up128(cols):
        raise ValueError("values are those of another shape")
    out, lddh = _out_like(out, (rows, halves * cols), dA.dtype, dA.device)
    ap, lda = None, 0
    if again:
        act, lda = _out_like(act, (rows, cols), dA.dtype, dA.device, "act")
        ap = act.data_ptr()
    elif act is not None:
        raise ValueError("again=False has no act")
    h, st = _call(d)
    check(lib.pmx_silu_checkpoint_grad(h, dA.data_ptr(), dt, rows, cols, ldda, values.data_ptr(), ldv,
                                       scales.data_ptr(), lds, halves - 1, out.data_ptr(), lddh, ap, lda, st),
          "silu_checkpoint_grad")
    return out, act


def fp8_product(A, A_scales, B, B_scales, offsets=None, out=None, out_dtype=None):
    """C[t] = A[t] B[e]^T for the rows offsets[e] <= t < offsets[e + 1] of group
    e, rows in no group zeros: A and its scales from fp8_store (rows x k), B and
    its scales from fp8_store_weight (groups x n x k; transposed for the input
    gradient).  One group needs no offsets.  C in bf16 (the default) or fp32,
    which also chooses the precision of the sums: fp32 adds exact products in
    fp32, bf16 may lose what lies below 2^-13 of the largest of eight
    neighbouring products."""
    d = _on(A, A_scales, B, B_scales, offsets, out)
    rows, k, lda, ldas = _fp8_of(A, A_scales)
    if B.dtype != _codes["e4m3"] or B_scales.dtype != _codes["byte"]:
        raise TypeError("values are float8_e4m3fn and scales uint8")
    groups, n, kb, ldb, sb = _matrices_of(B, "B")
    gs, ns, ks, ldbs, sbs = _matrices_of(B_scales, "B_scales")
    if kb != k:
        raise ValueError("A and B disagree about k")
    if gs != groups or ns * 128 != _up128(n) or ks * 128 != k:
        raise ValueError("B_scales has one value for each 128 x 128 of B")
    op, ot = None, 0
    if offsets is None:
        if groups != 1:
            raise ValueError("several groups need offsets")
    else:
        if _vector(offsets, "offsets") != groups + 1:
            raise ValueError("one offset per group and one more")
        op, ot = offsets.data_ptr(), _index_code(offsets)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else _torch().bfloat16
    out, ldc = _out_like(out, (rows, n), out_dtype, A.device)
    h, st = _call(d)
    check(lib.pmx_fp8_product(
        h, A.data_ptr(), rows, k, lda, A_scales.data_ptr(), ldas, B.data_ptr(), n, ldb, sb,
        B_scales.data_ptr(), ldbs, sbs, op, ot, groups, out.data_ptr(), _elem_code(out), ldc, st),
        "fp8_product")
    return out
