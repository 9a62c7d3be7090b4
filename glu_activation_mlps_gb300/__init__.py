"""Python binding of the fused gated-activation library (GB300, sm_103a).

``libglu_gb300.so`` exports the C ABI declared in ``include/glu.h``.  This
module only marshals arguments: every step of the computation runs in the
library's CUDA kernels.  There is no CPU fallback; if the library has not been
built, every call raises.

Two levels:
  * ``glu_fwd`` / ``glu_bwd`` / ``glu_status_string`` / ... : the C entry points
    with the same names and arguments (raw device addresses as ints, strides
    in elements, enum codes, the stream handle as an int);
  * ``fwd`` / ``bwd`` / ...: the same calls taking torch CUDA tensors, reading
    pointers and strides from the tensors' metadata.  The 8-bit calls
    (``quantize``, ``add_rmsnorm_q``, ``gemm_q_nt``, ``gemm_q_fwd``,
    ``mlp_q_fwd``) take float8_e4m3fn tensors with float32 scales; given a
    ``stream`` they allocate what they return from that stream's memory.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libglu_gb300.so")

ACT = {"silu": 0, "gelu_erf": 1, "gelu_tanh": 2, "relu": 3}
LAYOUT = {"split": 0, "concat": 1}
DTYPE = {"f32": 0, "f16": 1, "bf16": 2}
STATUS = {0: "GLU_OK", -1: "GLU_ERR_NULL", -2: "GLU_ERR_SHAPE", -3: "GLU_ERR_STRIDE",
          -4: "GLU_ERR_ALIAS", -5: "GLU_ERR_ENUM", -6: "GLU_ERR_CUDA", -7: "GLU_ERR_WORKSPACE",
          -8: "GLU_ERR_VALUE"}

# Every symbol include/glu.h declares.
EXPORTS = ("glu_fwd", "glu_bwd", "glu_fwd_host", "glu_bwd_host", "glu_fwd_host_noalloc",
           "glu_host_workspace_bytes",
           "glu_status_string", "glu_last_cuda_error", "glu_version", "glu_last_launch",
           "glu_set_tuning", "glu_get_tuning", "glu_wait_timeouts", "glu_wait_selftest", "glu_gemm_fwd",
           "glu_gemm_nt", "glu_mlp_fwd", "glu_mlp_workspace_bytes",
           "glu_add_rmsnorm_fwd", "glu_add_rmsnorm_bwd",
           "glu_quantize", "glu_add_rmsnorm_q", "glu_gemm_q_nt", "glu_gemm_q_fwd", "glu_gemm_q_grouped_nt",
           "glu_gemm_q_grouped_fwd", "glu_mlp_q_fwd", "glu_mlp_q_workspace_bytes")


class GluError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)} ({glu_status_string(status)})"
        if status == -6:
            msg += ": " + glu_last_cuda_error()
        super().__init__(msg)


class LaunchInfo(ctypes.Structure):
    _fields_ = [("launched", ctypes.c_int32), ("backward", ctypes.c_int32),
                ("vec_bytes", ctypes.c_int32), ("unroll", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("flattened", ctypes.c_int32), ("path", ctypes.c_int32),
                ("vector_units", ctypes.c_int64), ("tail_elems", ctypes.c_int64)]


class Tuning(ctypes.Structure):
    _fields_ = [("vec_bytes", ctypes.c_int32), ("unroll", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("dependent_launch", ctypes.c_int32),
                ("path", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    from . import _build
    return _build.build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(glu_activation_mlps_gb300.build()); there is no CPU fallback")
            L = ctypes.CDLL(LIB_PATH)
            i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
            L.glu_fwd.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ci, ci, ci, vp]
            L.glu_fwd.restype = ci
            L.glu_bwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, ci, ci, ci, vp]
            L.glu_bwd.restype = ci
            sz = ctypes.c_size_t
            L.glu_fwd_host.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ci, ci, ci, vp, sz, vp, vp, vp]
            L.glu_fwd_host.restype = ci
            L.glu_bwd_host.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, ci, ci, ci,
                                       vp, sz, vp, vp, vp]
            L.glu_bwd_host.restype = ci
            L.glu_fwd_host_noalloc.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ci, ci, ci, vp]
            L.glu_fwd_host_noalloc.restype = ci
            L.glu_host_workspace_bytes.argtypes = [i64, i64, ci, ci, ci]
            L.glu_host_workspace_bytes.restype = sz
            L.glu_status_string.argtypes = [ci]
            L.glu_status_string.restype = ctypes.c_char_p
            L.glu_last_cuda_error.argtypes = []
            L.glu_last_cuda_error.restype = ctypes.c_char_p
            L.glu_version.argtypes = []
            L.glu_version.restype = ci
            L.glu_last_launch.argtypes = [ctypes.POINTER(LaunchInfo)]
            L.glu_last_launch.restype = ci
            L.glu_set_tuning.argtypes = [ctypes.POINTER(Tuning)]
            L.glu_set_tuning.restype = ci
            L.glu_get_tuning.argtypes = [ctypes.POINTER(Tuning)]
            L.glu_get_tuning.restype = ci
            L.glu_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint), ci]
            L.glu_wait_timeouts.restype = ci
            L.glu_wait_selftest.argtypes = [vp]
            L.glu_wait_selftest.restype = ci
            L.glu_gemm_fwd.argtypes = [vp, i64, vp, vp, i64, vp, i64, i64, i64, i64, ci, ci, vp]
            L.glu_gemm_fwd.restype = ci
            L.glu_gemm_nt.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, ci, vp]
            L.glu_gemm_nt.restype = ci
            L.glu_mlp_fwd.argtypes = [vp, i64, vp, vp, i64, vp, i64, vp, i64, i64, i64, i64, ci, ci, vp, sz, vp]
            L.glu_mlp_fwd.restype = ci
            L.glu_mlp_workspace_bytes.argtypes = [i64, i64, ci]
            L.glu_mlp_workspace_bytes.restype = sz
            L.glu_add_rmsnorm_fwd.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, i64,
                                              ctypes.c_float, ci, vp]
            L.glu_add_rmsnorm_fwd.restype = ci
            L.glu_add_rmsnorm_bwd.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp, i64, i64,
                                              ci, vp]
            L.glu_add_rmsnorm_bwd.restype = ci
            L.glu_quantize.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ci, ci, vp]
            L.glu_quantize.restype = ci
            L.glu_add_rmsnorm_q.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp, i64, i64,
                                            ctypes.c_float, ci, vp]
            L.glu_add_rmsnorm_q.restype = ci
            L.glu_gemm_q_nt.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, ci, vp]
            L.glu_gemm_q_nt.restype = ci
            L.glu_gemm_q_fwd.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, vp, i64, vp, i64, vp, i64, i64, i64, i64,
                                         ci, vp]
            L.glu_gemm_q_fwd.restype = ci
            L.glu_gemm_q_grouped_nt.argtypes = [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64,
                                                vp, i64, ci, vp]
            L.glu_gemm_q_grouped_nt.restype = ci
            L.glu_gemm_q_grouped_fwd.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, i64, i64, vp, i64, vp,
                                                 i64, i64, i64, i64, vp, i64, ci, vp]
            L.glu_gemm_q_grouped_fwd.restype = ci
            L.glu_mlp_q_fwd.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, i64, i64, vp, i64, i64, vp, i64,
                                        i64, vp, i64, i64, i64, i64, vp, i64, ci, ci, vp, sz, vp]
            L.glu_mlp_q_fwd.restype = ci
            L.glu_mlp_q_workspace_bytes.argtypes = [i64, i64]
            L.glu_mlp_q_workspace_bytes.restype = sz
            _lib = L
    return _lib


# ---- the C entry points -------------------------------------------------------

def glu_fwd(a, a_stride, b, b_stride, y, y_stride, n_rows, n_cols, layout, act, dtype, stream) -> int:
    return lib().glu_fwd(a, a_stride, b, b_stride, y, y_stride, n_rows, n_cols,
                         layout, act, dtype, stream)


def glu_bwd(dc, dc_stride, a, a_stride, b, b_stride, da, da_stride, db, db_stride,
            n_rows, n_cols, layout, act, dtype, stream) -> int:
    return lib().glu_bwd(dc, dc_stride, a, a_stride, b, b_stride, da, da_stride, db, db_stride,
                         n_rows, n_cols, layout, act, dtype, stream)


def glu_fwd_host(a, a_stride, b, b_stride, y, y_stride, n_rows, n_cols, layout, act, dtype,
                 workspace, workspace_bytes, copy_in, compute, copy_out) -> int:
    return lib().glu_fwd_host(a, a_stride, b, b_stride, y, y_stride, n_rows, n_cols, layout, act, dtype,
                              workspace, workspace_bytes, copy_in, compute, copy_out)


def glu_bwd_host(dc, dc_stride, a, a_stride, b, b_stride, da, da_stride, db, db_stride, n_rows, n_cols,
                 layout, act, dtype, workspace, workspace_bytes, copy_in, compute, copy_out) -> int:
    return lib().glu_bwd_host(dc, dc_stride, a, a_stride, b, b_stride, da, da_stride, db, db_stride,
                              n_rows, n_cols, layout, act, dtype, workspace, workspace_bytes,
                              copy_in, compute, copy_out)


def glu_fwd_host_noalloc(a, a_stride, b, b_stride, y, y_stride, n_rows, n_cols, layout, act, dtype,
                         stream) -> int:
    """glu_fwd_host staged through the library's own fixed device array: for
    callers that cannot allocate device memory (see include/glu.h)."""
    return lib().glu_fwd_host_noalloc(a, a_stride, b, b_stride, y, y_stride, n_rows, n_cols, layout,
                                      act, dtype, stream)


def glu_host_workspace_bytes(rows_per_block, n_cols, layout, dtype, backward) -> int:
    return lib().glu_host_workspace_bytes(rows_per_block, n_cols, layout, dtype, backward)


def glu_status_string(status: int) -> str:
    return lib().glu_status_string(status).decode()


def glu_last_cuda_error() -> str:
    return lib().glu_last_cuda_error().decode()


def glu_version() -> int:
    return lib().glu_version()


def glu_last_launch() -> dict:
    info = LaunchInfo()
    st = lib().glu_last_launch(ctypes.byref(info))
    if st:
        raise GluError(st, "glu_last_launch")
    return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}


def glu_set_tuning(vec_bytes: int = 0, unroll: int = 0, ctas_per_sm: int = 0,
                   dependent_launch: int = 0, path: int = 0) -> None:
    t = Tuning(vec_bytes, unroll, ctas_per_sm, dependent_launch, path)
    st = lib().glu_set_tuning(ctypes.byref(t))
    if st:
        raise GluError(st, "glu_set_tuning")


def glu_wait_timeouts(reset: bool = False) -> int:
    c = ctypes.c_uint(0)
    st = lib().glu_wait_timeouts(ctypes.byref(c), int(reset))
    if st:
        raise GluError(st, "glu_wait_timeouts")
    return c.value


def glu_wait_selftest(stream=None) -> None:
    """Enqueue the bounded-wait self-test (one warp whose wait nothing
    completes; it returns after about a second and counts one timeout)."""
    st = lib().glu_wait_selftest(_stream(stream))
    if st:
        raise GluError(st, "glu_wait_selftest")


def glu_gemm_fwd(x, x_stride, w_gate, w_up, w_stride, y, y_stride, M, K, I, act, dtype, stream) -> int:
    return lib().glu_gemm_fwd(x, x_stride, w_gate, w_up, w_stride, y, y_stride, M, K, I, act, dtype, stream)


def glu_gemm_nt(a, a_stride, b, b_stride, d, d_stride, M, K, N, dtype, stream) -> int:
    return lib().glu_gemm_nt(a, a_stride, b, b_stride, d, d_stride, M, K, N, dtype, stream)


def glu_mlp_fwd(x, x_stride, w_gate, w_up, w_stride, w_down, w_down_stride, out, out_stride, M, H, I, act, dtype,
                workspace, workspace_bytes, stream) -> int:
    return lib().glu_mlp_fwd(x, x_stride, w_gate, w_up, w_stride, w_down, w_down_stride, out, out_stride, M, H, I,
                             act, dtype, workspace, workspace_bytes, stream)


def glu_mlp_workspace_bytes(M, I, dtype) -> int:
    return lib().glu_mlp_workspace_bytes(M, I, dtype)


def glu_add_rmsnorm_fwd(x, x_stride, residual, res_stride, gamma, h, h_stride, y, y_stride, rstd,
                        n_rows, n_cols, eps, dtype, stream) -> int:
    return lib().glu_add_rmsnorm_fwd(x, x_stride, residual, res_stride, gamma, h, h_stride, y, y_stride, rstd,
                                     n_rows, n_cols, eps, dtype, stream)


def glu_add_rmsnorm_bwd(dy, dy_stride, h, h_stride, rstd, gamma, dh, dh_stride, dx, dx_stride, dres, dres_stride,
                        dgamma, n_rows, n_cols, dtype, stream) -> int:
    return lib().glu_add_rmsnorm_bwd(dy, dy_stride, h, h_stride, rstd, gamma, dh, dh_stride, dx, dx_stride, dres,
                                     dres_stride, dgamma, n_rows, n_cols, dtype, stream)


def glu_quantize(x, x_stride, q, q_stride, scale, scale_stride, n_rows, n_cols, block_rows, dtype, stream) -> int:
    return lib().glu_quantize(x, x_stride, q, q_stride, scale, scale_stride, n_rows, n_cols, block_rows, dtype, stream)


def glu_add_rmsnorm_q(x, x_stride, residual, res_stride, gamma, h, h_stride, q, q_stride, scale, scale_stride, rstd,
                      n_rows, n_cols, eps, dtype, stream) -> int:
    return lib().glu_add_rmsnorm_q(x, x_stride, residual, res_stride, gamma, h, h_stride, q, q_stride, scale,
                                   scale_stride, rstd, n_rows, n_cols, eps, dtype, stream)


def glu_gemm_q_nt(a, a_stride, a_scale, a_scale_stride, b, b_stride, b_scale, b_scale_stride, d, d_stride, M, K, N,
                  dtype, stream) -> int:
    return lib().glu_gemm_q_nt(a, a_stride, a_scale, a_scale_stride, b, b_stride, b_scale, b_scale_stride, d,
                               d_stride, M, K, N, dtype, stream)


def glu_gemm_q_fwd(x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, gate_scale, up_scale, w_scale_stride,
                   y, y_stride, y_scale, y_scale_stride, M, K, I, act, stream) -> int:
    return lib().glu_gemm_q_fwd(x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, gate_scale, up_scale,
                                w_scale_stride, y, y_stride, y_scale, y_scale_stride, M, K, I, act, stream)


def glu_gemm_q_grouped_nt(a, a_stride, a_scale, a_scale_stride, b, b_stride, b_group, b_scale, b_scale_stride,
                          b_scale_group, d, d_stride, M, K, N, offsets, n_groups, dtype, stream) -> int:
    return lib().glu_gemm_q_grouped_nt(a, a_stride, a_scale, a_scale_stride, b, b_stride, b_group, b_scale,
                                       b_scale_stride, b_scale_group, d, d_stride, M, K, N, offsets, n_groups, dtype,
                                       stream)


def glu_gemm_q_grouped_fwd(x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, w_group, gate_scale,
                           up_scale, w_scale_stride, w_scale_group, y, y_stride, y_scale, y_scale_stride, M, K, I,
                           offsets, n_groups, act, stream) -> int:
    return lib().glu_gemm_q_grouped_fwd(x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, w_group,
                                        gate_scale, up_scale, w_scale_stride, w_scale_group, y, y_stride, y_scale,
                                        y_scale_stride, M, K, I, offsets, n_groups, act, stream)


def glu_mlp_q_fwd(x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, w_group, gate_scale, up_scale,
                  w_scale_stride, w_scale_group, w_down, w_down_stride, w_down_group, down_scale, down_scale_stride,
                  down_scale_group, out, out_stride, M, H, I, offsets, n_groups, act, dtype, workspace,
                  workspace_bytes, stream) -> int:
    return lib().glu_mlp_q_fwd(x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, w_group, gate_scale,
                               up_scale, w_scale_stride, w_scale_group, w_down, w_down_stride, w_down_group,
                               down_scale, down_scale_stride, down_scale_group, out, out_stride, M, H, I, offsets,
                               n_groups, act, dtype, workspace, workspace_bytes, stream)


def glu_mlp_q_workspace_bytes(M, I) -> int:
    return lib().glu_mlp_q_workspace_bytes(M, I)


def glu_get_tuning() -> dict:
    t = Tuning()
    st = lib().glu_get_tuning(ctypes.byref(t))
    if st:
        raise GluError(st, "glu_get_tuning")
    return {"vec_bytes": t.vec_bytes, "unroll": t.unroll, "ctas_per_sm": t.ctas_per_sm,
            "dependent_launch": t.dependent_launch, "path": t.path}


# ---- torch tensor marshalling -------------------------------------------------

def _dtype_code(t) -> int:
    import torch
    m = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if t.dtype not in m:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32, float16 or bfloat16")
    return m[t.dtype]


def _rows(t, name):
    """(n_rows, row stride) of a tensor viewed as a matrix over its last dim."""
    if t.dim() < 1 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor with at least one dimension")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if t.dim() == 1:
        return 1, t.shape[0]
    lead = t.shape[:-1]
    # leading dims must collapse to one row index with a single stride
    stride = t.stride(-2)
    expect = stride
    for d in range(t.dim() - 2, -1, -1):
        if t.shape[d] != 1 and t.stride(d) != expect:
            raise ValueError(f"{name}: leading dimensions do not collapse to one row stride")
        expect *= t.shape[d]
    n = 1
    for s in lead:
        n *= s
    return n, stride


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def fwd(a, b=None, *, y=None, act: str = "silu", layout: str = "split", stream=None):
    """y = act(a) * b on CUDA tensors.  SPLIT: a, b of one shape (..., I).
    CONCAT: a is x of shape (..., 2I), b is None.  ``y`` may be given (also as
    b, or as x[..., I:], for in-place); otherwise it is allocated."""
    import torch
    if layout not in LAYOUT:
        raise ValueError(layout)
    concat = layout == "concat"
    n_rows, a_stride = _rows(a, "a")
    if concat:
        if a.shape[-1] % 2:
            raise ValueError("concat input needs an even last dimension")
        n_cols = a.shape[-1] // 2
        b_ptr, b_stride = None, 0
        out_shape = (*a.shape[:-1], n_cols)
    else:
        if b is None or b.shape != a.shape or b.dtype != a.dtype:
            raise ValueError("b must match a in shape and dtype")
        n_cols = a.shape[-1]
        _, b_stride = _rows(b, "b")
        b_ptr = b.data_ptr()
        out_shape = a.shape
    if y is None:
        y = torch.empty(out_shape, dtype=a.dtype, device=a.device)
    if tuple(y.shape) != tuple(out_shape) or y.dtype != a.dtype:
        raise ValueError("y has the wrong shape or dtype")
    _, y_stride = _rows(y, "y")
    st = glu_fwd(a.data_ptr(), a_stride, b_ptr, b_stride, y.data_ptr(), y_stride,
                 n_rows, n_cols, LAYOUT[layout], ACT[act], _dtype_code(a), _stream(stream))
    if st:
        raise GluError(st, "glu_fwd")
    return y


def bwd(dc, a, b=None, *, da=None, db=None, act: str = "silu", layout: str = "split",
        inplace: bool = False, stream=None):
    """(da, db) = (dc * act'(a) * b, dc * act(a)).  SPLIT returns (da, db);
    CONCAT (a = x, b None) returns dx = [da | db].  ``inplace`` writes da over
    a and db over b (dx over x)."""
    import torch
    concat = layout == "concat"
    n_rows, a_stride = _rows(a, "a")
    _, dc_stride = _rows(dc, "dc")
    code = _dtype_code(a)
    if concat:
        n_cols = a.shape[-1] // 2
        if dc.shape[-1] != n_cols:
            raise ValueError("dc must have half the width of x")
        dx = a if inplace else (da if da is not None else torch.empty_like(a))
        _, dx_stride = _rows(dx, "dx")
        st = glu_bwd(dc.data_ptr(), dc_stride, a.data_ptr(), a_stride, None, 0,
                     dx.data_ptr(), dx_stride, None, 0, n_rows, n_cols,
                     LAYOUT[layout], ACT[act], code, _stream(stream))
        if st:
            raise GluError(st, "glu_bwd")
        return dx
    if b is None or b.shape != a.shape or dc.shape != a.shape:
        raise ValueError("dc, a and b must have one shape")
    n_cols = a.shape[-1]
    _, b_stride = _rows(b, "b")
    if inplace:
        da, db = a, b
    da = da if da is not None else torch.empty_like(a)
    db = db if db is not None else torch.empty_like(b)
    _, da_stride = _rows(da, "da")
    _, db_stride = _rows(db, "db")
    st = glu_bwd(dc.data_ptr(), dc_stride, a.data_ptr(), a_stride, b.data_ptr(), b_stride,
                 da.data_ptr(), da_stride, db.data_ptr(), db_stride, n_rows, n_cols,
                 LAYOUT[layout], ACT[act], code, _stream(stream))
    if st:
        raise GluError(st, "glu_bwd")
    return da, db


def gemm_fwd(x, w_gate, w_up, *, y=None, act: str = "silu", stream=None):
    """y = act(x @ w_gate^T) * (x @ w_up^T) on the tensor cores, the activation
    applied in the GEMM epilogue.  x is (..., K); the weights are (I, K) in the
    nn.Linear layout and share one row stride; f16 or bf16."""
    import torch
    n_rows, x_stride = _rows(x, "x")
    if w_gate.dim() != 2 or w_up.shape != w_gate.shape or w_gate.shape[1] != x.shape[-1]:
        raise ValueError("w_gate and w_up must both be (I, K) with K = x.shape[-1]")
    if w_gate.dtype != x.dtype or w_up.dtype != x.dtype:
        raise ValueError("x and the weights must have one dtype")
    _, wg_stride = _rows(w_gate, "w_gate")
    _, wu_stride = _rows(w_up, "w_up")
    if wg_stride != wu_stride:
        raise ValueError("w_gate and w_up must have one row stride")
    n_out, K = w_gate.shape
    if y is None:
        y = torch.empty((*x.shape[:-1], n_out), dtype=x.dtype, device=x.device)
    if tuple(y.shape) != (*x.shape[:-1], n_out) or y.dtype != x.dtype:
        raise ValueError("y has the wrong shape or dtype")
    _, y_stride = _rows(y, "y")
    st = glu_gemm_fwd(x.data_ptr(), x_stride, w_gate.data_ptr(), w_up.data_ptr(), wg_stride,
                      y.data_ptr(), y_stride, n_rows, K, n_out, ACT[act], _dtype_code(x), _stream(stream))
    if st:
        raise GluError(st, "glu_gemm_fwd")
    return y


def gemm_nt(a, b, *, d=None, stream=None):
    """d = a @ b^T on the tensor cores (the MLP's down projection).  a is
    (..., K); b is (N, K) in the nn.Linear layout; f16 or bf16."""
    import torch
    n_rows, a_stride = _rows(a, "a")
    if b.dim() != 2 or b.shape[1] != a.shape[-1] or b.dtype != a.dtype:
        raise ValueError("b must be (N, K) with K = a.shape[-1] and a's dtype")
    _, b_stride = _rows(b, "b")
    N, K = b.shape
    if d is None:
        d = torch.empty((*a.shape[:-1], N), dtype=a.dtype, device=a.device)
    if tuple(d.shape) != (*a.shape[:-1], N) or d.dtype != a.dtype:
        raise ValueError("d has the wrong shape or dtype")
    _, d_stride = _rows(d, "d")
    st = glu_gemm_nt(a.data_ptr(), a_stride, b.data_ptr(), b_stride, d.data_ptr(), d_stride, n_rows, K, N,
                     _dtype_code(a), _stream(stream))
    if st:
        raise GluError(st, "glu_gemm_nt")
    return d


def mlp_fwd(x, w_gate, w_up, w_down, *, out=None, act: str = "silu", workspace=None, stream=None):
    """out = (act(x @ w_gate^T) * (x @ w_up^T)) @ w_down^T; x is (..., H), the
    gate and up weights (I, H), the down weights (H, I).  The workspace (a
    uint8 device tensor) is allocated here when not given."""
    import torch
    n_rows, x_stride = _rows(x, "x")
    H = x.shape[-1]
    if w_gate.dim() != 2 or w_up.shape != w_gate.shape or w_gate.shape[1] != H:
        raise ValueError("w_gate and w_up must both be (I, H)")
    I = w_gate.shape[0]
    if tuple(w_down.shape) != (H, I):
        raise ValueError("w_down must be (H, I)")
    if any(w.dtype != x.dtype for w in (w_gate, w_up, w_down)):
        raise ValueError("x and the weights must have one dtype")
    _, wg_stride = _rows(w_gate, "w_gate")
    _, wu_stride = _rows(w_up, "w_up")
    if wg_stride != wu_stride:
        raise ValueError("w_gate and w_up must have one row stride")
    _, wd_stride = _rows(w_down, "w_down")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _, out_stride = _rows(out, "out")
    code = _dtype_code(x)
    if workspace is None:
        workspace = torch.empty(max(16, glu_mlp_workspace_bytes(max(n_rows, 1), max(I, 1), code)),
                                dtype=torch.uint8, device=x.device)
    st = glu_mlp_fwd(x.data_ptr(), x_stride, w_gate.data_ptr(), w_up.data_ptr(), wg_stride, w_down.data_ptr(),
                     wd_stride, out.data_ptr(), out_stride, n_rows, H, I, ACT[act], code, workspace.data_ptr(),
                     workspace.numel(), _stream(stream))
    if st:
        raise GluError(st, "glu_mlp_fwd")
    return out


def add_rmsnorm(x, residual, gamma, eps: float = 1e-5, *, h=None, y=None, rstd=None, stream=None):
    """h = x + residual and y = rmsnorm(h) * gamma over the last dimension, in one
    pass.  ``h`` and ``y`` may be given (h may be x or residual for an in-place
    residual update, y the other one); ``rstd`` may be a float32 tensor of one
    entry per row, or True to allocate it.  Returns (h, y) or (h, y, rstd)."""
    import torch
    n_rows, x_stride = _rows(x, "x")
    _, r_stride = _rows(residual, "residual")
    if residual.shape != x.shape or residual.dtype != x.dtype:
        raise ValueError("residual must match x in shape and dtype")
    H = x.shape[-1]
    if gamma.shape != (H,) or gamma.dtype != x.dtype or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous (H,) tensor of x's dtype")
    h = torch.empty_like(x) if h is None else h
    y = torch.empty_like(x) if y is None else y
    for t, n in ((h, "h"), (y, "y")):
        if t.shape != x.shape or t.dtype != x.dtype:
            raise ValueError(f"{n} must match x in shape and dtype")
    _, h_stride = _rows(h, "h")
    _, y_stride = _rows(y, "y")
    want_rstd = rstd is not None and rstd is not False
    if rstd is True:
        rstd = torch.empty(n_rows, dtype=torch.float32, device=x.device)
    if want_rstd and (rstd.dtype != torch.float32 or rstd.numel() != n_rows or not rstd.is_contiguous()):
        raise ValueError("rstd must be a contiguous float32 tensor with one entry per row")
    st = glu_add_rmsnorm_fwd(x.data_ptr(), x_stride, residual.data_ptr(), r_stride, gamma.data_ptr(),
                             h.data_ptr(), h_stride, y.data_ptr(), y_stride,
                             rstd.data_ptr() if want_rstd else None, n_rows, H, float(eps),
                             _dtype_code(x), _stream(stream))
    if st:
        raise GluError(st, "glu_add_rmsnorm_fwd")
    return (h, y, rstd) if want_rstd else (h, y)


def add_rmsnorm_bwd(dy, h, rstd, gamma, *, dh=None, dx=None, dres=None, dgamma=None, stream=None):
    """Gradients of add_rmsnorm: dx (= the residual's gradient) from dy, the
    stored sum h and rstd, plus dh if h also feeds the residual stream.  ``dres``
    may be a tensor receiving a second copy; ``dgamma`` a float32 (H,) tensor
    the row sums are added to, or True for a zeroed one.  Returns dx, or
    (dx, dgamma) when dgamma is requested."""
    import torch
    n_rows, dy_stride = _rows(dy, "dy")
    _, h_stride = _rows(h, "h")
    H = dy.shape[-1]
    if h.shape != dy.shape or h.dtype != dy.dtype:
        raise ValueError("h must match dy")
    if gamma.shape != (H,) or gamma.dtype != dy.dtype or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous (H,) tensor of dy's dtype")
    if rstd.dtype != torch.float32 or rstd.numel() != n_rows or not rstd.is_contiguous():
        raise ValueError("rstd must be a contiguous float32 tensor with one entry per row")
    dx = torch.empty_like(dy) if dx is None else dx
    _, dx_stride = _rows(dx, "dx")
    dh_ptr, dh_stride = (None, 0) if dh is None else (dh.data_ptr(), _rows(dh, "dh")[1])
    dr_ptr, dr_stride = (None, 0) if dres is None else (dres.data_ptr(), _rows(dres, "dres")[1])
    want_dg = dgamma is not None and dgamma is not False
    if dgamma is True:
        dgamma = torch.zeros(H, dtype=torch.float32, device=dy.device)
    if want_dg and (dgamma.dtype != torch.float32 or dgamma.shape != (H,) or not dgamma.is_contiguous()):
        raise ValueError("dgamma must be a contiguous float32 (H,) tensor")
    st = glu_add_rmsnorm_bwd(dy.data_ptr(), dy_stride, h.data_ptr(), h_stride, rstd.data_ptr(), gamma.data_ptr(),
                             dh_ptr, dh_stride, dx.data_ptr(), dx_stride, dr_ptr, dr_stride,
                             dgamma.data_ptr() if want_dg else None, n_rows, H, _dtype_code(dy), _stream(stream))
    if st:
        raise GluError(st, "glu_add_rmsnorm_bwd")
    return (dx, dgamma) if want_dg else dx


# ---- 8-bit floating point ----------------------------------------------------------

def _same_device(x, *others) -> int:
    """The index of x's device, which holds every other tensor and is the
    current one (the device the library launches on)."""
    import torch
    dev = x.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("the tensors must be on the current CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")
    return dev


def _raw_stream(dev: int) -> int:
    """The handle of the device's current stream."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev)


def _on_stream(stream, call, *args, **kw):
    """call(*args, **kw) with ``stream`` (a torch stream or a handle) current, so
    that what it allocates is that stream's memory: memory of the current stream
    may still be written by work queued there.  The allocator is told who uses
    what on a stream not its own, so that nothing is given out again too early.
    The caller orders the two streams' work on the operands and the results."""
    import torch
    if not isinstance(stream, torch.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream))
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for t in (*args, *kw.values()):
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    for t in (out,) if isinstance(out, torch.Tensor) else out:
        t.record_stream(here)
    return out


def _mat(t, name):
    """_rows of a CUDA tensor, quick for plain matrices."""
    if t.dim() == 2:
        stride, inner = t.stride()
        if inner == 1 or t.shape[1] <= 1:
            return t.shape[0], stride
    return _rows(t, name)


def _out_q(q, scale, shape, lead, like, name):
    """(q, scale, row stride of q, row stride of scale) of a result of the given
    shape (``lead``: its leading dimensions) quantised by rows.  What is None is
    allocated, q with rows on 16-byte boundaries (the products' rule)."""
    import torch
    n = shape[-1]
    groups = (n + 127) // 128
    if q is None:
        q_stride = n + -n % 16
        if q_stride == n:
            q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=like.device)
        elif len(shape) == 2:
            q = torch.empty_strided(shape, (q_stride, 1), dtype=torch.float8_e4m3fn, device=like.device)
        else:
            q = torch.empty((*lead, q_stride), dtype=torch.float8_e4m3fn, device=like.device)[..., :n]
    elif q.dtype != torch.float8_e4m3fn or q.shape != shape:
        raise ValueError(f"{name} must be float8_e4m3fn of shape {tuple(shape)}")
    else:
        q_stride = _mat(q, name)[1]
    if scale is None:
        scale = torch.empty((*lead, groups), dtype=torch.float32, device=like.device)
        return q, scale, q_stride, groups
    if scale.dtype != torch.float32 or scale.shape != (*lead, groups):
        raise ValueError(f"{name}'s scales must be float32 of shape {(*lead, groups)}")
    return q, scale, q_stride, _mat(scale, name)[1]


def _in_q(q, scale, name):
    """(n_rows, row stride, scale's row stride, K) of a matrix quantised by rows."""
    import torch
    if q.dtype != torch.float8_e4m3fn or scale.dtype != torch.float32:
        raise TypeError(f"{name} must be float8_e4m3fn with float32 scales")
    shape = q.shape
    K = shape[-1]
    if scale.shape != (*shape[:-1], (K + 127) // 128):
        raise ValueError(f"{name}'s scales must have shape {(*shape[:-1], (K + 127) // 128)}")
    n_rows, stride = _mat(q, name)
    return n_rows, stride, _mat(scale, name)[1], K


def _weight_q(w, s, K, name, grouped):
    """(N, row stride, expert stride, scale's row stride, scale's expert stride) of (N, K) or (E, N, K) weights."""
    import torch
    if w.dtype != torch.float8_e4m3fn or s.dtype != torch.float32:
        raise TypeError(f"{name} must be float8_e4m3fn with float32 scales")
    shape = w.shape
    if len(shape) != (3 if grouped else 2) or shape[-1] != K:
        raise ValueError(f"{name} must be {'(E, N, K)' if grouped else '(N, K)'} with K = {K}")
    N = shape[-2]
    if s.shape != (*shape[:-2], (N + 127) // 128, (K + 127) // 128):
        raise ValueError(f"{name}'s scales must have shape {(*shape[:-2], (N + 127) // 128, (K + 127) // 128)}")
    ws, ss = w.stride(), s.stride()
    if (ws[-1] != 1 and K > 1) or (ss[-1] != 1 and K > 128):
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return (N, ws[0], 0, ss[0], 0) if not grouped else (N, ws[1], ws[0], ss[1], ss[0])


def _offsets(offsets, w):
    import torch
    if offsets.dtype != torch.int32 or not offsets.is_contiguous() or offsets.shape != (w.shape[0] + 1,):
        raise ValueError("offsets must be a contiguous int32 tensor of one entry more than there are experts")
    return offsets.data_ptr()


def quantize(x, *, block_rows: int = 1, q=None, scale=None, stream=None):
    """(q, scale) of x in e4m3 with a float32 scale for each block of 128
    columns: of one row (``block_rows`` = 1, activations; x is (..., K) and
    scale (..., ceil(K / 128))), or of 128 rows (128, weights; x is (N, K), or
    (E, N, K) for the weights of E experts, and scale (.., ceil(N / 128),
    ceil(K / 128)))."""
    import torch
    if stream is not None:
        return _on_stream(stream, quantize, x, block_rows=block_rows, q=q, scale=scale)
    code = _dtype_code(x)
    shape = x.shape
    dev = _same_device(x, q, scale)
    s = _raw_stream(dev)
    if block_rows == 1:
        n_rows, x_stride = _mat(x, "x")
        q, scale, q_stride, s_stride = _out_q(q, scale, shape, shape[:-1], x, "q")
        st = glu_quantize(x.data_ptr(), x_stride, q.data_ptr(), q_stride, scale.data_ptr(), s_stride, n_rows,
                          shape[-1], 1, code, s)
        if st:
            raise GluError(st, "glu_quantize")
        return q, scale
    if block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    if len(shape) not in (2, 3):
        raise ValueError("x must be (N, K) or (E, N, K) for 128 x 128 blocks")
    K = shape[-1]
    blocks = (*shape[:-2], (shape[-2] + 127) // 128, (K + 127) // 128)
    if scale is None:
        scale = torch.empty(blocks, dtype=torch.float32, device=x.device)
    elif scale.dtype != torch.float32 or scale.shape != blocks:
        raise ValueError(f"q's scales must be float32 of shape {blocks}")
    if q is None:
        wide = K + -K % 16              # rows on 16-byte boundaries, the products' rule
        strides = (wide, 1) if len(shape) == 2 else (shape[1] * wide, wide, 1)
        q = torch.empty_strided(shape, strides, dtype=torch.float8_e4m3fn, device=x.device)
    elif q.dtype != torch.float8_e4m3fn or q.shape != shape:
        raise ValueError(f"q must be float8_e4m3fn of shape {tuple(shape)}")
    for xe, qe, se in (((x, q, scale),) if len(shape) == 2 else zip(x, q, scale)):
        n_rows, x_stride = _mat(xe, "x")
        st = glu_quantize(xe.data_ptr(), x_stride, qe.data_ptr(), _mat(qe, "q")[1], se.data_ptr(),
                          _mat(se, "scale")[1], n_rows, K, 128, code, s)
        if st:
            raise GluError(st, "glu_quantize")
    return q, scale


def add_rmsnorm_q(x, residual, gamma, eps: float = 1e-5, *, h=None, q=None, scale=None, rstd=None, stream=None):
    """h = x + residual, and rmsnorm(h) * gamma over the last dimension as
    (q, scale): e4m3 with a float32 scale for each 128 columns of a row, in one
    pass.  ``h`` may be x or residual; ``rstd`` as in add_rmsnorm.  Returns
    (h, q, scale) or (h, q, scale, rstd)."""
    import torch
    if stream is not None:
        return _on_stream(stream, add_rmsnorm_q, x, residual, gamma, eps, h=h, q=q, scale=scale, rstd=rstd)
    dev = _same_device(x, residual, gamma, h, q, scale)
    code = _dtype_code(x)
    shape, dtype = x.shape, x.dtype
    H = shape[-1]
    if residual.shape != shape or residual.dtype != dtype:
        raise ValueError("residual must match x in shape and dtype")
    if gamma.shape != (H,) or gamma.dtype != dtype or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous (H,) tensor of x's dtype")
    n_rows, x_stride = _mat(x, "x")
    r_stride = _mat(residual, "residual")[1]
    if h is None:
        h, h_stride = torch.empty(shape, dtype=dtype, device=x.device), H
    elif h.shape != shape or h.dtype != dtype:
        raise ValueError("h must match x in shape and dtype")
    else:
        h_stride = _mat(h, "h")[1]
    q, scale, q_stride, s_stride = _out_q(q, scale, shape, shape[:-1], x, "q")
    if rstd is None or rstd is False:
        rstd = None
    elif rstd is True:
        rstd = torch.empty(n_rows, dtype=torch.float32, device=x.device)
    elif (rstd.dtype != torch.float32 or rstd.numel() != n_rows or not rstd.is_contiguous() or
          rstd.get_device() != dev):
        raise ValueError("rstd must be a contiguous float32 tensor with one entry per row")
    st = glu_add_rmsnorm_q(x.data_ptr(), x_stride, residual.data_ptr(), r_stride, gamma.data_ptr(), h.data_ptr(),
                           h_stride, q.data_ptr(), q_stride, scale.data_ptr(), s_stride,
                           None if rstd is None else rstd.data_ptr(), n_rows, H, eps, code, _raw_stream(dev))
    if st:
        raise GluError(st, "glu_add_rmsnorm_q")
    return (h, q, scale) if rstd is None else (h, q, scale, rstd)


def gemm_q_nt(a, a_scale, b, b_scale, *, d=None, dtype=None, offsets=None, stream=None):
    """d = a @ b^T of quantised matrices on the tensor cores, in ``dtype``
    (float16 or bfloat16, the default; d's when d is given).  a is (..., K) with
    scales by rows, b (N, K) with scales by 128 x 128 blocks.  With ``offsets``
    (int32, E + 1 entries, on the device) b is (E, N, K) and a's rows offsets[e]
    .. offsets[e + 1] are multiplied by b[e]; rows of d that no expert has are
    left as they were."""
    import torch
    if stream is not None:
        return _on_stream(stream, gemm_q_nt, a, a_scale, b, b_scale, d=d, dtype=dtype, offsets=offsets)
    dev = _same_device(a, a_scale, b, b_scale, d, offsets)
    n_rows, a_stride, as_stride, K = _in_q(a, a_scale, "a")
    N, b_stride, b_group, bs_stride, bs_group = _weight_q(b, b_scale, K, "b", offsets is not None)
    shape = (*a.shape[:-1], N)
    if d is None:
        d, d_stride = torch.empty(shape, dtype=dtype or torch.bfloat16, device=a.device), N
    elif d.shape != shape or (dtype is not None and d.dtype != dtype):
        raise ValueError("d has the wrong shape or dtype")
    else:
        d_stride = _mat(d, "d")[1]
    code = _dtype_code(d)
    s = _raw_stream(dev)
    if offsets is None:
        st = glu_gemm_q_nt(a.data_ptr(), a_stride, a_scale.data_ptr(), as_stride, b.data_ptr(), b_stride,
                           b_scale.data_ptr(), bs_stride, d.data_ptr(), d_stride, n_rows, K, N, code, s)
    else:
        st = glu_gemm_q_grouped_nt(a.data_ptr(), a_stride, a_scale.data_ptr(), as_stride, b.data_ptr(), b_stride,
                                   b_group, b_scale.data_ptr(), bs_stride, bs_group, d.data_ptr(), d_stride, n_rows,
                                   K, N, _offsets(offsets, b), b.shape[0], code, s)
    if st:
        raise GluError(st, "glu_gemm_q_nt" if offsets is None else "glu_gemm_q_grouped_nt")
    return d


def gemm_q_fwd(x, x_scale, w_gate, gate_scale, w_up, up_scale, *, y=None, y_scale=None, act: str = "silu",
               offsets=None, stream=None):
    """(y, y_scale): act(x @ w_gate^T) * (x @ w_up^T) of quantised matrices, on
    the tensor cores, quantised by rows in the epilogue.  x is (..., K), the
    weights (I, K) with one row stride, or (E, I, K) with ``offsets`` (see
    gemm_q_nt)."""
    if stream is not None:
        return _on_stream(stream, gemm_q_fwd, x, x_scale, w_gate, gate_scale, w_up, up_scale, y=y, y_scale=y_scale,
                          act=act, offsets=offsets)
    dev = _same_device(x, x_scale, w_gate, gate_scale, w_up, up_scale, y, y_scale, offsets)
    n_rows, x_stride, xs_stride, K = _in_q(x, x_scale, "x")
    gate = _weight_q(w_gate, gate_scale, K, "w_gate", offsets is not None)
    if w_up.shape != w_gate.shape or _weight_q(w_up, up_scale, K, "w_up", offsets is not None) != gate:
        raise ValueError("w_gate and w_up (and their scales) must have one shape and one stride")
    N, w_stride, w_group, s_stride, s_group = gate
    lead = x.shape[:-1]
    y, y_scale, y_stride, ys_stride = _out_q(y, y_scale, (*lead, N), lead, x, "y")
    s = _raw_stream(dev)
    if offsets is None:
        st = glu_gemm_q_fwd(x.data_ptr(), x_stride, x_scale.data_ptr(), xs_stride, w_gate.data_ptr(), w_up.data_ptr(),
                            w_stride, gate_scale.data_ptr(), up_scale.data_ptr(), s_stride, y.data_ptr(), y_stride,
                            y_scale.data_ptr(), ys_stride, n_rows, K, N, ACT[act], s)
    else:
        st = glu_gemm_q_grouped_fwd(x.data_ptr(), x_stride, x_scale.data_ptr(), xs_stride, w_gate.data_ptr(),
                                    w_up.data_ptr(), w_stride, w_group, gate_scale.data_ptr(), up_scale.data_ptr(),
                                    s_stride, s_group, y.data_ptr(), y_stride, y_scale.data_ptr(), ys_stride, n_rows,
                                    K, N, _offsets(offsets, w_gate), w_gate.shape[0], ACT[act], s)
    if st:
        raise GluError(st, "glu_gemm_q_fwd" if offsets is None else "glu_gemm_q_grouped_fwd")
    return y, y_scale


def mlp_q_fwd(x, x_scale, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, *, out=None, dtype=None,
              act: str = "silu", offsets=None, workspace=None, stream=None):
    """out = y @ w_down^T with y = act(x @ w_gate^T) * (x @ w_up^T) quantised by
    rows: gemm_q_fwd and gemm_q_nt through a workspace (a uint8 device tensor of
    glu_mlp_q_workspace_bytes(rows, I) bytes, allocated here when not given).
    x is (..., H), the gate and up weights (I, H), the down weights (H, I); with
    ``offsets`` (E, I, H) and (E, H, I) (see gemm_q_nt)."""
    import torch
    if stream is not None:
        return _on_stream(stream, mlp_q_fwd, x, x_scale, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, out=out,
                          dtype=dtype, act=act, offsets=offsets, workspace=workspace)
    grouped = offsets is not None
    dev = _same_device(x, x_scale, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, out, offsets, workspace)
    n_rows, x_stride, xs_stride, H = _in_q(x, x_scale, "x")
    gate = _weight_q(w_gate, gate_scale, H, "w_gate", grouped)
    if w_up.shape != w_gate.shape or _weight_q(w_up, up_scale, H, "w_up", grouped) != gate:
        raise ValueError("w_gate and w_up (and their scales) must have one shape and one stride")
    I, w_stride, w_group, s_stride, s_group = gate
    N, d_stride, d_group, ds_stride, ds_group = _weight_q(w_down, down_scale, I, "w_down", grouped)
    if N != H or (grouped and w_down.shape[0] != w_gate.shape[0]):
        raise ValueError("w_down must be (H, I), for as many experts as w_gate")
    if out is None:
        out = torch.empty(x.shape, dtype=dtype or torch.bfloat16, device=x.device)
    elif out.shape != x.shape or (dtype is not None and out.dtype != dtype):
        raise ValueError("out has the wrong shape or dtype")
    if workspace is None:
        workspace = torch.empty(max(16, glu_mlp_q_workspace_bytes(max(n_rows, 1), max(I, 1))), dtype=torch.uint8,
                                device=x.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    st = glu_mlp_q_fwd(x.data_ptr(), x_stride, x_scale.data_ptr(), xs_stride, w_gate.data_ptr(), w_up.data_ptr(),
                       w_stride, w_group, gate_scale.data_ptr(), up_scale.data_ptr(), s_stride, s_group,
                       w_down.data_ptr(), d_stride, d_group, down_scale.data_ptr(), ds_stride, ds_group,
                       out.data_ptr(), _mat(out, "out")[1], n_rows, H, I,
                       _offsets(offsets, w_gate) if grouped else None, w_gate.shape[0] if grouped else 0, ACT[act],
                       _dtype_code(out), workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
    if st:
        raise GluError(st, "glu_mlp_q_fwd")
    return out


# ---- host tensors ---------------------------------------------------------------

def _host_rows(t, name):
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dim() == 1:
        return 1, t.shape[0]
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    n = 1
    for s_ in t.shape[:-1]:
        n *= s_
    return n, t.stride(-2)


class HostPipeline:
    """Device workspace and the three streams the host-memory entry points
    use.  Allocation is torch's (plumbing); the copies and kernels are the
    library's."""

    def __init__(self, workspace_bytes: int = 256 << 20, device=None):
        import torch
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.workspace = torch.empty(workspace_bytes, dtype=torch.uint8, device=dev)
        self.copy_in = torch.cuda.Stream(dev)
        self.copy_out = torch.cuda.Stream(dev)

    def args(self, compute=None):
        import torch
        compute = torch.cuda.current_stream() if compute is None else compute
        return (self.workspace.data_ptr(), self.workspace.numel(), self.copy_in.cuda_stream,
                compute.cuda_stream, self.copy_out.cuda_stream)


def fwd_host(pipe: HostPipeline, a, b=None, *, y=None, act="silu", layout="split", compute=None):
    """glu_fwd_host on CPU tensors (page-locked for overlap).  Returns y (a CPU
    tensor); synchronise the compute stream before reading it."""
    import torch
    concat = layout == "concat"
    n_rows, a_stride = _host_rows(a, "a")
    n_cols = a.shape[-1] // 2 if concat else a.shape[-1]
    if y is None:
        shape = (*a.shape[:-1], n_cols)
        y = torch.empty(shape, dtype=a.dtype, pin_memory=a.is_pinned())
    _, y_stride = _host_rows(y, "y")
    b_ptr, b_stride = (None, 0) if concat else (b.data_ptr(), _host_rows(b, "b")[1])
    st = glu_fwd_host(a.data_ptr(), a_stride, b_ptr, b_stride, y.data_ptr(), y_stride, n_rows, n_cols,
                      LAYOUT[layout], ACT[act], _dtype_code(a), *pipe.args(compute))
    if st:
        raise GluError(st, "glu_fwd_host")
    return y


def bwd_host(pipe: HostPipeline, dc, a, b=None, *, da=None, db=None, act="silu", layout="split",
             compute=None):
    """glu_bwd_host on CPU tensors.  SPLIT returns (da, db); CONCAT returns dx."""
    import torch
    concat = layout == "concat"
    n_rows, a_stride = _host_rows(a, "a")
    _, dc_stride = _host_rows(dc, "dc")
    n_cols = dc.shape[-1]
    pin = a.is_pinned()
    if da is None:
        da = torch.empty(a.shape, dtype=a.dtype, pin_memory=pin)
    _, da_stride = _host_rows(da, "da")
    if concat:
        st = glu_bwd_host(dc.data_ptr(), dc_stride, a.data_ptr(), a_stride, None, 0, da.data_ptr(), da_stride,
                          None, 0, n_rows, n_cols, LAYOUT[layout], ACT[act], _dtype_code(a), *pipe.args(compute))
        if st:
            raise GluError(st, "glu_bwd_host")
        return da
    if db is None:
        db = torch.empty(b.shape, dtype=b.dtype, pin_memory=pin)
    _, b_stride = _host_rows(b, "b")
    _, db_stride = _host_rows(db, "db")
    st = glu_bwd_host(dc.data_ptr(), dc_stride, a.data_ptr(), a_stride, b.data_ptr(), b_stride, da.data_ptr(),
                      da_stride, db.data_ptr(), db_stride, n_rows, n_cols, LAYOUT[layout], ACT[act],
                      _dtype_code(a), *pipe.args(compute))
    if st:
        raise GluError(st, "glu_bwd_host")
    return da, db
