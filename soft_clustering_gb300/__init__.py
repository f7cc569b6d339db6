"""Python binding of libgmm (include/gmm.h, include/gmm_experts.h): the fused
GMM EM step, top-m soft assignment, and local experts behind it, on one GB300.

Argument marshalling only.  Every function here has the name of the C entry
point it calls and forwards device pointers taken from torch tensors (or
plain integers) plus sizes; all arithmetic runs in the library's CUDA
kernels.  There is no CPU fallback: if ``_build/libgmm.so`` has not been
built (``python -m soft_clustering_gb300.build``) every call raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libgmm.so")

GMM_COV_FULL, GMM_COV_DIAG, GMM_COV_ISO = 0, 1, 2
GMM_F32, GMM_F16, GMM_BF16 = 0, 1, 2
GMM_OK, GMM_ERR_INVALID_ARG, GMM_ERR_UNSUPPORTED, GMM_ERR_NOT_PD = 0, 1, 2, 3
GMM_ERR_NONFINITE, GMM_ERR_WORKSPACE, GMM_ERR_TIMEOUT, GMM_ERR_CUDA = 4, 5, 6, 7
GMM_FLAG_RIDGE, GMM_FLAG_NOT_PD, GMM_FLAG_FLOOR, GMM_FLAG_EMPTY = 1, 2, 4, 8
GMM_OPT_CUDA_CORES = 1

EXPORTS = (
    "gmm_default_opts", "gmm_status_string", "gmm_workspace_bytes", "gmm_prepared_bytes",
    "gmm_prepare", "gmm_em_step", "gmm_workspace_bytes_host", "gmm_em_step_host",
    "gmm_assign_topm", "gmm_last_device_status", "gmm_profile_enable", "gmm_profile_read",
    "gmm_profile_reset", "gmm_em_step_noalloc", "gmm_debug_tc_gemm", "gmm_ivf_lists_ws_bytes",
    "gmm_ivf_lists", "gmm_route_ws_bytes", "gmm_route", "gmm_spread", "gmm_collect",
    "gmm_expert_ws_bytes", "gmm_expert_product", "gmm_expert_product_dx",
    "gmm_expert_product_dw", "gmm_adamw_step", "gmm_adamw_step_counted", "gmm_adamw_moments",
)


class gmm_params(ctypes.Structure):
    _fields_ = [("pi", ctypes.c_void_p), ("mu", ctypes.c_void_p), ("cov", ctypes.c_void_p)]


class gmm_opts(ctypes.Structure):
    _fields_ = [("ridge_rel", ctypes.c_float), ("var_floor", ctypes.c_float),
                ("min_s0", ctypes.c_float), ("flags", ctypes.c_int)]


class gmm_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int)]


class gmm_adamw_opts(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("grad_scale", ctypes.c_double), ("step", ctypes.c_int64),
                ("state_bits", ctypes.c_int), ("rounding", ctypes.c_int),
                ("skip", ctypes.c_void_p)]


class GmmError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = int(status)
        super().__init__("%s: %s" % (what, status_string(status)))


_lib = None


def lib():
    """The loaded libgmm.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libgmm.so not built (%s); run python -m soft_clustering_gb300.build"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER
        L.gmm_default_opts.restype = gmm_opts
        L.gmm_status_string.argtypes = [i32]
        L.gmm_status_string.restype = ctypes.c_char_p
        L.gmm_workspace_bytes.argtypes = [i64, i32, i32, i32, i32]
        L.gmm_workspace_bytes.restype = sz
        L.gmm_workspace_bytes_host.argtypes = [i64, i32, i32, i32, i32, i64]
        L.gmm_workspace_bytes_host.restype = sz
        L.gmm_prepared_bytes.argtypes = [i32, i32, i32]
        L.gmm_prepared_bytes.restype = sz
        L.gmm_prepare.argtypes = [P(gmm_params), i32, i32, i32, P(gmm_opts), vp, vp, vp]
        L.gmm_em_step.argtypes = [vp, i32, i64, i32, i32, P(gmm_params), i32, P(gmm_opts), vp, sz,
                                  vp, vp, vp, vp]
        L.gmm_em_step_host.argtypes = [vp, i32, i64, i32, i32, P(gmm_params), i32, P(gmm_opts),
                                       vp, sz, i64, vp, vp, vp, vp]
        L.gmm_assign_topm.argtypes = [vp, i32, i64, i32, i32, vp, i32, i32, vp, vp, vp, vp, sz, vp]
        L.gmm_last_device_status.argtypes = [vp, vp]
        L.gmm_em_step_noalloc.argtypes = [vp, i32, i64, i32, i32, P(gmm_params), i32,
                                          P(gmm_opts), vp, vp, vp, vp]
        L.gmm_debug_tc_gemm.argtypes = [vp, vp, vp, i32, i32, vp, vp]
        L.gmm_debug_tc_gemm.restype = i32
        L.gmm_ivf_lists_ws_bytes.argtypes = [i64, i32, i32]
        L.gmm_ivf_lists_ws_bytes.restype = sz
        L.gmm_ivf_lists.argtypes = [vp, vp, i64, i32, i32, ctypes.c_float, vp, vp, vp, vp, sz, vp]
        L.gmm_route_ws_bytes.argtypes = [i64, i32, i32]
        L.gmm_route_ws_bytes.restype = sz
        L.gmm_route.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, sz, vp]
        L.gmm_spread.argtypes = [vp, i32, i64, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp]
        L.gmm_collect.argtypes = [vp, i32, i64, i32, i32, i64, vp, vp, vp, vp]
        L.gmm_expert_ws_bytes.argtypes = [i64, i32, i32, i32, i32]
        L.gmm_expert_ws_bytes.restype = sz
        for f in ("gmm_expert_product", "gmm_expert_product_dx"):
            getattr(L, f).argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, vp, vp, sz, vp]
        L.gmm_expert_product_dw.argtypes = [vp, vp, i32, i64, i32, i32, i32, vp, vp, i32, vp, sz,
                                            vp]
        L.gmm_adamw_step.argtypes = [P(gmm_adamw_tensor), i32, P(gmm_adamw_opts), vp]
        L.gmm_adamw_step_counted.argtypes = [P(gmm_adamw_tensor), i32, P(gmm_adamw_opts), vp, vp]
        L.gmm_adamw_moments.argtypes = [P(gmm_adamw_tensor), i32, i32, P(vp), P(vp), vp]
        L.gmm_profile_enable.argtypes = [i32]
        L.gmm_profile_enable.restype = None
        L.gmm_profile_read.argtypes = [P(ctypes.c_char_p), P(ctypes.c_double), P(ctypes.c_long),
                                       i32]
        L.gmm_profile_read.restype = i32
        L.gmm_profile_reset.restype = None
        for f in ("gmm_prepare", "gmm_em_step", "gmm_em_step_host", "gmm_assign_topm",
                  "gmm_last_device_status", "gmm_em_step_noalloc", "gmm_ivf_lists",
                  "gmm_route", "gmm_spread", "gmm_collect", "gmm_expert_product",
                  "gmm_expert_product_dx", "gmm_expert_product_dw", "gmm_adamw_step",
                  "gmm_adamw_step_counted", "gmm_adamw_moments"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def _ptr(x):
    """Device/host address of a torch tensor, numpy array or integer (None -> NULL)."""
    try:
        return x.data_ptr()
    except AttributeError:
        pass
    if x is None or isinstance(x, int):
        return x
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError(type(x))


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_raw_stream = None


def _current_stream():
    """The current torch stream's handle, without a Stream object where torch
    offers that (3 us less a call)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()  # initialises CUDA
        c = torch._C
        if hasattr(c, "_cuda_getCurrentRawStream") and hasattr(c, "_cuda_getDevice"):
            of, dev = c._cuda_getCurrentRawStream, c._cuda_getDevice
            _raw_stream = lambda: of(dev())  # noqa: E731
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


def _check(status, what, raise_on_error=True):
    if raise_on_error and status != GMM_OK:
        raise GmmError(status, what)
    return status


def status_string(status) -> str:
    return lib().gmm_status_string(int(status)).decode()


def gmm_default_opts(**overrides) -> gmm_opts:
    o = lib().gmm_default_opts()
    for k, v in overrides.items():
        setattr(o, k, v)
    return o


def gmm_workspace_bytes(N, D, K, cov, xdtype) -> int:
    return int(lib().gmm_workspace_bytes(N, D, K, cov, xdtype))


def gmm_workspace_bytes_host(N, D, K, cov, xdtype, chunk_rows) -> int:
    return int(lib().gmm_workspace_bytes_host(N, D, K, cov, xdtype, chunk_rows))


def gmm_prepared_bytes(D, K, cov) -> int:
    return int(lib().gmm_prepared_bytes(D, K, cov))


def make_params(pi, mu, cov) -> gmm_params:
    return gmm_params(_ptr(pi), _ptr(mu), _ptr(cov))


def gmm_prepare(pi, mu, cov, D, K, cov_type, prepared, flags=None, opts=None, stream=None,
                raise_on_error=True):
    p = make_params(pi, mu, cov)
    o = opts if opts is not None else gmm_default_opts()
    st = lib().gmm_prepare(ctypes.byref(p), D, K, cov_type, ctypes.byref(o), _ptr(prepared),
                           _ptr(flags), _stream(stream))
    return _check(st, "gmm_prepare", raise_on_error)


def gmm_em_step(X, xdtype, N, D, K, pi, mu, cov, cov_type, ws, ws_bytes, loglik, lse=None,
                flags=None, opts=None, stream=None, raise_on_error=True):
    p = make_params(pi, mu, cov)
    o = opts if opts is not None else gmm_default_opts()
    st = lib().gmm_em_step(_ptr(X), xdtype, N, D, K, ctypes.byref(p), cov_type, ctypes.byref(o),
                           _ptr(ws), ws_bytes, _ptr(loglik), _ptr(lse), _ptr(flags),
                           _stream(stream))
    return _check(st, "gmm_em_step", raise_on_error)


def gmm_em_step_host(X_host, xdtype, N, D, K, pi, mu, cov, cov_type, ws, ws_bytes, chunk_rows,
                     loglik, loglik_host=None, flags=None, opts=None, stream=None,
                     raise_on_error=True):
    p = make_params(pi, mu, cov)
    o = opts if opts is not None else gmm_default_opts()
    st = lib().gmm_em_step_host(_ptr(X_host), xdtype, N, D, K, ctypes.byref(p), cov_type,
                                ctypes.byref(o), _ptr(ws), ws_bytes, chunk_rows, _ptr(loglik),
                                _ptr(loglik_host), _ptr(flags), _stream(stream))
    return _check(st, "gmm_em_step_host", raise_on_error)


def gmm_assign_topm(X, xdtype, N, D, K, prepared, cov_type, m, ids, gamma, lse, ws, ws_bytes,
                    stream=None, raise_on_error=True):
    st = lib().gmm_assign_topm(_ptr(X), xdtype, N, D, K, _ptr(prepared), cov_type, m, _ptr(ids),
                               _ptr(gamma), _ptr(lse), _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "gmm_assign_topm", raise_on_error)


def gmm_em_step_noalloc(X, xdtype, N, D, K, pi, mu, cov, cov_type, loglik, lse, flags=None,
                        opts=None, stream=None, raise_on_error=True):
    """The EM step without a workspace, for callers that cannot allocate
    device memory (scratch is a fixed 64 MiB array inside the library).
    Synchronises the stream; returns the call's status."""
    p = make_params(pi, mu, cov)
    o = opts if opts is not None else gmm_default_opts()
    st = lib().gmm_em_step_noalloc(_ptr(X), xdtype, N, D, K, ctypes.byref(p), cov_type,
                                   ctypes.byref(o), _ptr(loglik), _ptr(lse), _ptr(flags),
                                   _stream(stream))
    return _check(st, "gmm_em_step_noalloc", raise_on_error)


def gmm_ivf_lists_ws_bytes(N, m, K) -> int:
    return int(lib().gmm_ivf_lists_ws_bytes(N, m, K))


def gmm_ivf_lists(ids, gamma, N, m, K, gamma_min, offsets, list_pts, list_gamma, ws, ws_bytes,
                  stream=None, raise_on_error=True):
    st = lib().gmm_ivf_lists(_ptr(ids), _ptr(gamma), N, m, K, float(gamma_min), _ptr(offsets),
                             _ptr(list_pts), _ptr(list_gamma), _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "gmm_ivf_lists", raise_on_error)


def gmm_route_ws_bytes(N, m, K) -> int:
    return int(lib().gmm_route_ws_bytes(N, m, K))


def gmm_route(ids, N, m, K, offsets, entry, slot, ws, ws_bytes, stream=None,
              raise_on_error=True):
    st = lib().gmm_route(_ptr(ids), N, m, K, _ptr(offsets), _ptr(entry), _ptr(slot), _ptr(ws),
                         ws_bytes, _stream(stream))
    return _check(st, "gmm_route", raise_on_error)


def gmm_spread(X, xdtype, N, D, m, K, R, slot, offsets, gamma, Z, Y, dgamma, stream=None,
               raise_on_error=True):
    st = lib().gmm_spread(_ptr(X), xdtype, N, D, m, K, R, _ptr(slot), _ptr(offsets), _ptr(gamma),
                          _ptr(Z), _ptr(Y), _ptr(dgamma), _stream(stream))
    return _check(st, "gmm_spread", raise_on_error)


def gmm_collect(Z, xdtype, N, D, m, R, slot, gamma, out, stream=None, raise_on_error=True):
    st = lib().gmm_collect(_ptr(Z), xdtype, N, D, m, R, _ptr(slot), _ptr(gamma), _ptr(out),
                           _stream(stream))
    return _check(st, "gmm_collect", raise_on_error)


def gmm_expert_ws_bytes(R, d_in, d_out, K, xdtype) -> int:
    return int(lib().gmm_expert_ws_bytes(R, d_in, d_out, K, xdtype))


def gmm_expert_product(A, xdtype, R, d_in, d_out, K, offsets, W, Y, ws, ws_bytes, stream=None,
                       raise_on_error=True):
    st = lib().gmm_expert_product(_ptr(A), xdtype, R, d_in, d_out, K, _ptr(offsets), _ptr(W),
                                  _ptr(Y), _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "gmm_expert_product", raise_on_error)


def gmm_expert_product_dx(dY, xdtype, R, d_in, d_out, K, offsets, W, dA, ws, ws_bytes,
                          stream=None, raise_on_error=True):
    st = lib().gmm_expert_product_dx(_ptr(dY), xdtype, R, d_in, d_out, K, _ptr(offsets), _ptr(W),
                                     _ptr(dA), _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "gmm_expert_product_dx", raise_on_error)


def gmm_expert_product_dw(dY, A, xdtype, R, d_in, d_out, K, offsets, dW, wdtype, ws, ws_bytes,
                          stream=None, raise_on_error=True):
    st = lib().gmm_expert_product_dw(_ptr(dY), _ptr(A), xdtype, R, d_in, d_out, K, _ptr(offsets),
                                     _ptr(dW), wdtype, _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "gmm_expert_product_dw", raise_on_error)


def gmm_adamw_step(tensors, count, opts, stream=None, raise_on_error=True):
    """tensors: a ctypes array of gmm_adamw_tensor; opts: gmm_adamw_opts."""
    st = lib().gmm_adamw_step(tensors, count, ctypes.byref(opts), _stream(stream))
    return _check(st, "gmm_adamw_step", raise_on_error)


def gmm_adamw_step_counted(tensors, count, opts, steps, stream=None, raise_on_error=True):
    """As gmm_adamw_step, with the steps taken in a device int64."""
    st = lib().gmm_adamw_step_counted(tensors, count, ctypes.byref(opts), _ptr(steps),
                                      _stream(stream))
    return _check(st, "gmm_adamw_step_counted", raise_on_error)


def gmm_adamw_moments(tensors, count, state_bits, m_out, v_out, stream=None,
                      raise_on_error=True):
    """m_out, v_out: ctypes arrays of device addresses."""
    st = lib().gmm_adamw_moments(tensors, count, state_bits, m_out, v_out, _stream(stream))
    return _check(st, "gmm_adamw_moments", raise_on_error)


def gmm_last_device_status(ws, stream=None) -> int:
    return int(lib().gmm_last_device_status(_ptr(ws), _stream(stream)))


def gmm_profile_enable(on: bool = True):
    lib().gmm_profile_enable(1 if on else 0)


def gmm_profile_reset():
    lib().gmm_profile_reset()


def gmm_profile_read(max_kernels: int = 32) -> dict:
    """{kernel name: (total ms, launches)} since the last reset (synchronises)."""
    names = (ctypes.c_char_p * max_kernels)()
    ms = (ctypes.c_double * max_kernels)()
    n_l = (ctypes.c_long * max_kernels)()
    n = lib().gmm_profile_read(names, ms, n_l, max_kernels)
    return {names[i].decode(): (ms[i], n_l[i]) for i in range(min(n, max_kernels))}


def gmm_debug_tc_gemm(A, B, C, kdim, n, status, stream=None) -> int:
    """Test-only: C = A B^T through the tensor-core building blocks."""
    return int(lib().gmm_debug_tc_gemm(_ptr(A), _ptr(B), _ptr(C), kdim, n, _ptr(status),
                                       _stream(stream)))
