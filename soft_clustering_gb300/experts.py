"""Local experts behind the mixture's soft assignment.

A fitted mixture gates a layer of experts (a localised gating network): each
point's top-m components (``Assigner.assign``: ids, gamma) each apply their
own matrix to the point's row, and the answers are summed with gamma.

``Router`` puts the entries of a top-m table in the order of their components
and moves rows there and back; ``ExpertProduct`` is the product of every
component's rows with its matrix, and its gradients; ``LocalExperts`` is the
layer of both, with its backward pass.  Everything runs on the current torch
stream (or ``stream``) in the library's kernels; tensors are dense, on one
device, and have to stay valid until that work is done.  No arithmetic
happens here.
"""
from __future__ import annotations

import contextlib

import torch

from . import (GMM_F32, gmm_collect, gmm_expert_product, gmm_expert_product_dw,
               gmm_expert_product_dx, gmm_expert_ws_bytes, gmm_last_device_status, gmm_route,
               gmm_route_ws_bytes, gmm_spread)
from .torch_api import TORCH_XDTYPE

STATUS_BYTES = 256  # of a products' workspace, at its head


def _need(t, name, shape, dtype, device):
    """A dense tensor of this shape (a tuple), type and device, or ValueError."""
    if (torch.is_tensor(t) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t
    if not torch.is_tensor(t):
        raise ValueError("%s is not a tensor" % name)
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError("%s: expected %s %s on %s, got %s %s on %s"
                         % (name, shape, dtype, device, tuple(t.shape), t.dtype, t.device))
    raise ValueError("%s is not dense (strides %s)" % (name, t.stride()))


def _device(device):
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError("device %s: expected a CUDA device" % d)
    if d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


def _here(device):
    """The library launches on the current device: ValueError if that is not the
    tensors' one."""
    if torch.cuda.current_device() != device.index:
        raise ValueError("tensors are on %s, the current device is cuda:%d"
                         % (device, torch.cuda.current_device()))


def _on(stream):
    """torch work within goes to `stream` (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(_current(stream, None))


def _current(stream, device):
    """`stream` as torch's Stream (None: the current one)."""
    if stream is None:
        return torch.cuda.current_stream(device)
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream)


def _empty(shape, dtype, device, stream):
    """A new tensor for work on `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _xdtype(t, name):
    x = TORCH_XDTYPE.get(t.dtype)
    if x is None:
        raise ValueError("%s: type %s is not supported" % (name, t.dtype))
    return x


def _rows_of(t, name):
    """(rows, width) of a tensor with two dimensions."""
    try:
        rows, width = t.shape
    except (AttributeError, TypeError, ValueError):
        raise ValueError("%s: expected a tensor of two dimensions" % name) from None
    return rows, width


class Router:
    """Places of N points' top-m entries among K components' rows.

    After ``route``: offsets [K+1] int64 (component k owns the rows
    offsets[k] .. offsets[k+1]-1), entry [N*m] int32 (the entry n*m + t of each
    row, -1 past offsets[K]) and slot [N, m] int32 (the row of each entry, -1
    where its id is outside [0, K)), device tensors that the next ``route``
    overwrites.
    """

    def __init__(self, N, m, K, device="cuda"):
        self.N, self.m, self.K, self.rows = int(N), int(m), int(K), int(N) * int(m)
        self.ws_bytes = gmm_route_ws_bytes(self.N, self.m, self.K)
        if self.ws_bytes == 0:
            raise ValueError("unsupported sizes N=%d m=%d K=%d" % (N, m, K))
        self.device = dev = _device(device)
        self.offsets = torch.zeros(self.K + 1, dtype=torch.int64, device=dev)
        self.entry = torch.full((self.rows,), -1, dtype=torch.int32, device=dev)
        self.slot = torch.full((self.N, self.m), -1, dtype=torch.int32, device=dev)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.routes = 0  # calls of ``route`` so far

    def route(self, ids, stream=None):
        """ids: [N, m] int32, as ``Assigner.ids``."""
        _need(ids, "ids", (self.N, self.m), torch.int32, self.device)
        _here(self.device)
        self.routes += 1
        gmm_route(ids, self.N, self.m, self.K, self.offsets, self.entry, self.slot, self.ws,
                  self.ws_bytes, stream=stream)

    def spread(self, X, gamma=None, Z=None, out=None, stream=None):
        """Y[slot[n, t]] = gamma[n, t] X[n] (gamma None: 1), zeros past the last
        row used.  With Z [N*m, D]: returns (Y, dgamma), dgamma[n, t] =
        <X[n], Z[slot[n, t]]>: with X = d out the gradient of ``collect``."""
        D, x, dt, dev = _rows_of(X, "X")[1], _xdtype(X, "X"), X.dtype, self.device
        _need(X, "X", (self.N, D), dt, dev)
        _here(dev)
        if gamma is not None:
            _need(gamma, "gamma", (self.N, self.m), torch.float32, dev)
        dgamma = None
        if Z is not None:
            _need(Z, "Z", (self.rows, D), dt, dev)
            dgamma = _empty((self.N, self.m), torch.float32, dev, stream)
        if out is None:
            out = _empty((self.rows, D), dt, dev, stream)
        else:
            _need(out, "out", (self.rows, D), dt, dev)
        gmm_spread(X, x, self.N, D, self.m, self.K, self.rows, self.slot, self.offsets, gamma, Z,
                   out, dgamma, stream=stream)
        return out if Z is None else (out, dgamma)

    def collect(self, Z, gamma=None, out=None, stream=None):
        """out[n] = sum_t gamma[n, t] Z[slot[n, t]] (gamma None: 1): the answers
        of a point's components, or the gradient of ``spread``."""
        D, x, dt, dev = _rows_of(Z, "Z")[1], _xdtype(Z, "Z"), Z.dtype, self.device
        _need(Z, "Z", (self.rows, D), dt, dev)
        _here(dev)
        if gamma is not None:
            _need(gamma, "gamma", (self.N, self.m), torch.float32, dev)
        if out is None:
            out = _empty((self.N, D), dt, dev, stream)
        else:
            _need(out, "out", (self.N, D), dt, dev)
        gmm_collect(Z, x, self.N, D, self.m, self.rows, self.slot, gamma, out, stream=stream)
        return out


class ExpertProduct:
    """Products of K components' rows with their own [d_out, d_in] matrices,
    for up to max_rows rows.  offsets is a ``Router``'s; rows past offsets[K]
    come back as zeros."""

    def __init__(self, K, d_in, d_out, dtype, max_rows, device="cuda"):
        self.K, self.d_in, self.d_out, self.max_rows = int(K), int(d_in), int(d_out), int(max_rows)
        if dtype not in TORCH_XDTYPE:
            raise ValueError("type %s is not supported" % dtype)
        self.dtype, self.xdtype, self.device = dtype, TORCH_XDTYPE[dtype], _device(device)
        self.ws_bytes = gmm_expert_ws_bytes(self.max_rows, self.d_in, self.d_out, self.K,
                                            self.xdtype)
        if self.ws_bytes == 0:
            raise ValueError("unsupported sizes K=%d d_in=%d d_out=%d rows=%d"
                             % (K, d_in, d_out, max_rows))
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self._offsets_shape, self._w_shape = (self.K + 1,), (self.K, self.d_out, self.d_in)

    def _rows(self, t, name, width):
        R = _rows_of(t, name)[0]
        if R > self.max_rows:
            raise ValueError("%s: %d rows, at most %d" % (name, R, self.max_rows))
        _need(t, name, (R, width), self.dtype, self.device)
        return R

    def _common(self, offsets, W):
        _here(self.device)
        _need(offsets, "offsets", self._offsets_shape, torch.int64, self.device)
        if W is not None:
            _need(W, "W", self._w_shape, self.dtype, self.device)

    def _out(self, out, shape, dtype, stream):
        if out is None:
            return _empty(shape, dtype, self.device, stream)
        return _need(out, "out", shape, dtype, self.device)

    def forward(self, A, offsets, W, out=None, stream=None):
        """Y[r] = W_k A[r]."""
        R = self._rows(A, "A", self.d_in)
        self._common(offsets, W)
        out = self._out(out, (R, self.d_out), self.dtype, stream)
        gmm_expert_product(A, self.xdtype, R, self.d_in, self.d_out, self.K, offsets, W, out,
                           self.ws, self.ws_bytes, stream=stream)
        return out

    def backward_rows(self, dY, offsets, W, out=None, stream=None):
        """dA[r] = W_k^T dY[r]."""
        R = self._rows(dY, "dY", self.d_out)
        self._common(offsets, W)
        out = self._out(out, (R, self.d_in), self.dtype, stream)
        gmm_expert_product_dx(dY, self.xdtype, R, self.d_in, self.d_out, self.K, offsets, W, out,
                              self.ws, self.ws_bytes, stream=stream)
        return out

    def backward_weights(self, dY, A, offsets, out=None, out_dtype=None, stream=None):
        """dW_k = sum over the rows of k of dY[r] A[r]^T, in the weights' type or
        (out_dtype) float32."""
        R = self._rows(dY, "dY", self.d_out)
        if self._rows(A, "A", self.d_in) != R:
            raise ValueError("dY has %d rows, A %d" % (R, A.shape[0]))
        self._common(offsets, None)
        wt = out_dtype or (out.dtype if out is not None else self.dtype)
        if wt not in (self.dtype, torch.float32):
            raise ValueError("out_dtype %s: expected %s or float32" % (wt, self.dtype))
        out = self._out(out, self._w_shape, wt, stream)
        gmm_expert_product_dw(dY, A, self.xdtype, R, self.d_in, self.d_out, self.K, offsets, out,
                              GMM_F32 if wt == torch.float32 else self.xdtype, self.ws,
                              self.ws_bytes, stream=stream)
        return out

    def device_status(self, stream=None):
        """The first failure on the device in any call so far, or GMM_OK; it
        stays until ``clear_status``.  Waits for `stream`."""
        return gmm_last_device_status(self.ws, stream)

    def clear_status(self, stream=None):
        with _on(stream):
            self.ws[:STATUS_BYTES].zero_()


class LocalExperts:
    """A layer of K experts y = sum_t gamma[n, t] W[ids[n, t]] x[n] for N points.

    W [K, d_out, d_in] is the caller's (``adamw.AdamW`` trains it).  ``forward``
    keeps what ``backward`` needs until the next ``forward``, gamma by value: its
    buffer may be written again in between (the next batch's assignment).  autograd
    records neither: gradients are what ``backward`` returns.
    """

    def __init__(self, N, m, K, d_in, d_out, dtype, device="cuda"):
        self.router = Router(N, m, K, device)
        self.product = ExpertProduct(K, d_in, d_out, dtype, self.router.rows, device)
        self._gamma = torch.empty(self.router.N, self.router.m, dtype=torch.float32,
                                  device=self.router.device)
        self._kept = None

    def forward(self, X, ids, gamma, W, stream=None):
        """X [N, d_in], ids and gamma [N, m] as ``Assigner`` holds them -> [N, d_out]."""
        r = self.router
        _need(gamma, "gamma", (r.N, r.m), torch.float32, r.device)
        self._kept = None  # its rows lose their places now
        r.route(ids, stream=stream)
        A = r.spread(X, stream=stream)
        Y = self.product.forward(A, r.offsets, W, stream=stream)
        with _on(stream):
            self._gamma.copy_(gamma)
        self._kept = (A, Y, r.routes, _current(stream, r.device).cuda_stream)
        return r.collect(Y, gamma, stream=stream)

    def backward(self, dout, W, weight_dtype=None, stream=None):
        """(dX, dgamma, dW) of the last ``forward`` for the answer's gradient."""
        if self._kept is None:
            raise RuntimeError("backward before forward")
        A, Y, routes, made_on = self._kept
        r = self.router
        if r.routes != routes:
            raise RuntimeError("the router was given other ids after forward")
        s = _current(stream, r.device)
        if s.cuda_stream != made_on:
            # their memory goes back to the stream they were made on
            A.record_stream(s)
            Y.record_stream(s)
        dY, dgamma = r.spread(dout, self._gamma, Y, stream=stream)
        dA = self.product.backward_rows(dY, r.offsets, W, stream=stream)
        dW = self.product.backward_weights(dY, A, r.offsets, out_dtype=weight_dtype, stream=stream)
        return r.collect(dA, stream=stream), dgamma, dW

    def device_status(self, stream=None):
        """``ExpertProduct.device_status`` of all three products."""
        return self.product.device_status(stream)
