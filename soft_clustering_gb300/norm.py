"""Layer norm of the rows that enter a layer of experts.

``LayerNorm`` holds sizes and a workspace, not weights: those are the caller's
(``adamw.AdamW`` trains them).  Everything runs on the current torch stream (or
``stream``) in the library's kernels; tensors are dense, on one device, and they
and these objects have to be kept until that work is done.  An object owns its
workspace: backward passes that overlap need an object each.  No arithmetic
happens here.
"""
from __future__ import annotations

import torch

from . import gmm_layer_norm, gmm_layer_norm_grad, gmm_layer_norm_ws_bytes
from .experts import _device, _empty, _here, _need, _rows_of
from .gate import _like, _type


class LayerNorm:
    """y = weight (x - mean) / sqrt(var + eps) + bias over rows of D.

    dtype: of the rows; weight_dtype: of weight and bias, dtype (None) or
    float32.  ``backward`` takes the rows' statistics again from X, so ``forward``
    keeps nothing."""

    def __init__(self, D, dtype, eps=1e-5, weight_dtype=None, device="cuda"):
        self.D, self.dtype, self.eps = int(D), dtype, float(eps)
        self.weight_dtype = weight_dtype or dtype
        self.xdtype, self.wdtype = _type(dtype), _type(self.weight_dtype)
        if self.weight_dtype not in (dtype, torch.float32):
            raise ValueError("weight_dtype %s: expected %s or float32" % (weight_dtype, dtype))
        self.ws_bytes = gmm_layer_norm_ws_bytes(self.D)
        if self.ws_bytes == 0:
            raise ValueError("unsupported size D=%d" % self.D)
        if not 0.0 <= self.eps < float("inf"):
            raise ValueError("eps %r" % (eps,))
        self.device = _device(device)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self._weight = (self.D,)

    def _rows(self, t, name, N=None):
        rows = _rows_of(t, name)[0] if N is None else N
        _need(t, name, (rows, self.D), self.dtype, self.device)
        return rows

    def _param(self, t, name):
        if t is not None:
            _need(t, name, self._weight, self.weight_dtype, self.device)

    def forward(self, X, weight=None, bias=None, out=None, stream=None):
        """X [N, D] -> Y [N, D] (weight None: 1, bias None: 0)."""
        N = self._rows(X, "X")
        self._param(weight, "weight")
        self._param(bias, "bias")
        _here(self.device)
        if out is None:
            out = _like(X, stream)
        else:
            self._rows(out, "out", N)
        gmm_layer_norm(X, self.xdtype, N, self.D, self.eps, weight, bias, self.wdtype, out,
                       stream=stream)
        return out

    def backward(self, dY, X, weight=None, out=None, weight_grads=True, stream=None):
        """(dX, dweight, dbias) for the gradient of Y; without weight_grads
        (dX, None, None)."""
        N = self._rows(X, "X")
        self._rows(dY, "dY", N)
        self._param(weight, "weight")
        _here(self.device)
        if out is None:
            out = _like(X, stream)
        else:
            self._rows(out, "out", N)
        dw = db = None
        if weight_grads:
            dw = _empty(self._weight, self.weight_dtype, self.device, stream)
            db = _empty(self._weight, self.weight_dtype, self.device, stream)
        gmm_layer_norm_grad(dY, X, self.xdtype, N, self.D, self.eps, weight, self.wdtype, out, dw,
                            db, self.ws if weight_grads else None, self.ws_bytes, stream=stream)
        return out, dw, db
