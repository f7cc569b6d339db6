"""A learned gate for the local experts, in the place of the mixture's own.

``Gate`` answers a row of logits with its m largest components and their share
of the softmax, as ``Assigner`` answers with ids and gamma, and gives the
gradient of the logits, with the balance loss that keeps all components in use;
``Distiller`` compares logits with a teacher's top entries, the mixture's ids
and gamma among them, and gives that loss's gradient.  Everything runs on the
current torch stream (or ``stream``) in the library's kernels; tensors are
dense, on one device, and they and these objects have to be kept until that work
is done.  Objects own their outputs and workspaces: calls that overlap (two
streams, two graphs replayed at once) need an object each.  No arithmetic happens
here.
"""
from __future__ import annotations

import torch

from . import (GMM_DISTILL_ADD, GMM_GATE_NORMALISED, GMM_TEACHER_GAMMA, GMM_TEACHER_LOGITS,
               gmm_distill, gmm_distill_ws_bytes, gmm_gate, gmm_gate_grad, gmm_gate_ws_bytes)
from .experts import _device, _empty, _here, _need
from .torch_api import TORCH_XDTYPE

MAX_TEACHER = 64
MAX_STUDENT = 1 << 18


def _like(t, stream):
    """A new tensor as dense `t`, for work on `stream` (None: the current one)."""
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def _type(dtype):
    if dtype not in TORCH_XDTYPE:
        raise ValueError("type %s is not supported" % dtype)
    return TORCH_XDTYPE[dtype]


class Gate:
    """The m largest of K logits for each of N rows.

    After ``forward``: ids [N, m] int32 and gamma [N, m] float32, what
    ``LocalExperts.forward`` takes; lse [N]; with ``balance`` also counts [K]
    int64, mass [K], share [K] and loss [1]: device tensors that the next
    ``forward`` overwrites (those of the balance loss the next that has it, until
    which they stay).  normalised: the m shares of a row sum to one.
    """

    def __init__(self, N, K, m, dtype, normalised=False, device="cuda"):
        self.N, self.K, self.m, self.dtype = int(N), int(K), int(m), dtype
        self.xdtype, self.flags = _type(dtype), GMM_GATE_NORMALISED if normalised else 0
        self.ws_bytes = gmm_gate_ws_bytes(self.N, self.K, self.m)
        if self.ws_bytes == 0:
            raise ValueError("unsupported sizes N=%d K=%d m=%d" % (N, K, m))
        self.device = dev = _device(device)
        self.ids = torch.empty(self.N, self.m, dtype=torch.int32, device=dev)
        self.gamma = torch.empty(self.N, self.m, dtype=torch.float32, device=dev)
        self.lse = torch.empty(self.N, dtype=torch.float32, device=dev)
        self.counts = self.mass = self.share = self.loss = self.ws = None
        self._shape, self._small = (self.N, self.K), (self.N, self.m)
        self._balanced = None  # of the last forward; None: there was none

    def _live(self, live):
        return live if live is None else _need(live, "live", (self.N,), torch.bool, self.device)

    def _room(self, stream):
        """The balance outputs, made when they are first asked for."""
        dev, K = self.device, self.K
        self.counts = _empty((K,), torch.int64, dev, stream)
        self.mass = _empty((K,), torch.float32, dev, stream)
        self.share = _empty((K,), torch.float32, dev, stream)
        self.loss = _empty((1,), torch.float32, dev, stream)
        self.ws = _empty((self.ws_bytes,), torch.uint8, dev, stream)

    def forward(self, logits, live=None, balance=False, stream=None):
        """logits [N, K] -> (ids, gamma).  live [N] bool: rows that are not
        padding; the others get ids -1 and count nowhere."""
        _need(logits, "logits", self._shape, self.dtype, self.device)
        live = self._live(live)
        _here(self.device)
        self._balanced = None
        if balance:
            if self.ws is None:
                self._room(stream)
            gmm_gate(logits, self.xdtype, self.N, self.K, self.m, self.flags, live, self.ids,
                     self.gamma, self.lse, self.counts, self.mass, self.share, self.loss, self.ws,
                     self.ws_bytes, stream=stream)
        else:
            gmm_gate(logits, self.xdtype, self.N, self.K, self.m, self.flags, live, self.ids,
                     self.gamma, self.lse, None, None, None, None, None, 0, stream=stream)
        self._balanced = bool(balance)
        return self.ids, self.gamma

    def backward(self, logits, dgamma=None, live=None, balance=0.0, out=None, stream=None):
        """The gradient of the logits that the last ``forward`` had (with the
        same ``live``), from that of gamma (None: 0) and of balance * loss."""
        if self._balanced is None:
            raise RuntimeError("backward before forward")
        if balance and not self._balanced:
            raise RuntimeError("the last forward had no balance")
        _need(logits, "logits", self._shape, self.dtype, self.device)
        live = self._live(live)
        if dgamma is not None:
            _need(dgamma, "dgamma", self._small, torch.float32, self.device)
        if out is None:
            out = _like(logits, stream)
        else:
            _need(out, "out", self._shape, self.dtype, self.device)
        _here(self.device)
        gmm_gate_grad(logits, self.xdtype, self.N, self.K, self.m, self.flags, live, self.ids,
                      self.gamma, dgamma, self.share if balance else None, float(balance), out,
                      stream=stream)
        return out


class Distiller:
    """N rows of K student logits against a teacher's m entries each.

    teacher: "gamma" (the shares of a mixture or a gate: ids and gamma of an
    ``Assigner`` or a ``Gate``) or "logits".  The loss is scale * T^2 times the
    rows' weighted divergences in all (scale None: 1 / N, a mean); ``rows`` [N]
    and ``total`` [1] hold them and are overwritten by the next call.
    """

    def __init__(self, N, K, m, dtype, teacher="gamma", temperature=1.0, scale=None, device="cuda"):
        self.N, self.K, self.m, self.dtype = int(N), int(K), int(m), dtype
        self.xdtype = _type(dtype)
        kinds = {"gamma": GMM_TEACHER_GAMMA, "logits": GMM_TEACHER_LOGITS}
        if teacher not in kinds:
            raise ValueError("teacher %r: expected 'gamma' or 'logits'" % (teacher,))
        if not (self.N >= 0 and 1 <= self.K <= MAX_STUDENT and 1 <= self.m <= MAX_TEACHER
                and self.N * self.m <= 2 ** 31 - 1):
            raise ValueError("unsupported sizes N=%d K=%d m=%d" % (N, K, m))
        self.kind, self.temperature = kinds[teacher], float(temperature)
        if not 1e-30 <= self.temperature <= 1e30:
            raise ValueError("temperature %r" % (temperature,))
        self.scale = 1.0 / max(1, self.N) if scale is None else float(scale)
        self.device = dev = _device(device)
        self.rows = torch.empty(self.N, dtype=torch.float32, device=dev)
        self.total = torch.empty(1, dtype=torch.float32, device=dev)
        self.ws_bytes = gmm_distill_ws_bytes()
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self._shape, self._small = (self.N, self.K), (self.N, self.m)

    def _call(self, logits, ids, values, weights, out, flags, stream):
        dev = self.device
        _need(logits, "logits", self._shape, self.dtype, dev)
        _need(ids, "ids", self._small, torch.int32, dev)
        _need(values, "values", self._small, torch.float32, dev)
        if weights is not None:
            _need(weights, "weights", (self.N,), torch.float32, dev)
        _here(dev)
        gmm_distill(logits, self.xdtype, self.N, self.K, self.m, self.kind, flags,
                    self.temperature, self.scale, ids, values, weights, self.rows, self.total, out,
                    self.ws, self.ws_bytes, stream=stream)

    def loss(self, logits, ids, values, weights=None, stream=None):
        """The loss alone: ``total`` [1]."""
        self._call(logits, ids, values, weights, None, 0, stream)
        return self.total

    def step(self, logits, ids, values, weights=None, out=None, add=False, stream=None):
        """(loss, gradient of the logits) in one pass; with ``add`` the gradient
        is added to what ``out`` holds (``Gate.backward``'s)."""
        if out is None:
            if add:
                raise ValueError("add without out")
            _need(logits, "logits", self._shape, self.dtype, self.device)
            out = _like(logits, stream)
        else:
            _need(out, "out", self._shape, self.dtype, self.device)
        self._call(logits, ids, values, weights, out, GMM_DISTILL_ADD if add else 0, stream)
        return self.total, out
