"""AdamW over a list of tensors in one launch, moments in 32 or 8 bits.

``AdamW`` holds the parameters' moments as torch tensors and calls
``gmm_adamw_step`` on the current torch stream.  No arithmetic happens here.
"""
from __future__ import annotations

import ctypes
import warnings
from operator import is_

import torch

from . import (gmm_adamw_moments, gmm_adamw_opts, gmm_adamw_step, gmm_adamw_step_counted,
               gmm_adamw_tensor)
from .experts import _empty, _here
from .torch_api import TORCH_XDTYPE

BLOCK = 256  # elements that share one scale of an 8-bit moment
ROUNDINGS = {"nearest": 0, "seeded": 1}


def _dense(t, name, n, dtypes, device):
    if not torch.is_tensor(t) or t.numel() != n or t.dtype not in dtypes or t.device != device:
        raise ValueError("%s: expected %d elements of %s on %s" % (name, n, dtypes, device))
    if not t.is_contiguous():
        raise ValueError("%s is not dense (strides %s)" % (name, t.stride()))
    return t


def _apart(named):
    """ValueError if two of the tensors (name, tensor) have memory in common."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name)
                   for name, t in named if t is not None and t.numel())
    for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError("%s and %s have memory in common" % (a, b))


class AdamW:
    """Decoupled weight decay Adam on `params`, dense float32 / float16 / bfloat16
    CUDA tensors, updated in place.

    state_bits: 32 (float moments) or 8 (codes with a scale per 256 elements).
    rounding, of 8-bit moments: "seeded" rounds up or down by random numbers of
    the step, the tensor's place in the list and the element (results repeat), so
    that both averages are held without bias: the one to train with.  "nearest"
    (what None stands for, with a warning) loses every change below half a code:
    v does not fall again and m does not end, so it is for comparisons and a few
    steps.
    master: hold 16-bit parameters in float32 as well (``self.state["master"]``;
    None for a float32 one).  A step reads them there, so a parameter that is
    written by hand is written there too.
    state, step: resume; a dict of lists m, v (and m_scale, v_scale in 8 bits,
    master with master=True) as ``self.state`` holds them, and the steps taken.

    capturable: the steps taken are counted on the device, so that a step
    captured in a CUDA graph goes on at every replay; otherwise the number is
    part of the captured call, and every replay is that one step again.
    ``steps`` is the number of steps taken (capturable: reading it waits for the
    device).

    ``params`` and the lists of ``state`` are the caller's to change between
    calls: every call goes to the tensors that they hold then, wherever those
    have their storage, and refuses ones of another size or type.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, master=False, state=None, step=0, capturable=False,
                 rounding=None):
        self.params = list(params)
        if state_bits not in (8, 32):
            raise ValueError("state_bits %s: expected 8 or 32" % (state_bits,))
        if rounding is not None and rounding not in ROUNDINGS:
            raise ValueError("rounding %r: expected one of %s" % (rounding, tuple(ROUNDINGS)))
        if rounding is None and state_bits == 8:
            warnings.warn("8-bit moments rounded to the nearest code do not follow their averages "
                          "over more than a few steps: train with rounding=\"seeded\"",
                          stacklevel=2)
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self._count, self._steps = state_bits, None, int(step)
        for i, p in enumerate(self.params):
            if not torch.is_tensor(p) or p.device.type != "cuda":
                raise ValueError("params[%d] is not a CUDA tensor" % i)
        self._device = self.params[0].device if self.params else None
        self._given = [(p.numel(), p.dtype) for p in self.params]
        self._check_params()
        if capturable:
            self._count = torch.full((1,), int(step), dtype=torch.int64,
                                     device=self._device or "cuda")
        self.state = self._state(state, master)
        self._master = "master" in self.state
        self._opts, self._values = gmm_adamw_opts(), None
        self._opts.state_bits, self._opts.rounding = state_bits, ROUNDINGS[rounding or "nearest"]
        self._fill_table()

    @property
    def steps(self):
        return self._steps if self._count is None else int(self._count.item())

    @steps.setter
    def steps(self, n):
        if self._count is None:
            self._steps = int(n)
        else:
            self._count.fill_(int(n))

    def _check_params(self):
        if len(self.params) != len(self._given):
            raise ValueError("%d parameters, %d at first" % (len(self.params), len(self._given)))
        for i, (p, (n, dt)) in enumerate(zip(self.params, self._given)):
            _dense(p, "params[%d]" % i, n, (dt,) if dt in TORCH_XDTYPE else tuple(TORCH_XDTYPE),
                   self._device)

    def _flat(self):
        out = list(self.params)
        for ts in self.state.values():
            out += ts
        return out

    def _fill_table(self):
        """The tensors' addresses for the library, and what `_bind` knows them by."""
        # one launch writes them all, in no order
        _apart([("params[%d]" % i, p) for i, p in enumerate(self.params)]
               + [("state[%s][%d]" % (k, i), t) for k, ts in self.state.items()
                  for i, t in enumerate(ts)])
        self._table = (gmm_adamw_tensor * max(1, len(self.params)))()
        self._rows = [(self._table[i], n, self._device.index) for i, (n, _) in enumerate(self._given)]
        for i, p in enumerate(self.params):
            e = self._table[i]
            e.param, e.n, e.param_dtype = p.data_ptr(), p.numel(), TORCH_XDTYPE[p.dtype]
            for k, ts in self.state.items():
                setattr(e, k, ts[i].data_ptr() if ts[i] is not None else None)
        self._held = self._flat()
        self._lookups = [t.data_ptr for t in self._held if t is not None]
        for p in self.params:
            self._lookups += [p.numel, p.is_contiguous]
        self._found = [f() for f in self._lookups]
        self._types = [p.dtype for p in self.params]

    def _bind(self):
        """Brings the table up to date where a list holds another tensor than at
        the last call, or a tensor has other storage."""
        if self._device is not None:
            _here(self._device)
        flat = self._flat()
        if (len(flat) == len(self._held) and all(map(is_, flat, self._held))
                and [f() for f in self._lookups] == self._found
                and [p.dtype for p in self.params] == self._types):
            return
        self._check_params()
        self.state = self._state(self.state, self._master)
        self._fill_table()

    def _state(self, given, master):
        bits = self.state_bits
        types = {"m": torch.float32 if bits == 32 else torch.int8,
                 "v": torch.float32 if bits == 32 else torch.uint8}
        if bits == 8:
            types.update(m_scale=torch.float32, v_scale=torch.float32)
        out = {}
        for k, dt in types.items():
            size = (lambda p: -(-p.numel() // BLOCK)) if k.endswith("scale") else (lambda p: p.numel())
            if given is None:
                out[k] = [torch.zeros(size(p), dtype=dt, device=p.device) for p in self.params]
            else:
                out[k] = [_dense(t, "state[%s][%d]" % (k, i), size(p), (dt,), p.device)
                          for i, (t, p) in enumerate(zip(given[k], self.params, strict=True))]
        if master:
            low = [p.dtype != torch.float32 for p in self.params]
            if given is not None and "master" in given:
                out["master"] = [_dense(t, "state[master][%d]" % i, p.numel(), (torch.float32,),
                                        p.device) if l else None
                                 for i, (t, p, l) in enumerate(zip(given["master"], self.params, low,
                                                                   strict=True))]
            else:
                out["master"] = [p.detach().float().reshape(-1) if l else None
                                 for p, l in zip(self.params, low)]
        return out

    def step(self, grads, grad_scale=1.0, skip=None, stream=None):
        """One step with `grads` (one tensor per parameter), each multiplied by
        grad_scale; skip: an int32 device tensor, nothing changes where it is
        not 0 (the step still counts)."""
        if len(grads) != len(self.params):
            raise ValueError("%d gradients for %d parameters" % (len(grads), len(self.params)))
        self._bind()
        for g, (e, n, index) in zip(grads, self._rows):
            try:
                e.grad, e.grad_dtype = g.data_ptr(), TORCH_XDTYPE[g.dtype]
                if g.numel() == n and g.get_device() == index and g.is_contiguous():
                    continue
            except (AttributeError, KeyError, TypeError):
                pass
            for i, (g, (n, _)) in enumerate(zip(grads, self._given)):  # says which and why
                _dense(g, "grads[%d]" % i, n, tuple(TORCH_XDTYPE), self._device)
        if skip is not None:
            _dense(skip, "skip", 1, (torch.int32,), self._device or skip.device)
        o = self._opts
        values = (self.lr, self.betas, self.eps, self.weight_decay, grad_scale)
        if values != self._values:
            o.lr, (o.beta1, o.beta2), o.eps, o.weight_decay, o.grad_scale = values
            self._values = values
        o.step = self._steps + 1
        o.skip = skip.data_ptr() if skip is not None else None
        if self._count is None:
            if torch.cuda.is_current_stream_capturing():
                warnings.warn("AdamW.step captured without capturable=True: every replay of the "
                              "graph takes step %d again" % o.step, stacklevel=2)
            r = gmm_adamw_step(self._table, len(self.params), o, stream=stream)
            self._steps += 1
        else:
            r = gmm_adamw_step_counted(self._table, len(self.params), o, self._count,
                                       stream=stream)
        torch.autograd.graph.increment_version(self.params)  # autograd sees the change
        return r

    def moments(self, m_out=None, v_out=None, stream=None):
        """The moments in float32: two lists of tensors (given ones are written)."""
        self._bind()

        def outs(ts, name):
            if ts is None:
                return [_empty(p.shape, torch.float32, p.device, stream) for p in self.params]
            if len(ts) != len(self.params):
                raise ValueError("%s: %d tensors for %d parameters" % (name, len(ts), len(self.params)))
            for i, (t, p) in enumerate(zip(ts, self.params)):
                _dense(t, "%s[%d]" % (name, i), p.numel(), (torch.float32,), p.device)
            return ts
        m_out, v_out = outs(m_out, "m_out"), outs(v_out, "v_out")
        n = len(self.params)
        ptrs = lambda ts: (ctypes.c_void_p * max(1, n))(*[t.data_ptr() for t in ts])  # noqa: E731
        gmm_adamw_moments(self._table, n, self.state_bits, ptrs(m_out), ptrs(v_out), stream=stream)
        return m_out, v_out
