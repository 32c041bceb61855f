"""Muon, the optimiser for matrices: momentum, orthogonalised by Newton-Schulz
products before it is applied.

Argument marshalling only, as in ``training``: the work is done by libar.so's
HIP kernels, on the current stream unless a call names another.
"""

import ctypes
from array import array
from itertools import chain

import torch

from . import binding
from .binding import DTYPES, SUCCESS, ArError, MuonStep, MuonTensor, lib
from .training import _current_device, _current_stream, _flat, _handle, _in_use, _training


class Muon:
    """Muon over many matrices at once (see ar_muon_step).

    ``params`` are contiguous GPU tensors (float32 or bfloat16) of two or more
    dimensions; the last two are a matrix's rows and columns, those before count
    matrices that are treated one by one, as in the weights [experts, in, out]
    of a mixture of experts.  ``grads`` (float32 or bfloat16) have the same
    shapes, or are flat; ``copies`` optionally lists bfloat16 working copies of float32
    params, rewritten by every step.  Everything is checked once, here; the
    tensors' storage must not move while the object is in use, and every step
    reads the gradients from the same ``grads``.

    ``state`` hands over an existing ``{"momentum": [...]}`` (float32, shaped
    like ``grads``), updated in place; by default it starts at zero.  A step
    moves a matrix by ``lr`` times ``sqrt(max(1, rows / cols))``, or with
    ``match_rms`` times ``match_rms * sqrt(max(rows, cols))`` (0.2 gives updates
    of about AdamW's size), along the orthogonalised momentum.  The first is
    meant for weights that stand as [out, in], as torch's linear layers keep
    theirs; for [in, out], as in the experts' [experts, in, out], it gives its
    factor to the wrong ones of two matrices.  Take ``match_rms`` there, which is
    the same for both.  ``grad_scale`` multiplies every gradient first, e.g.
    ``1 / N`` where they are sums over N ranks.

    The object keeps memory on the GPU to work in, which the steps share: they
    must be ordered.  It is 8 bytes an element and 8 for each element of the
    shorter sides' squares, for all matrices at once, sides rounded up to a
    multiple of 64, or of 128 from 256 tiles of 128 x 128 in all on, and up to
    34 MB more; none where no matrix has more than 128 rows or columns.  The
    plan takes some 300 bytes a matrix or more.  A step may be captured into a
    graph, whose replays repeat it with its ``lr`` and are ordered with the
    other steps by the caller.
    """

    def __init__(self, params, grads, copies=None, *, state=None, momentum=0.95, nesterov=True,
                 ns_steps=5, eps=1e-7, weight_decay=0.0, match_rms=None, grad_scale=1.0):
        params = list(params)
        if not params:
            raise ValueError("need at least one parameter")
        if not isinstance(params[0], torch.Tensor) or not params[0].is_cuda:
            raise TypeError("params must be GPU tensors")
        dev = params[0].get_device()
        sizes = [p.numel() for p in params]
        real = (torch.float32, torch.bfloat16)
        self.params = _flat(params, "params", dev, real, sizes)
        if any(p.dim() < 2 for p in params):
            raise ValueError("params must be matrices, or tensors of matrices")
        self.grads = _flat(grads, "grads", dev, real, sizes)
        self.copies = None
        if copies is not None:
            if params[0].dtype != torch.float32:
                raise TypeError("copies are offered for float32 params only")
            self.copies = _flat(copies, "copies", dev, (torch.bfloat16,), sizes)
        if state is None:
            state = {"momentum": [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in params]}
        if set(state) != {"momentum"}:
            raise ValueError(f"state must hold ['momentum'], not {sorted(state)}")
        self.state = {"momentum": _flat(state["momentum"], "momentum", dev, (torch.float32,), sizes)}
        for what, tensors in (("grads", self.grads), ("copies", self.copies or []),
                              ("momentum", self.state["momentum"])):
            if any(t.dim() != 1 and t.shape != p.shape for t, p in zip(tensors, params)):
                raise ValueError(f"{what} must have the parameters' shapes, or be flat")
        if int(ns_steps) != ns_steps:
            raise ValueError("ns_steps must be a whole number")
        if match_rms is not None and not match_rms > 0:
            raise ValueError("match_rms must be positive")
        self._args = MuonStep(0.0, float(momentum), float(eps), float(weight_decay), float(grad_scale),
                              0.0 if match_rms is None else float(match_rms), 1 if nesterov else 0,
                              int(ns_steps))
        self._written = [t for ts in (self.params, self.copies or []) for t in ts]

        # a row of ar_muon_tensor_t per tensor
        none = [0] * len(params)
        columns = [[t.data_ptr() for t in ts] if ts else none
                   for ts in (self.params, self.grads, self.copies, self.state["momentum"])]
        shapes = [(p.shape[:-2].numel(), p.shape[-2], p.shape[-1]) for p in params]
        rows = array("Q", chain.from_iterable((*at, *shape) for at, shape in zip(zip(*columns), shapes)))
        table = (MuonTensor * len(params)).from_buffer(rows)
        kind = (len(params), DTYPES[binding._torch_dtype_name(params[0])],
                DTYPES[binding._torch_dtype_name(self.grads[0])])
        size = lib().ar_muon_plan_bytes(table, *kind)
        self._host = (ctypes.c_char * max(size, 16))()
        binding._check(lib().ar_muon_plan(table, *kind, self._host, size), "Muon")
        self._dev = dev
        with binding._on_device(dev):
            self._device = torch.frombuffer(self._host, dtype=torch.uint8).to(params[0].device)
            # (a step takes an address also where it works in none)
            self._workspace = torch.empty(max(lib().ar_muon_workspace_used(self._host), 256), dtype=torch.uint8,
                                          device=params[0].device)
        self._host_ptr, self._device_ptr = ctypes.addressof(self._host), self._device.data_ptr()
        self._workspace_ptr = self._workspace.data_ptr()
        self._step_args = ctypes.byref(self._args)
        self._streams = set()     # named streams that the tensors are known to be in use on
        self._fn = lib().ar_muon_step

    def step(self, lr, stream=None):
        """One step in place: params, copies and the momentum are overwritten,
        and autograd notices it for params and copies."""
        dev = self._dev
        if _current_device() != dev:
            with binding._on_device(dev):
                return self.step(lr, stream)
        self._args.lr = lr
        handle = _current_stream(dev) if stream is None else _handle(stream, dev)
        status = self._fn(self._host_ptr, self._device_ptr, self._workspace_ptr, self._step_args, handle)
        if status != SUCCESS:
            raise ArError(status, "step")
        # once a stream: the allocator remembers it for as long as a tensor lives
        if stream is not None and handle not in self._streams and \
                _in_use(stream, self.params, self.grads, self.copies, self.state["momentum"],
                        (self._device, self._workspace)):
            self._streams.add(handle)
        _training.written(self._written)
