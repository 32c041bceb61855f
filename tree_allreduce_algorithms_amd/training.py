"""The training step next to the collectives: AdamW over many tensors at once
and the router of a mixture of experts.

Argument marshalling only, as in ``binding``: the work is done by libar.so's
HIP kernels, on the current stream unless a call names another.  The calls
that take lists of tensors or allocate their results go through _training.so,
which is built with the library.

Where a call names a torch stream, the allocator is told that the tensors it
was given are in use there, so that they may be dropped after the call; what
it returns belongs to that stream.  Another library's stream (a raw handle or
a torch.cuda.ExternalStream) may be gone when a tensor is freed, so there the
caller keeps the tensors until the work is done.  Ordering the streams is the
caller's, as with every call of torch.
"""

import ctypes
import importlib.util
import os
from array import array
from itertools import chain

import torch

from . import binding
from .binding import DTYPES, SUCCESS, AdamwStep, AdamwTensor, ArError, lib

BLOCK = 256   # elements that share one scale of an 8-bit state
MAX_EXPERTS, MAX_TOP_K = 1024, 8
ROUTE_WORKSPACE = 2386432   # AR_ROUTE_WORKSPACE


def _load_module():
    path = os.path.join(binding.PKG, "_training.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run "
                           "`python -m tree_allreduce_algorithms_amd.build_lib` first")
    lib()       # the library that it calls, from the same folder
    spec = importlib.util.spec_from_file_location("_training", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_training = _load_module()
_INF = float("inf")


def _current_stream(dev):
    """hipStream_t of the current stream of device `dev`."""
    return torch.cuda.current_stream(dev).cuda_stream


# the same numbers without objects and initialisation around them, where torch
# offers that (a GPU tensor is at hand, so the device is initialised)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _handle(stream, dev):
    """hipStream_t of a torch stream, a raw handle, or (None) the current stream."""
    if stream is None:
        return _current_stream(dev)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _capturing(stream, handle, dev):
    """Whether `stream` (None: the current one), of this handle, is being
    captured into a graph.  The null stream cannot be."""
    if not handle:
        return False
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(_stream_of(stream, dev)):
        return torch.cuda.is_current_stream_capturing()


def _stream_of(stream, dev):
    """`stream` (a torch stream or a raw handle), or the current one of device `dev`."""
    if stream is None:
        return torch.cuda.current_stream(dev)
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=dev)


def _in_use(stream, *groups):
    """Tells the allocator that these tensors (lists of them, None for none) are
    in use on `stream`, a call's argument (see above); whether it was told."""
    if not isinstance(stream, torch.cuda.Stream) or isinstance(stream, torch.cuda.ExternalStream):
        return False
    for group in groups:
        for t in group or ():
            t.record_stream(stream)
    return True


def _flat(tensors, what, dev, dtypes, sizes):
    """`tensors` as a list: contiguous GPU tensors of one of `dtypes` (all the
    same) on `dev`, of these sizes."""
    tensors = list(tensors)
    if len(tensors) != len(sizes):
        raise ValueError(f"{what}: {len(tensors)} tensors for {len(sizes)} parameters")
    kind = getattr(tensors[0], "dtype", None)
    for t, n in zip(tensors, sizes):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{what} must be GPU tensors")
        if t.dtype is not kind or kind not in dtypes:
            raise TypeError(f"{what}: unsupported or mixed dtype {t.dtype}")
        if t.get_device() != dev or t.numel() != n:
            raise ValueError(f"{what} must share the parameters' device and sizes")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
    return tensors


class AdamW:
    """AdamW over many tensors, one launch a step (see ar_adamw_step).

    ``params`` and ``grads`` are lists of contiguous GPU tensors (float32 or
    bfloat16 each), for instance the shards that ``reduce_scatter`` leaves
    with their owners; ``copies`` optionally lists bfloat16 working copies of
    float32 params, rewritten by every step.  Everything is checked once,
    here; the tensors' storage must not move while the object is in use, and
    every step reads the gradients from the same ``grads``.

    ``state_bits`` is 32 (``exp_avg`` and ``exp_avg_sq`` in float32) or 8
    (int8 and uint8 codes, with one float32 scale per 256 elements of a tensor
    in ``exp_avg_scale`` and ``exp_avg_sq_scale``; see ar_adamw_tensor_t and
    ``dequantize``).  ``state`` hands over existing lists of these names, which
    are updated in place; by default they start at zero.  ``steps`` counts the
    steps taken so far.  ``grad_scale`` multiplies every gradient first, e.g.
    ``1 / N`` where they are sums over N ranks.

    Calls run on the current stream, or on ``stream``; those of one object must
    be ordered.  ``grad_norm`` may be captured into a graph, ``step`` may not
    (its bias corrections are those of one step).  Once a bounded norm has been
    captured, ``step(clip=True)`` is taken without an eager one before it, and
    it is the caller who replays the graph before each such step: nothing here
    sees a replay, and without one the step has the factor of the norm before
    (NaN if there was none).
    """

    def __init__(self, params, grads, copies=None, *, state_bits=32, state=None, steps=0,
                 betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=1.0):
        params = list(params)
        if not params:
            raise ValueError("need at least one parameter")
        if not isinstance(params[0], torch.Tensor) or not params[0].is_cuda:
            raise TypeError("params must be GPU tensors")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, not {state_bits!r}")
        if int(steps) != steps or steps < 0:
            raise ValueError("steps must be a whole number of steps taken, at least 0")
        dev = params[0].get_device()
        sizes = [p.numel() for p in params]
        real = (torch.float32, torch.bfloat16)
        self.params = _flat(params, "params", dev, real, sizes)
        self.grads = _flat(grads, "grads", dev, real, sizes)
        self.copies = None
        if copies is not None:
            if params[0].dtype != torch.float32:
                raise TypeError("copies are offered for float32 params only")
            self.copies = _flat(copies, "copies", dev, (torch.bfloat16,), sizes)
        kinds = {"exp_avg": (torch.float32, sizes), "exp_avg_sq": (torch.float32, sizes)}
        if state_bits == 8:
            blocks = [-(-n // BLOCK) for n in sizes]
            kinds = {"exp_avg": (torch.int8, sizes), "exp_avg_sq": (torch.uint8, sizes),
                     "exp_avg_scale": (torch.float32, blocks),
                     "exp_avg_sq_scale": (torch.float32, blocks)}
        if state is None:
            state = {k: [torch.zeros(n, dtype=dt, device=params[0].device) for n in ns]
                     for k, (dt, ns) in kinds.items()}
        if set(state) != set(kinds):
            raise ValueError(f"state must hold {sorted(kinds)}, not {sorted(state)}")
        self.state = {k: _flat(state[k], k, dev, (dt,), ns) for k, (dt, ns) in kinds.items()}
        self.state_bits, self.steps = state_bits, int(steps)
        self._clip_ready = False      # a bounded norm was enqueued since the last step
        self._clip_captured = False   # one is in a graph, whose replays are not seen here
        self._args = AdamwStep(0.0, float(betas[0]), float(betas[1]), float(eps),
                               float(weight_decay), float(grad_scale), 0, 0)
        self._grad_scale = float(grad_scale)

        self._written = [t for ts in (self.params, self.copies or []) for t in ts]

        # a row of ar_adamw_tensor_t per tensor
        none = [0] * len(params)
        columns = [[t.data_ptr() for t in ts] if ts else none
                   for ts in (self.params, self.grads, self.copies,
                              *(self.state.get(k) for k in ("exp_avg", "exp_avg_sq", "exp_avg_scale",
                                                            "exp_avg_sq_scale")))]
        rows = array("Q", chain.from_iterable(zip(*columns, sizes)))
        table = (AdamwTensor * len(params)).from_buffer(rows)
        kind = (len(params), DTYPES[binding._torch_dtype_name(params[0])],
                DTYPES[binding._torch_dtype_name(self.grads[0])], state_bits)
        size = lib().ar_adamw_plan_bytes(table, *kind)
        self._host = (ctypes.c_char * max(size, 16))()
        binding._check(lib().ar_adamw_plan(table, *kind, self._host, size), "AdamW")
        self._dev = dev
        with binding._on_device(dev):
            self._norm = torch.zeros((), dtype=torch.float32, device=params[0].device)
            self._device = torch.frombuffer(self._host, dtype=torch.uint8).to(params[0].device)
        self._host_ptr, self._device_ptr = ctypes.addressof(self._host), self._device.data_ptr()
        self._norm_ptr = self._norm.data_ptr()
        self._step_args = ctypes.byref(self._args)
        self._streams = set()     # named streams that the tensors are known to be in use on
        self._fn_norm, self._fn_step = lib().ar_adamw_grad_norm, lib().ar_adamw_step

    def _on(self, stream, handle):
        # once a stream: the allocator remembers it for as long as a tensor lives
        if handle not in self._streams and \
                _in_use(stream, self.params, self.grads, self.copies, *self.state.values(),
                        (self._device, self._norm)):
            self._streams.add(handle)

    def grad_norm(self, max_norm=None, stream=None):
        """The 2-norm over all gradients (times ``grad_scale``), a float32 GPU
        scalar that the next call overwrites.  With ``max_norm`` the factor
        ``min(1, max_norm / norm)`` is kept for ``step(clip=True)``; nothing
        waits for the GPU."""
        dev = self._dev
        if _current_device() != dev:
            with binding._on_device(dev):
                return self.grad_norm(max_norm, stream)
        handle = _current_stream(dev) if stream is None else _handle(stream, dev)
        status = self._fn_norm(self._host_ptr, self._device_ptr, _INF if max_norm is None else max_norm,
                               self._grad_scale, self._norm_ptr, handle)
        if status != SUCCESS:
            raise ArError(status, "grad_norm")
        if stream is not None:
            self._on(stream, handle)
        if max_norm is not None and _capturing(stream, handle, dev):
            self._clip_captured = True
        else:
            self._clip_ready = max_norm is not None
        return self._norm

    def step(self, lr, clip=False, stream=None):
        """One step in place: params, copies and states are overwritten, and
        autograd notices it for params and copies.  ``clip=True`` scales the gradients by the factor
        of ``grad_norm(max_norm=...)``, which must have been called since the
        step before, or be part of a graph that has been replayed since."""
        if clip and not (self._clip_ready or self._clip_captured):
            raise ValueError("step(clip=True) needs grad_norm(max_norm=...) on these gradients first")
        dev = self._dev
        if _current_device() != dev:
            with binding._on_device(dev):
                return self.step(lr, clip, stream)
        args = self._args
        args.lr, args.step, args.clip = lr, self.steps + 1, 1 if clip else 0
        handle = _current_stream(dev) if stream is None else _handle(stream, dev)
        status = self._fn_step(self._host_ptr, self._device_ptr, self._step_args, handle)
        if status != SUCCESS:
            raise ArError(status, "step")
        if stream is not None:
            self._on(stream, handle)
        self.steps += 1
        self._clip_ready = False
        # a backward pass that saved one of these before the step must not
        # take the new values for the old
        _training.written(self._written)


def dequantize(codes, scales, stream=None):
    """float32 values of the codes of an 8-bit AdamW state: int8 codes of
    ``exp_avg`` or uint8 codes of ``exp_avg_sq``, with one scale per 256."""
    dev = codes.get_device() if isinstance(codes, torch.Tensor) else -1
    if dev < 0:
        raise TypeError("codes and scales must be GPU tensors")
    if stream is not None or _current_device() != dev:
        # the result belongs to that stream: its memory is not handed out
        # again before the kernel there has run
        with torch.cuda.stream(_stream_of(stream, dev)):
            out = dequantize(codes, scales)
        _in_use(stream, (codes, scales))
        return out
    status, out = _training.dequantize(codes, scales, _current_stream(dev))
    if status != SUCCESS:
        raise ArError(status, "dequantize")
    return out


# --- the router ------------------------------------------------------------------

class Routing:
    """What ``route`` found, for the expert exchange and for ``route_grad``:
    ``indices`` [ranks, tokens, top_k] int32, ``weights`` (same shape, float32),
    ``counts`` [ranks, experts] int32, ``loss`` (float32 scalar) and ``share``
    [experts] float32 (see ar_route).  It keeps the masks, which must be as
    they were when ``route_grad`` looks at them again."""

    __slots__ = ("indices", "weights", "counts", "loss", "share", "_dtype", "_mask", "_renormalize")

    def __init__(self, indices, weights, counts, loss, share, dtype, mask, renormalize):
        self.indices, self.weights, self.counts = indices, weights, counts
        self.loss, self.share, self._dtype = loss, share, dtype
        self._mask, self._renormalize = mask, renormalize


_route_workspaces = {}   # (device index, stream handle) -> workspace


def _route_workspace(dev, handle):
    """The current stream's workspace, which every call leaves ready for the
    next: one for each of torch's own streams, which last as long as the
    process.  Other calls get one of their own, cleared on the stream: captured
    ones, whose replays may run beside the stream's other calls (the null
    stream cannot be captured), and those on another library's stream, whose
    handle may come back as that of a new stream beside the old one's work."""
    if handle and torch.cuda.is_current_stream_capturing():
        return torch.zeros(ROUTE_WORKSPACE, dtype=torch.uint8, device=f"cuda:{dev}")
    ws = _route_workspaces.get((dev, handle))
    if ws is None:
        ws = torch.zeros(ROUTE_WORKSPACE, dtype=torch.uint8, device=f"cuda:{dev}")
        if not handle or torch.cuda.current_stream(dev).stream_id != handle:   # an external stream's id is its handle
            _route_workspaces[dev, handle] = ws
    return ws


def _list(tensors):
    return tensors if tensors is None or type(tensors) is list else list(tensors)


def route(logits, top_k, mask=None, renormalize=False, stream=None):
    """Chooses ``top_k`` experts for every token (see ar_route).

    ``logits`` lists one [tokens, experts] tensor a rank (float32 or bfloat16;
    rows may be strided); ``mask`` optionally lists one boolean [tokens] tensor
    a rank, False for what is no token.  Returns a ``Routing``.  Up to 1,024
    experts and 8 choices.

    Autograd records nothing: the outputs have no ``grad_fn``, whatever the
    logits have.  Where a graph made the logits, hand it their gradient:
    ``torch.autograd.backward(logits, list(route_grad(logits, r, ...)))``."""
    logits, mask = _list(logits), _list(mask)
    dev = _training.device(logits)
    if stream is not None or _current_device() != dev:
        with torch.cuda.stream(_stream_of(stream, dev)):
            routing = route(logits, top_k, mask, renormalize)
        _in_use(stream, logits, mask)
        return routing
    handle = _current_stream(dev)
    workspace = _route_workspace(dev, handle)
    status, *outputs = _training.route(logits, top_k, mask, renormalize, workspace.data_ptr(), handle)
    if status != SUCCESS:
        raise ArError(status, "route")
    return Routing(*outputs, logits[0].dtype, mask, renormalize)


def route_grad(logits, routing, dweights=None, dloss=None, stream=None):
    """Gradient of ``sum(dweights * weights) + dloss * loss`` with respect to
    the logits, [ranks, tokens, experts] of their type (see ar_route_grad).

    ``logits`` are those that ``route`` took for ``routing``; ``dweights``
    lists one float32 [tokens, top_k] tensor a rank, ``dloss`` is a float32 GPU
    scalar; either may be left out."""
    logits, dweights = _list(logits), _list(dweights)
    dev = _training.device(logits)
    if stream is not None or _current_device() != dev:
        with torch.cuda.stream(_stream_of(stream, dev)):
            dlogits = route_grad(logits, routing, dweights, dloss)
        _in_use(stream, logits, routing._mask, dweights, () if dloss is None else (dloss,),
                (routing.indices, routing.share))
        return dlogits
    status, dlogits = _training.route_grad(logits, routing._dtype, routing.indices, routing.share,
                                           routing._mask, routing._renormalize, dweights, dloss,
                                           _current_stream(dev))
    if status != SUCCESS:
        raise ArError(status, "route_grad")
    return dlogits
