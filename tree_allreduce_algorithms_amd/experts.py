"""The experts' products: what follows the router, forward and backward.

``expert_order`` puts the chosen (token, choice) pairs in order by expert, and
the products take their rows in that order, as many for each expert as chose
it; the counts stay on the GPU.  A layer of experts with a nonlinearity ``f``:

    r = ar.route(logits, top_k)
    o = ar.expert_order(r.indices, experts)
    h = ar.expert_matmul(x, w1, o, gather=True)
    y = ar.expert_matmul(f(h), w2, o)
    out = ar.expert_combine(y, o, r.weights)

and backward:

    dy, dweights = ar.expert_combine_grad(dout, y, o, r.weights)
    dw2 = ar.expert_weight_grad(f(h), dy, o)
    dh = f'(h) * ar.expert_matmul(dy, w2.transpose(1, 2), o)
    dw1 = ar.expert_weight_grad(x, dh, o, gather=True)
    dx = ar.expert_combine(ar.expert_matmul(dh, w1.transpose(1, 2), o), o)

Matrices are bfloat16; sums are float32 and rounded once, where a result is
stored.  Autograd records nothing of these calls.  They run on the current
stream, or on ``stream``, which is treated as in ``training``.
"""

import torch

from .binding import ArError
from .training import _current_device, _current_stream, _in_use, _stream_of, _training


class ExpertOrder:
    """The pairs of ``expert_order`` in order (see ar_expert_order): ``order``
    [pairs] int32, the pairs ``token * top_k + choice`` by expert, -1 behind the
    last that has one; ``position`` [..., top_k] int32, each pair's row, -1 for
    none; ``offsets`` [experts + 1] int32, where each expert's rows begin."""

    __slots__ = ("order", "position", "offsets", "top_k")

    def __init__(self, order, position, offsets, top_k):
        self.order, self.position, self.offsets, self.top_k = order, position, offsets, top_k


_training.hooks(_current_device, _current_stream, ExpertOrder, ArError)


def _elsewhere(call, first, stream, used, order=None):
    """`call()` with `stream` current, or (None) the current stream of the device
    of `first`; `used` and the order's tensors are what it reads or writes."""
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise TypeError("tensors must be GPU tensors")
    with torch.cuda.stream(_stream_of(stream, first.get_device())):
        result = call()
    if order is not None:
        used += (order.order, order.position, order.offsets)
    _in_use(stream, [t for t in used if isinstance(t, torch.Tensor)])
    return result


def expert_order(indices, experts, stream=None):
    """The order of the pairs by expert, as an ``ExpertOrder``: stable, so that
    an expert's rows are in the order of their tokens.  ``indices`` is a
    contiguous int32 GPU tensor [..., top_k], for instance a routing's or one
    rank's of it; a number outside [0, experts) is no expert.  Up to 1,024
    experts."""
    found = _training.expert_order(indices, experts) if stream is None else None
    if found is None:
        return _elsewhere(lambda: expert_order(indices, experts), indices, stream, (indices,))
    return ExpertOrder(*found, indices.shape[-1])


def expert_matmul(x, weight, order, gather=False, stream=None):
    """Every row times its expert's matrix: [pairs, out] bfloat16, rows in order,
    0 for those without an expert (see ar_expert_matmul).

    ``x`` is [pairs, in], rows in order, or with ``gather`` [tokens, in], from
    which each pair takes its token's row; rows may be strided.  ``weight`` is
    [experts, in, out], an expert's rows or its columns contiguous, so that
    ``weight.transpose(1, 2)`` gives the gradient with respect to the rows."""
    y = _training.expert_matmul(x, weight, order, gather) if stream is None else None
    if y is None:
        return _elsewhere(lambda: expert_matmul(x, weight, order, gather), x, stream, (x, weight), order)
    return y


def expert_weight_grad(x, dy, order, gather=False, dtype=torch.float32, out=None, stream=None):
    """The weights' gradient [experts, in, out]: for each expert the sum over its
    rows of x^T dy, 0 for an expert without rows (see ar_expert_weight_grad).

    ``x`` and ``gather`` are those of the product, ``dy`` [pairs, out] is the
    gradient of its rows.  ``dtype`` is float32 or bfloat16; ``out``, contiguous
    and of either type, is overwritten instead of a new tensor."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dtype must be float32 or bfloat16, not {dtype}")
    dw = _training.expert_weight_grad(x, dy, order, gather, dtype is torch.float32, out) if stream is None else None
    if dw is None:
        return _elsewhere(lambda: expert_weight_grad(x, dy, order, gather, dtype, out), x, stream, (x, dy, out),
                          order)
    return dw if out is None else out


def expert_combine(y, order, weights=None, stream=None):
    """The tokens' sums [tokens, size] bfloat16: the rows ``y`` [pairs, size] of a
    token's choices, times ``weights`` (float32, one a pair; None: 1), added up
    in float32 in the order of the choices (see ar_expert_combine).  Without
    weights it is also the gradient of the rows that ``gather`` takes."""
    sums = _training.expert_combine(y, order, weights) if stream is None else None
    if sums is None:
        return _elsewhere(lambda: expert_combine(y, order, weights), y, stream, (y, weights), order)
    return sums


def expert_combine_grad(dout, y, order, weights, stream=None):
    """Gradients of ``expert_combine(y, order, weights)``, given ``dout`` [tokens,
    size]: those of the rows, [pairs, size] bfloat16 (0 for rows without a
    pair), and of the weights, [tokens, top_k] float32 (0 for a choice without
    an expert)."""
    grads = _training.expert_combine_grad(dout, y, order, weights) if stream is None else None
    if grads is None:
        return _elsewhere(lambda: expert_combine_grad(dout, y, order, weights), dout, stream, (dout, y, weights),
                          order)
    return grads
