"""CPU tests of the training calls of the C ABI: plans, argument errors and
the reported launch failure.  Nothing is launched (an armed injection stands in
for the launch), so the fake device addresses are never dereferenced."""

import ctypes
import os

import pytest

import tree_allreduce_algorithms_amd as ar
from tree_allreduce_algorithms_amd import binding
from tree_allreduce_algorithms_amd.binding import AdamwStep, AdamwTensor, RouteShape

INT32, F32, BF16, ACC32 = 0, 1, 2, 3
OK, INVALID, UNSUPPORTED, HIP = (binding.SUCCESS, binding.INVALID_ARGUMENT, binding.UNSUPPORTED,
                                 binding.HIP_ERROR)
GAP = 1 << 36


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    yield
    ar.debug_fail_launch(0)


def tensors(counts, bits=32, copy=False, base=0x7F0000000000):
    """Tensors at distinct, aligned fake addresses."""
    out = []
    for i, n in enumerate(counts):
        at = lambda k: base + (8 * i + k) * GAP  # noqa: E731
        out.append(AdamwTensor(at(0), at(1), at(2) if copy else None, at(3), at(4),
                               at(5) if bits == 8 else None, at(6) if bits == 8 else None, n))
    return out


def plan(ts, pd=F32, gd=F32, bits=32):
    """(status, host image or None) of a plan."""
    table = (AdamwTensor * max(1, len(ts)))(*ts)
    lib = ar.lib()
    size = lib.ar_adamw_plan_bytes(table, len(ts), pd, gd, bits)
    image = (ctypes.c_char * max(size, 16))()
    status = lib.ar_adamw_plan(table, len(ts), pd, gd, bits, image, size)
    assert (size > 0) == (status == OK)
    return status, image if status == OK else None


def tiles_of(image):
    """(tensor, first element, end) of every tile: the image's head is sixteen
    32-bit words of sizes and offsets, as the kernels read it."""
    head = (ctypes.c_uint32 * 8).from_buffer(image)
    _, ntensors, ntiles, per = head[:4]
    at = (ctypes.c_uint64 * 4).from_buffer(image, 32)
    raw = (ctypes.c_uint32 * (2 * ntiles)).from_buffer(image, at[3])
    return ntensors, per, [(raw[2 * i], raw[2 * i + 1]) for i in range(ntiles)]


@pytest.mark.parametrize("counts", [[1], [1024, 1, 1025], [0, 5, 0, 4096, 0], [300_000_000] * 2,
                                    [7] * 1000, [(1 << 33) + 5]])
def test_plan_tiles_cover_every_element_once(counts):
    status, image = plan(tensors(counts))
    assert status == OK
    ntensors, per, tiles = tiles_of(image)
    live = [n for n in counts if n]
    assert ntensors == len(live) and per % 1024 == 0
    want = [(i, j) for i, n in enumerate(live) for j in range(-(-n // per))]
    assert tiles == want


def test_plan_of_empty_tensors_only():
    status, image = plan(tensors([0, 0]))
    assert status == OK and tiles_of(image)[2] == []
    args = AdamwStep(1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0, 1, 0)
    ar.debug_fail_launch(1)
    try:    # nothing to do: no launch is made
        assert ar.lib().ar_adamw_step(image, 0x7F0000000000, ctypes.byref(args), None) == OK
    finally:
        ar.debug_fail_launch(0)


def change(ts, i, **fields):
    for k, v in fields.items():
        setattr(ts[i], k, v)
    return ts


A = 0x7F0000000000


@pytest.mark.parametrize("ts, kind, want", [
    ([], {}, INVALID),
    (tensors([4]), {"pd": INT32}, UNSUPPORTED),
    (tensors([4]), {"gd": ACC32}, UNSUPPORTED),
    (tensors([4]), {"bits": 16}, UNSUPPORTED),
    (change(tensors([4, 4]), 1, param=None), {}, INVALID),
    (change(tensors([4, 4]), 1, grad=None), {}, INVALID),
    (change(tensors([4]), 0, exp_avg=None), {}, INVALID),
    (change(tensors([4]), 0, exp_avg_sq=None), {}, INVALID),
    (change(tensors([4]), 0, param=A + 2), {}, INVALID),               # misaligned
    (change(tensors([4]), 0, grad=A + GAP + 1), {"gd": BF16}, INVALID),
    (change(tensors([4], 8), 0, exp_avg_scale=A + 5 * GAP + 2), {"bits": 8}, INVALID),
    (tensors([4]), {"bits": 8}, INVALID),                              # scales missing
    (tensors([4], 8), {"bits": 32}, INVALID),                          # scales given
    (tensors([4], copy=True), {"pd": BF16}, INVALID),                  # a copy of bfloat16
    (change(tensors([4, 4], copy=True), 1, copy=None), {}, INVALID),   # copies of some
    (change(tensors([4]), 0, exp_avg=A), {}, INVALID),                 # m over p
    (change(tensors([4, 8]), 1, param=A + 12), {}, INVALID),           # p over the other's tail
    (change(tensors([4]), 0, grad=A), {}, INVALID),                    # g over p
    (change(tensors([300], 8), 0, exp_avg_sq_scale=A + 5 * GAP + 4), {"bits": 8}, INVALID),
    (change(tensors([4]), 0, count=1 << 62), {}, INVALID),             # past the address space
])
def test_plan_refusals(ts, kind, want):
    assert plan(ts, **kind)[0] == want


def test_plan_takes_neighbours_shared_gradients_and_odd_addresses():
    ts = change(tensors([4, 4]), 1, param=A + 16, grad=A + GAP)         # one gradient read twice
    assert plan(ts)[0] == OK
    ts = change(tensors([5], 8), 0, exp_avg=A + 3 * GAP + 1, param=A + 4)
    assert plan(ts, bits=8)[0] == OK
    short = (ctypes.c_char * 16)()
    table = (AdamwTensor * 1)(*tensors([4]))
    assert ar.lib().ar_adamw_plan(table, 1, F32, F32, 32, short, 16) == INVALID
    assert ar.lib().ar_adamw_plan(table, 1, F32, F32, 32, None, 1 << 20) == INVALID
    assert ar.lib().ar_adamw_plan(None, 1, F32, F32, 32, short, 16) == INVALID


GOOD = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, grad_scale=1.0, step=1)


@pytest.mark.parametrize("bad", [
    {"lr": -1.0}, {"lr": float("nan")}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0},
    {"beta2": float("nan")}, {"eps": -1e-8}, {"weight_decay": -0.1}, {"grad_scale": float("inf")},
    {"step": 0}, {"step": -3}])
def test_step_refusals(bad):
    _, image = plan(tensors([4]))
    args = AdamwStep(**{**GOOD, **bad})
    assert ar.lib().ar_adamw_step(image, A, ctypes.byref(args), None) == INVALID


def test_calls_refuse_what_is_no_plan():
    lib, args = ar.lib(), AdamwStep(**GOOD)
    _, image = plan(tensors([4]))
    zeros = (ctypes.c_char * 4096)()
    for host, dev in ((None, A), (zeros, A), (image, None), (image, A + 8)):
        assert lib.ar_adamw_step(host, dev, ctypes.byref(args), None) == INVALID
        assert lib.ar_adamw_grad_norm(host, dev, 1.0, 1.0, None, None) == INVALID
    assert lib.ar_adamw_step(image, A, None, None) == INVALID
    assert lib.ar_adamw_grad_norm(image, A, -1.0, 1.0, None, None) == INVALID
    assert lib.ar_adamw_grad_norm(image, A, float("nan"), 1.0, None, None) == INVALID
    assert lib.ar_adamw_grad_norm(image, A, 1.0, float("nan"), None, None) == INVALID
    assert lib.ar_adamw_grad_norm(image, A, 1.0, 1.0, A + 2, None) == INVALID


def test_dequantize_refusals():
    f = ar.lib().ar_adamw_dequantize
    assert f(None, None, 0, 1, None, None) == OK                       # nothing to do
    assert f(None, A, 4, 1, A + GAP, None) == INVALID
    assert f(A, None, 4, 1, A + GAP, None) == INVALID
    assert f(A, A + GAP, 4, 1, None, None) == INVALID
    assert f(A, A + GAP + 2, 4, 1, A + 2 * GAP, None) == INVALID
    assert f(A, A + GAP, 4, 1, A + 2 * GAP + 1, None) == INVALID
    assert f(A, A + GAP, 4, 1, A, None) == INVALID                     # over its codes
    assert f(A, A + GAP, 4, 1, A + GAP - 12, None) == INVALID          # over its scales
    assert f(A, A + GAP, 1 << 62, 1, A + 2 * GAP, None) == INVALID


def test_injected_launch_failures_are_reported():
    lib, args = ar.lib(), AdamwStep(**GOOD)
    _, image = plan(tensors([4]))
    calls = [lambda: lib.ar_adamw_step(image, A, ctypes.byref(args), None),
             lambda: lib.ar_adamw_grad_norm(image, A, 1.0, 1.0, None, None),
             lambda: lib.ar_adamw_dequantize(A, A + GAP, 4, 1, A + 2 * GAP, None)]
    for call in calls:
        ar.debug_fail_launch(1)
        assert call() == HIP
        assert lib.ar_last_hip_error() == 719


def test_python_refusals_need_no_gpu():
    import torch
    x = torch.zeros(4)
    with pytest.raises(ValueError, match="at least one"):
        ar.AdamW([], [])
    with pytest.raises(TypeError, match="GPU"):
        ar.AdamW([x], [x])
    with pytest.raises(TypeError, match="GPU"):
        ar.dequantize(x, x)


# --- the router ---------------------------------------------------------------------

def addresses(n, first=A):
    return (ctypes.c_void_p * n)(*[first + i * GAP for i in range(n)]) if n else None


def route_call(shape, logits="default", masks=None, outs=None, workspace=A + 200 * GAP):
    outs = outs or [A + (100 + i) * GAP for i in range(5)]
    logits = addresses(max(1, min(shape.nranks, 64))) if logits == "default" else logits
    return ar.lib().ar_route(logits, masks, ctypes.byref(shape), *outs, workspace, None)


def grad_call(shape, logits="default", masks=None, indices=A + 100 * GAP, share=A + 101 * GAP,
              dweights=None, dloss=None, dlogits=A + 102 * GAP):
    logits = addresses(max(1, min(shape.nranks, 64))) if logits == "default" else logits
    return ar.lib().ar_route_grad(logits, masks, ctypes.byref(shape), indices, share, dweights, dloss,
                                  dlogits, None)


def shape(nranks=2, tokens=5, experts=16, row_stride=None, top_k=2, renormalize=0, dtype=F32):
    return RouteShape(nranks, tokens, experts, experts if row_stride is None else row_stride, top_k,
                      renormalize, dtype)


@pytest.mark.parametrize("kw, want", [
    ({"nranks": 0}, INVALID), ({"nranks": 65}, INVALID), ({"experts": 0}, INVALID),
    ({"top_k": 0}, INVALID), ({"top_k": 17}, INVALID), ({"row_stride": 15}, INVALID),
    ({"dtype": INT32}, UNSUPPORTED), ({"dtype": ACC32}, UNSUPPORTED),
    ({"experts": 1025}, UNSUPPORTED), ({"top_k": 9}, UNSUPPORTED),
    ({"tokens": 1 << 31}, UNSUPPORTED), ({"tokens": (1 << 30) - 1, "row_stride": 1 << 34}, INVALID)])
def test_router_shape_refusals(kw, want):
    assert route_call(shape(**kw)) == want
    assert grad_call(shape(**kw)) == want


def test_router_pointer_refusals():
    s = shape()
    two = lambda *p: (ctypes.c_void_p * 2)(*p)  # noqa: E731
    for call in (route_call, grad_call):
        assert call(s, logits=None) == INVALID
        assert call(s, logits=two(A, None)) == INVALID
        assert call(s, logits=two(A, A + GAP + 2)) == INVALID
        assert call(s, masks=two(A, None)) == INVALID
    good = [A + (100 + i) * GAP for i in range(5)]
    for i in range(5):
        for bad in (None, good[i] + 2):
            assert route_call(s, outs=good[:i] + [bad] + good[i + 1:]) == INVALID
    assert route_call(s, workspace=None) == INVALID
    assert route_call(s, workspace=A + 8) == INVALID
    assert grad_call(s, indices=None) == INVALID
    assert grad_call(s, share=None) == INVALID
    assert grad_call(s, dlogits=None) == INVALID
    assert grad_call(s, dlogits=A + 2) == INVALID
    assert grad_call(s, dloss=A + 2) == INVALID
    assert grad_call(s, dweights=two(A, None)) == INVALID
    assert grad_call(s, dweights=two(A, A + GAP + 2)) == INVALID
    assert ar.lib().ar_route(addresses(2), None, None, *good, A, None) == INVALID


def test_router_injected_launch_failures():
    for call in (route_call, grad_call):
        ar.debug_fail_launch(1)
        assert call(shape()) == HIP
        assert ar.lib().ar_last_hip_error() == 719
    assert grad_call(shape(tokens=0), logits=addresses(2)) == OK       # nothing to do


def test_router_python_refusals_need_no_gpu():
    import torch
    with pytest.raises(ValueError, match="ranks"):
        ar.route([], 1)
    with pytest.raises(TypeError, match="GPU"):
        ar.route([torch.zeros(4, 8)], 1)


def test_router_workspace_size_is_the_headers():
    from tree_allreduce_algorithms_amd import training
    text = open(os.path.join(os.path.dirname(binding.PKG), "include", "ar.h")).read()
    for name, value in (("AR_ROUTE_WORKSPACE", training.ROUTE_WORKSPACE),
                        ("AR_MAX_EXPERTS", training.MAX_EXPERTS), ("AR_MAX_TOP_K", training.MAX_TOP_K),
                        ("AR_ADAMW_BLOCK", training.BLOCK)):
        assert f"#define {name} {value}\n" in text
