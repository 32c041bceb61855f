"""CPU tests of the experts' and Muon's calls of the C ABI: plans, argument
errors and the reported launch failure.  Nothing is launched (an armed
injection stands in for the launch), so the fake device addresses are never
dereferenced."""

import ctypes
import os

import pytest

import tree_allreduce_algorithms_amd as ar
from tree_allreduce_algorithms_amd import binding
from tree_allreduce_algorithms_amd.binding import ExpertRows, MuonStep, MuonTensor

INT32, F32, BF16 = 0, 1, 2
OK, INVALID, UNSUPPORTED, HIP = (binding.SUCCESS, binding.INVALID_ARGUMENT, binding.UNSUPPORTED,
                                 binding.HIP_ERROR)
A, GAP = 0x7F0000000000, 1 << 36


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    yield
    ar.debug_fail_launch(0)


def launched(call):
    """The status of a call whose launch is made to fail: HIP if it got that far."""
    ar.debug_fail_launch(1)
    try:
        return call()
    finally:
        ar.debug_fail_launch(0)


def at(i):
    return A + i * GAP


# --- experts -----------------------------------------------------------------------

def rows(**change):
    r = dict(x=at(0), x_rows=100, x_stride=64, order=at(1), top_k=2, offsets=at(2), pairs=200, experts=8,
             inputs=64, outputs=96, dtype=BF16)
    r.update(change)
    return ExpertRows(**r)


def order(pairs=200, experts=8, indices=at(0), out=at(1), position=at(2), offsets=at(3), workspace=None):
    return launched(lambda: ar.lib().ar_expert_order(indices, pairs, experts, out, position, offsets, workspace, None))


def test_order_workspace():
    size = ar.lib().ar_expert_order_workspace
    assert size(0, 8) == size(32768, 1024) == 0 and size(32769, 8) == 9 * 8 * 4
    assert size(2 ** 31 - 1, 1024) == 64 * 1024 * 4
    assert size(100, 0) == size(100, 1025) == size(2 ** 31, 8) == 0


@pytest.mark.parametrize("change,want", [
    ({}, HIP), ({"pairs": 0, "indices": None, "out": None, "position": None}, HIP), ({"experts": 0}, INVALID),
    ({"experts": 1025}, UNSUPPORTED), ({"pairs": 2 ** 31}, UNSUPPORTED), ({"offsets": None}, INVALID),
    ({"indices": None}, INVALID), ({"out": None}, INVALID), ({"position": None}, INVALID),
    ({"indices": at(0) + 2}, INVALID), ({"offsets": at(3) + 1}, INVALID), ({"pairs": 50000}, INVALID),
    ({"pairs": 50000, "workspace": at(4)}, HIP), ({"pairs": 50000, "workspace": at(4) + 8}, INVALID),
])
def test_order_arguments(change, want):
    assert order(**change) == want


def matmul(change, weight=at(3), strides=(64 * 96, 96, 1), y=at(4)):
    return launched(lambda: ar.lib().ar_expert_matmul(ctypes.byref(rows(**change)), weight, *strides, y, None))


@pytest.mark.parametrize("change,more,want", [
    ({}, {}, HIP), ({"order": None, "x_rows": 200}, {}, HIP), ({"order": None}, {}, INVALID),
    ({}, {"strides": (64 * 96, 1, 64)}, HIP), ({}, {"strides": (64 * 96, 1, 63)}, INVALID),
    ({}, {"strides": (64 * 96, 95, 1)}, INVALID), ({}, {"strides": (64 * 96, 2, 3)}, INVALID),
    ({}, {"strides": (0, 96, 1)}, HIP), ({"inputs": 1, "x_stride": 1}, {"strides": (96, 5, 1)}, HIP),
    ({"inputs": 1}, {"strides": (96, 1, 1)}, HIP), ({"outputs": 1}, {"strides": (64, 1, 9)}, HIP),
    ({"dtype": F32}, {}, UNSUPPORTED), ({"experts": 0}, {}, INVALID), ({"experts": 1025}, {}, UNSUPPORTED),
    ({"pairs": 2 ** 31}, {}, UNSUPPORTED), ({"inputs": 0}, {}, INVALID), ({"outputs": 0}, {}, INVALID),
    ({"top_k": 0}, {}, INVALID), ({"offsets": None}, {}, INVALID), ({"x": None}, {}, INVALID),
    ({"x": at(0) + 1}, {}, INVALID), ({"x_stride": 63}, {}, INVALID), ({"x_rows": 1, "x_stride": 0}, {}, HIP),
    ({"x_stride": 2 ** 60}, {}, INVALID), ({}, {"weight": None}, INVALID), ({}, {"weight": at(3) + 1}, INVALID),
    # the last of 8 experts 7 * 2^61 bytes away, inside the address space, and 7 * 2^63
    ({}, {"strides": (2 ** 60, 96, 1)}, HIP), ({}, {"strides": (2 ** 62, 96, 1)}, INVALID), ({}, {"y": None}, INVALID), ({}, {"y": at(4) + 1}, INVALID),
    ({"pairs": 0}, {"y": None}, OK),
    ({"pairs": 2 ** 31 - 1, "outputs": 2 ** 20}, {"strides": (2 ** 26, 2 ** 20, 1)}, UNSUPPORTED),   # tiles
])
def test_matmul_arguments(change, more, want):
    assert matmul(change, **more) == want


@pytest.mark.parametrize("change,dy,stride,dw,dtype,want", [
    ({}, at(3), 96, at(4), F32, HIP), ({}, at(3), 96, at(4), BF16, HIP), ({}, at(3), 96, at(4), INT32, UNSUPPORTED),
    ({}, None, 96, at(4), F32, INVALID), ({}, at(3), 95, at(4), F32, INVALID), ({}, at(3), 96, None, F32, INVALID),
    ({}, at(3), 96, at(4) + 2, F32, INVALID), ({}, at(3), 96, at(4) + 2, BF16, HIP),
    ({"pairs": 0}, None, 0, at(4), F32, HIP), ({}, at(3), 96, at(0) + 64, F32, INVALID),
    ({}, at(3), 96, at(3) + 64, F32, INVALID), ({}, at(3), 96, at(2), F32, INVALID), ({}, at(3), 96, at(1), F32, INVALID),
    ({"inputs": 2 ** 20, "outputs": 2 ** 20, "x_stride": 2 ** 20}, at(3), 2 ** 20, at(9), F32, UNSUPPORTED),
    ({"inputs": 2 ** 31 - 1, "outputs": 2 ** 31 - 1, "x_stride": 2 ** 31}, at(3), 2 ** 31, at(9), F32, INVALID),
])
def test_weight_grad_arguments(change, dy, stride, dw, dtype, want):
    assert launched(lambda: ar.lib().ar_expert_weight_grad(ctypes.byref(rows(**change)), dy, stride, dw, dtype,
                                                           None, None)) == want


def test_weight_grad_workspace():
    """Only few tiles with many rows share them, and then need memory."""
    size = ar.lib().ar_expert_weight_grad_workspace
    assert size(200, 8, 64, 96) == size(0, 1, 64, 96) == size(2 ** 20, 128, 2048, 1024) == 0
    assert size(2 ** 20, 1, 64, 96) == 16 * 4 * 64 * 96 and size(1024, 1, 64, 96) == 4 * 4 * 64 * 96 and size(1024, 2, 64, 96) == 0
    assert size(2 ** 31 - 1, 1, 2 ** 31 - 1, 2 ** 31 - 1) == size(100, 0, 64, 96) == size(100, 8, 0, 96) == 0
    for workspace, want in ((None, INVALID), (at(5) + 8, INVALID), (at(5), HIP)):
        assert launched(lambda: ar.lib().ar_expert_weight_grad(
            ctypes.byref(rows(pairs=1024, experts=1, x_rows=512)), at(3), 96, at(4), F32, workspace, None)) == want


def combine(**change):
    a = dict(y=at(0), stride=96, pairs=200, size=96, dtype=BF16, position=at(1), weights=at(2), tokens=100, top_k=2,
             out=at(3))
    a.update(change)
    return launched(lambda: ar.lib().ar_expert_combine(*a.values(), None))


@pytest.mark.parametrize("change,want", [
    ({}, HIP), ({"weights": None}, HIP), ({"tokens": 0, "out": None}, OK), ({"pairs": 0, "y": None}, HIP),
    ({"size": 0}, INVALID), ({"top_k": 0}, INVALID), ({"dtype": F32}, UNSUPPORTED), ({"pairs": 2 ** 31}, UNSUPPORTED),
    ({"tokens": 2 ** 30, "top_k": 3}, UNSUPPORTED), ({"position": None}, INVALID), ({"y": None}, INVALID),
    ({"stride": 95}, INVALID), ({"y": at(0) + 1}, INVALID), ({"out": None}, INVALID), ({"weights": at(2) + 2}, INVALID),
    ({"size": 2 ** 28, "stride": 2 ** 28}, UNSUPPORTED),
])
def test_combine_arguments(change, want):
    assert combine(**change) == want


def combine_grad(**change):
    a = dict(dout=at(0), dout_stride=96, y=at(1), stride=96, pairs=200, size=96, dtype=BF16, position=at(2),
             offsets=at(3), experts=8, weights=at(4), tokens=100, top_k=2, dy=at(5), dweights=at(6))
    a.update(change)
    return launched(lambda: ar.lib().ar_expert_combine_grad(*a.values(), None))


@pytest.mark.parametrize("change,want", [
    ({}, HIP), ({"tokens": 0, "pairs": 0}, OK), ({"tokens": 0, "dout": None}, HIP), ({"offsets": None}, INVALID),
    ({"experts": 0}, INVALID), ({"experts": 1025}, UNSUPPORTED), ({"weights": None}, INVALID), ({"dout": None}, INVALID),
    ({"dweights": None}, INVALID), ({"dy": None}, INVALID), ({"dout_stride": 95}, INVALID), ({"dtype": F32}, UNSUPPORTED),
    ({"dy": at(5) + 1}, INVALID), ({"dweights": at(6) + 2}, INVALID),
])
def test_combine_grad_arguments(change, want):
    assert combine_grad(**change) == want


# --- Muon ------------------------------------------------------------------------------

def tensors(shapes, copy=False):
    return [MuonTensor(at(8 * i), at(8 * i + 1), at(8 * i + 2) if copy else None, at(8 * i + 3), *s)
            for i, s in enumerate(shapes)]


def plan(ts, pd=F32, gd=F32):
    """(status, host image or None) of a plan."""
    table = (MuonTensor * max(1, len(ts)))(*ts)
    lib = ar.lib()
    size = lib.ar_muon_plan_bytes(table, len(ts), pd, gd)
    image = (ctypes.c_char * max(size, 16))()
    status = lib.ar_muon_plan(table, len(ts), pd, gd, image, size)
    assert (size > 0) == (status == OK)
    return status, image if status == OK else None


def head(image):
    """The image's head: twelve 32-bit words, then 64-bit sizes and offsets."""
    small = (ctypes.c_uint32 * 11).from_buffer(image)
    large = (ctypes.c_uint64 * 9).from_buffer(image, 48)
    return dict(zip(("matrices", "chunks", "squares", "polys", "tiles", "side", "square_side"), small[1:])), \
        dict(zip(("bytes", "workspace", "matrices_at", "chunks_at", "squares_at", "polys_at", "tiles_at"), large))


@pytest.mark.parametrize("shapes", [[(1, 1, 1)], [(3, 61, 100)], [(2, 0, 5), (1, 100, 61), (0, 4, 4)],
                                    [(40, 300, 500)], [(1, 8192, 4096), (2, 129, 127)], [(1, 1, 4_000_000)], [(6, 1024, 1024), (3, 64, 512)]])
def test_plan_covers_every_matrix_once(shapes):
    status, image = plan(tensors(shapes))
    assert status == OK
    small, large = head(image)
    live = [(r, c) for n, r, c in shapes for _ in range(n if r and c else 0)]
    side, square = small["side"], small["square_side"]
    assert side in (64, 128) and side % square == 0 and square in (64, 128) and small["matrices"] == len(live)
    read = lambda where, n: (ctypes.c_uint32 * (2 * n)).from_buffer(image, large[where])  # noqa: E731
    chunks = read("chunks_at", small["chunks"])
    assert [(chunks[2 * i], chunks[2 * i + 1]) for i in range(small["chunks"])] == \
        [(i, j) for i, (r, c) in enumerate(live) for j in range(-(-r * c // 8192))]

    def unpack(where, n, steps):
        """The tiles of a table, each once; its parts cover its steps."""
        words = (ctypes.c_uint32 * (8 * n)).from_buffer(image, large[where])
        parts = {}
        for i in range(n):
            matrix, at, first, count, part, of, slot, counter = words[8 * i:8 * i + 8]
            if matrix != 2 ** 32 - 1:
                parts.setdefault((matrix, at & 0xFFFF, at >> 16), []).append((part, of, first, count, slot, counter))
        for (matrix, _, _), p in parts.items():
            p.sort()
            assert [q[0] for q in p] == list(range(p[0][1])) and all(q[1] == len(p) <= 8 for q in p)
            assert [q[2] for q in p] == [sum(r[3] for r in p[:i]) for i in range(len(p))]
            assert sum(q[3] for q in p) == steps(matrix) and len({q[4:] for q in p}) == 1 and min(q[3] for q in p) > 0
        split = [p[0] for p in parts.values() if len(p) > 1]
        assert len({q[5] for q in split}) == len(split)               # a counter each, and sums apart
        taken = [s for q in split for s in range(q[4], q[4] + q[1])]
        assert len(set(taken)) == len(taken)
        return list(parts)

    size = [tuple(-(-s // side) for s in (min(m), max(m))) for m in live]
    short = lambda i: size[i][0] * side // 32  # noqa: E731
    assert sorted(unpack("tiles_at", small["tiles"], short)) == \
        [(i, a, b) for i, (h, w) in enumerate(size) for a in range(h) for b in range(w)]
    assert sorted(unpack("squares_at", small["squares"], lambda i: size[i][1] * side // 32)) == \
        sorted(unpack("polys_at", small["polys"], short)) == \
        [(i, a, b) for i, (h, _) in enumerate(size) for a in range(h * side // square) for b in range(a, h * side // square)]
    # no XCD (entries 8 apart) has much more to do than another
    if len(live) > 1:
        for where, n in (("tiles_at", small["tiles"]), ("squares_at", small["squares"]), ("polys_at", small["polys"])):
            words = list((ctypes.c_uint32 * (8 * n)).from_buffer(image, large[where]))
            of = [sum(w != 2 ** 32 - 1 for w in words[8 * x::64]) for x in range(8)]
            assert max(of) * 8 == n and (len(set(size)) > 1 or min(of) >= max(of) - 32)
    assert large["workspace"] >= sum(8 * h * w * side ** 2 + 8 * h * h * side ** 2 for h, w in size)
    assert ar.lib().ar_muon_workspace(image) == large["workspace"]


def changed(ts, i, **fields):
    for k, v in fields.items():
        setattr(ts[i], k, v)
    return ts


ONE = [(1, 8, 8)]


@pytest.mark.parametrize("ts,kind,want", [
    ([], {}, INVALID), (tensors(ONE), {"pd": INT32}, UNSUPPORTED), (tensors(ONE), {"gd": INT32}, UNSUPPORTED),
    (changed(tensors(ONE * 2), 1, param=None), {}, INVALID), (changed(tensors(ONE), 0, grad=None), {}, INVALID),
    (changed(tensors(ONE), 0, momentum=None), {}, INVALID), (changed(tensors(ONE), 0, param=A + 2), {}, INVALID),
    (changed(tensors(ONE), 0, momentum=at(3) + 2), {}, INVALID), (changed(tensors(ONE), 0, grad=at(1) + 1), {"gd": BF16}, INVALID),
    (tensors(ONE, copy=True), {"pd": BF16}, INVALID), (changed(tensors(ONE * 2, copy=True), 1, copy=None), {}, INVALID),
    (changed(tensors(ONE), 0, momentum=A), {}, INVALID), (changed(tensors(ONE * 2), 1, param=A + 252), {}, INVALID),
    (changed(tensors(ONE), 0, grad=A), {}, INVALID), (changed(tensors(ONE, copy=True), 0, copy=at(3) + 8), {}, INVALID),
    (tensors([(1, 2 ** 31, 2 ** 31)]), {}, UNSUPPORTED), (tensors([(1, 32768, 32769)]), {}, UNSUPPORTED),
    (tensors([(1, 1, 4_194_241)]), {}, UNSUPPORTED), (tensors([(2 ** 62, 8, 8)]), {}, INVALID),
    (tensors([(2 ** 30, 8, 8)]), {}, INVALID),       # 2^38 bytes, over the next tensor at 2^36
    (tensors([(2 ** 22, 8, 8)]), {}, UNSUPPORTED),   # one tile more than there may be
])
def test_plan_refusals(ts, kind, want):
    assert plan(ts, **kind)[0] == want


def test_plan_takes_neighbours_and_shared_gradients():
    assert plan(changed(tensors(ONE * 2), 1, param=A + 256, grad=at(1)))[0] == OK
    assert plan(tensors(ONE, copy=True))[0] == OK
    assert plan(tensors([(1, 32768, 32768)]))[0] == OK


def step(image, **change):
    a = dict(lr=0.02, momentum=0.95, eps=1e-7, weight_decay=0.0, grad_scale=1.0, match_rms=0.0, nesterov=1, ns_steps=5)
    device, workspace = change.pop("device", at(100)), change.pop("workspace", at(101))
    a.update(change)
    return launched(lambda: ar.lib().ar_muon_step(image, device, workspace, ctypes.byref(MuonStep(**a)), None))


def test_step_arguments():
    image = plan(tensors(ONE))[1]
    assert step(image) == HIP
    for change in ({"lr": -1.0}, {"lr": float("nan")}, {"momentum": 1.0}, {"momentum": -0.1}, {"eps": -1e-9},
                   {"weight_decay": -1.0}, {"grad_scale": float("inf")}, {"match_rms": -0.1}, {"ns_steps": 0},
                   {"ns_steps": 33}, {"device": None}, {"device": at(100) + 16}, {"workspace": None},
                   {"workspace": at(101) + 16}):
        assert step(image, **change) == INVALID, change
    blank = (ctypes.c_char * 4096)()
    assert step(blank) == INVALID and ar.lib().ar_muon_workspace(blank) == 0
    assert step(plan(tensors([(0, 8, 8)]))[1], workspace=None) == OK      # nothing to do
