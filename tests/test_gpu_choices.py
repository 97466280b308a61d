"""Gathering rows into the order of a grouping and combining them back, with their gradients, against
the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import moves_reference as ref
import rows_reference
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, DTYPES, close, matrix, same, values

pytestmark = pytest.mark.gpu

# rows, top_k, experts, align, width, elements between rows, elements before the first
SHAPES = [
    (1, 1, 1, 1, 1, 0, 0), (1, 8, 128, 16, 64, 0, 0), (3, 2, 5, 4, 7, 3, 1), (17, 3, 9, 1, 33, 0, 0),
    (64, 5, 16, 8, 128, 8, 0), (5, 8, 64, 16, 512, 0, 0), (33, 4, 7, 16, 513, 1, 3), (9, 6, 20, 1, 1000, 0, 2),
    (40, 12, 30, 8, 257, 0, 0), (6, 64, 64, 2, 96, 5, 0), (11, 9, 300, 1, 2048, 0, 0), (3, 7, 8, 4, 4099, 0, 0),
    (700, 2, 3, 100, 16, 0, 0), (2, 3, 4, 128, 5120, 0, 8),
]


def choices(rng, rows, k, experts, dropped=0.2):
    """Distinct experts of each row where there are enough, some rows without any, some choices without one."""
    ids = np.empty((rows, k), np.int32)
    for t in range(rows):
        ids[t] = rng.permutation(experts)[:k] if k <= experts else rng.integers(0, experts, k)
    ids[rng.random(rows) < dropped] = -1
    ids[rng.random((rows, k)) < dropped / 4] = -1
    return ids


def grouped(ids, experts, align):
    """group_choices' order and place, which its own tests check."""
    order, place, _, _ = rs.group_choices(torch.from_numpy(ids).to(DEV), experts, align=align)
    return order, place


def weights_of(rng, rows, k):
    return rng.standard_normal((rows, k)).astype(np.float32)


def on(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def room_of(shape):
    rows, k, experts, align = shape[:4]
    return rows * k + experts * (align - 1)


def guarded(rows, cols, dtype, pad):
    """A matrix to be written, and a check that what lies between its rows was not."""
    whole = torch.full((rows, cols + pad), 7.0, dtype=DTYPES[dtype], device=DEV)

    def untouched():
        assert (whole[:, cols:] == 7.0).all(), "written between the rows"
    return whole[:, :cols], untouched


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_gather(shape, weighted, dtype):
    print("gather", shape, weighted, dtype, flush=True)
    rows, k, experts, align, width, pad, shift = shape
    rng = np.random.default_rng(rows * 1000 + width)
    order, place = grouped(choices(rng, rows, k, experts), experts, align)
    x = matrix(rng.standard_normal((rows, width)), dtype, pad, shift)
    w = weights_of(rng, rows, k) if weighted else None
    want, bound = ref.gather(values(x), order.cpu().numpy(), k, w)
    got = rs.gather_choices(x, order, place, weights=None if w is None else on(w))
    assert got.dtype == x.dtype and got.is_contiguous()
    close(got, want, bound, "y", dtype)
    out, untouched = guarded(room_of(shape), width, dtype, pad)
    assert rs.gather_choices(x, order, place, weights=None if w is None else on(w), out=out) is out
    assert torch.equal(out, got)
    untouched()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_combine(shape, weighted, dtype):
    """Rows of the padding hold NaN: they are not read."""
    print("combine", shape, weighted, dtype, flush=True)
    rows, k, experts, align, width, pad, shift = shape
    rng = np.random.default_rng(rows * 1000 + width + 1)
    order, place = grouped(choices(rng, rows, k, experts), experts, align)
    y = rng.standard_normal((room_of(shape), width))
    y[order.cpu().numpy() < 0] = np.nan
    y = matrix(y, dtype, pad, shift)
    w = weights_of(rng, rows, k) if weighted else None
    want, bound = ref.combine(values(y), place.cpu().numpy(), w)
    got = rs.combine_choices(y, place, weights=None if w is None else on(w))
    assert got.dtype == y.dtype and got.shape == (rows, width)
    close(got, want, bound, "out", dtype)
    out, untouched = guarded(rows, width, dtype, pad)
    assert rs.combine_choices(y, place, weights=None if w is None else on(w), out=out) is out
    assert torch.equal(out, got)
    untouched()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(shape, dtype):
    print("gradients", shape, dtype, flush=True)
    rows, k, experts, align, width, pad, shift = shape
    rng = np.random.default_rng(rows * 1000 + width + 2)
    order, place = grouped(choices(rng, rows, k, experts), experts, align)
    o, p = order.cpu().numpy(), place.cpu().numpy()
    x = matrix(rng.standard_normal((rows, width)), dtype, pad, shift)
    y = rng.standard_normal((room_of(shape), width))
    y[o < 0] = np.nan
    y = matrix(y, dtype, shift, pad)
    w = weights_of(rng, rows, k)
    want, bound = ref.combine(values(y), p, w)
    dwant, dbound = ref.dots(values(x), values(y), p)
    dx, dw = rs.gather_choices_grad(y, x, place, on(w))
    close(dx, want, bound, "gather dx", dtype)
    close(dw, dwant, dbound, "gather dw")
    want, bound = ref.gather(values(x), o, k, w)
    dy, dw = rs.combine_choices_grad(x, y, order, place, on(w))
    close(dy, want, bound, "combine dy", dtype)
    close(dw, dwant, dbound, "combine dw")
    out, untouched = guarded(rows, width, dtype, pad)
    to, dw2 = rs.gather_choices_grad(y, x, place, on(w), out=out)
    assert to is out and torch.equal(out, dx) and torch.equal(dw2, dw)
    untouched()
    out, untouched = guarded(room_of(shape), width, dtype, pad)
    to, dw2 = rs.combine_choices_grad(x, y, order, place, on(w), out=out)
    assert to is out and torch.equal(out, dy) and torch.equal(dw2, dw)
    untouched()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("width", [1003, 530])
def test_many_rows(width, dtype):
    """So many that a wave takes several vectors of a row, with ends off their borders."""
    print("many rows", width, dtype, flush=True)
    rng = np.random.default_rng(width)
    rows, k = 4200, 2
    order, place = grouped(choices(rng, rows, k, 16), 16, 8)
    o, p = order.cpu().numpy(), place.cpu().numpy()
    x = matrix(rng.standard_normal((rows, width)), dtype, 1)
    y = matrix(rng.standard_normal((len(o), width)), dtype)
    w = weights_of(rng, rows, k)
    for weights in (None, w):
        given = None if weights is None else on(weights)
        close(rs.gather_choices(x, order, place, weights=given), *ref.gather(values(x), o, k, weights), "y", dtype)
        close(rs.combine_choices(y, place, weights=given), *ref.combine(values(y), p, weights), "out", dtype)
    dy, dw = rs.combine_choices_grad(x, y, order, place, on(w))
    close(dy, *ref.gather(values(x), o, k, w), "dy", dtype)
    close(dw, *ref.dots(values(x), values(y), p), "dw")


@pytest.mark.parametrize("width", [5, 300, 2100])
@pytest.mark.parametrize("k", [1, 3, 8, 20])
def test_any_order_and_place(width, k):
    """What is written by position goes by order alone, what is summed by place alone: places and
    choices that occur twice, that name nothing and that do not belong together."""
    print("any order and place", width, k, flush=True)
    rng = np.random.default_rng(width + k)
    rows, room = 23, 150
    o = rng.integers(-3, rows * k + 3, room).astype(np.int32)
    p = rng.integers(-3, room + 3, (rows, k)).astype(np.int32)
    belong = rng.random(room) < 0.5   # half of them do
    for i in np.nonzero(belong)[0]:
        if 0 <= o[i] < rows * k:
            p.reshape(-1)[o[i]] = i
    p[0] = 5
    p[1] = -1
    p[2] = 0x7FFFFFFF
    o[7:9] = 3
    o[9] = 0x7FFFFFFF
    order, place = on(o), on(p)
    x = matrix(rng.standard_normal((rows, width)), "bf16")
    y = matrix(rng.standard_normal((room, width)), "bf16")
    w = weights_of(rng, rows, k)
    for weights in (None, w):
        given = None if weights is None else on(weights)
        close(rs.gather_choices(x, order, place, weights=given), *ref.gather(values(x), o, k, weights), "y", "bf16")
        close(rs.combine_choices(y, place, weights=given), *ref.combine(values(y), p, weights), "out", "bf16")
    dx, dw = rs.gather_choices_grad(y, x, place, on(w))
    close(dx, *ref.combine(values(y), p, w), "dx", "bf16")
    close(dw, *ref.dots(values(x), values(y), p), "dw")
    dy, dw = rs.combine_choices_grad(x, y, order, place, on(w))
    close(dy, *ref.gather(values(x), o, k, w), "dy", "bf16")
    close(dw, *ref.dots(values(x), values(y), p), "dw")


def test_special_values():
    """A copy keeps every bit; weights of 0 and infinity, and NaN, go through as in the formulas; only
    a row's own choices reach it."""
    print("special values", flush=True)
    rng = np.random.default_rng(3)
    ids = np.array([[0, 1], [1, 2], [2, 0], [-1, 1]], np.int32)
    order, place = grouped(ids, 3, 4)
    bits = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, (4, 70)).astype(np.int16)).to(DEV)
    for dtype in ("f16", "bf16"):
        y = rs.gather_choices(bits.view(DTYPES[dtype]), order, place).view(torch.int16)
        o = order.long()
        assert torch.equal(y[o >= 0], bits[o[o >= 0] // 2])
    x = np.ones((4, 70))
    x[0], x[1, ::2], x[2, 3] = np.inf, np.nan, -np.inf
    w = np.array([[1, 0], [2, -1], [np.inf, 0.5], [3, 0.25]], np.float32)
    with np.errstate(all="ignore"):
        xt = matrix(x, "f32")
        want = ref.gather(x, order.cpu().numpy(), 2, w)[0]
        close(rs.gather_choices(xt, order, place, weights=on(w)), want, 1e-6, "y")
        y = np.ones((len(order), 70))
        y[int(place[0, 0])] = np.nan
        y[int(place[3, 1])] = np.inf
        want = ref.combine(y, place.cpu().numpy(), w)[0]
        got = rs.combine_choices(matrix(y, "f32"), place, weights=on(w))
    close(got, want, 1e-6, "out")


def test_order_that_ends_early():
    """The positions of the segments alone, without the room behind the last of them."""
    print("short order", flush=True)
    rng = np.random.default_rng(8)
    ids = choices(rng, 50, 4, 12, dropped=0.3)
    order, place, starts, _ = rs.group_choices(on(ids), 12, align=16)
    n = int(starts[-1])
    x = matrix(rng.standard_normal((50, 200)), "f16")
    whole = rs.gather_choices(x, order, place)
    assert torch.equal(rs.gather_choices(x, order[:n], place), whole[:n])
    half = n // 2   # choices behind it count as without place
    assert torch.equal(rs.gather_choices(x, order[:half], place), whole[:half])
    want = ref.combine(values(whole[:half]), place.cpu().numpy())
    close(rs.combine_choices(whole[:half], place), *want, "half", "f16")


def test_nothing():
    print("nothing", flush=True)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    x = torch.ones(0, 40, device=DEV)
    y = rs.gather_choices(x, torch.full((9,), -1, dtype=torch.int32, device=DEV), none.view(0, 3))
    assert y.shape == (9, 40) and (y == 0).all()
    x = torch.ones(5, 40, device=DEV)
    place = torch.full((5, 3), -1, dtype=torch.int32, device=DEV)
    assert rs.gather_choices(x, none, place).shape == (0, 40)
    w = torch.ones(5, 3, device=DEV)
    out, dw = rs.gather_choices_grad(x[:0], x, place, w)
    assert (out == 0).all() and (dw == 0).all()
    assert (rs.combine_choices(x[:0], place) == 0).all()
    dy, dw = rs.combine_choices_grad(x, x[:0], none, place, w)
    assert dy.shape == (0, 40) and (dw == 0).all()


def test_strides():
    """One row for all (stride 0), rows in reverse distance, overlapping rows."""
    print("strides", flush=True)
    rng = np.random.default_rng(5)
    ids = choices(rng, 30, 3, 10)
    order, place = grouped(ids, 10, 8)
    o, p = order.cpu().numpy(), place.cpu().numpy()
    w = weights_of(rng, 30, 3)
    base = matrix(rng.standard_normal((1, 900)), "bf16")
    for x, y in ((base[:, :500].expand(30, 500), base[:, 100:600].expand(len(o), 500)),
                 (torch.as_strided(base, (30, 500), (3, 1)), torch.as_strided(base, (len(o), 500), (1, 1)))):
        close(rs.gather_choices(x, order, place, weights=on(w)), *ref.gather(values(x), o, 3, w), "y", "bf16")
        dx, dw = rs.gather_choices_grad(y, x, place, on(w))
        close(dx, *ref.combine(values(y), p, w), "dx", "bf16")
        close(dw, *ref.dots(values(x), values(y), p), "dw")
        dy, dw = rs.combine_choices_grad(x, y, order, place, on(w))
        close(dy, *ref.gather(values(x), o, 3, w), "dy", "bf16")
        close(dw, *ref.dots(values(x), values(y), p), "dw")


def test_equal_calls_give_equal_bits():
    print("equal bits", flush=True)
    rng = np.random.default_rng(6)
    order, place = grouped(choices(rng, 300, 8, 32), 32, 16)
    x = matrix(rng.standard_normal((300, 700)), "bf16")
    y = matrix(rng.standard_normal((order.numel(), 700)), "bf16")
    w = on(weights_of(rng, 300, 8))
    first = None
    for _ in range(4):
        now = [rs.gather_choices(x, order, place, weights=w), rs.combine_choices(y, place, weights=w),
               *rs.gather_choices_grad(y, x, place, w), *rs.combine_choices_grad(x, y, order, place, w)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 bytes: rows at both ends."""
    print("large matrices", flush=True)
    rows, k, width = 1200, 2, 1 << 20
    rng = np.random.default_rng(7)
    order, place = grouped(choices(rng, rows, k, 4, dropped=0.01), 4, 1)
    x = torch.empty(rows, width, dtype=torch.bfloat16, device=DEV)   # 2.5 GB, the gathered rows 5 GB
    x.copy_(torch.arange(rows, device=DEV)[:, None] % 251)
    x[:, -1] = 3
    y = rs.gather_choices(x, order, place)
    real = order >= 0
    row = (order.clamp(min=0) // k) % 251
    want = torch.where(real, row, 0).to(torch.bfloat16)
    assert torch.equal(y[:, 0], want) and torch.equal(y[:, width // 2 + 1], want)
    assert torch.equal(y[:, -1], torch.where(real, 3, 0).to(torch.bfloat16))
    del x
    out = rs.combine_choices(y, place)
    n = (place >= 0).sum(1)
    t = torch.arange(rows, device=DEV) % 251
    assert torch.equal(out[:, 5], (n * t).to(torch.bfloat16))
    assert torch.equal(out[:, -1], (n * 3).to(torch.bfloat16))


def test_replays_of_a_graph():
    """A router's step in a graph: routed, grouped, gathered, combined, with gradients."""
    print("graph", flush=True)
    rng = np.random.default_rng(9)
    scores = on(rng.standard_normal((120, 16)).astype(np.float32))
    x = matrix(rng.standard_normal((120, 264)), "bf16")
    dout = matrix(rng.standard_normal((120, 264)), "bf16")

    def step():
        ids, w = rs.route_topk(scores, 4)
        order, place, _, _ = rs.group_choices(ids, 16, align=16)
        y = rs.gather_choices(x, order, place)
        out = rs.combine_choices(y, place, weights=w)
        dy, dw = rs.combine_choices_grad(dout, y, order, place, w)
        dx = rs.combine_choices(dy, place)
        return out, dx, rs.route_topk_grad(scores, ids, w, dw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        scores.copy_(torch.randn(120, 16, device=DEV))
        x.copy_(torch.randn(120, 264, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        for g, want in zip(got, step()):
            assert torch.equal(g, want)
        torch.cuda.synchronize()


def test_reference_of_the_grouping():
    """What these tests take from group_choices is what its reference gives."""
    ids = choices(np.random.default_rng(1), 60, 3, 9)
    order, place = grouped(ids, 9, 8)
    o, p, _, _ = rows_reference.group(ids.reshape(-1), 9, 8)
    same(order, o, "order")
    same(place.reshape(-1), p, "place")
