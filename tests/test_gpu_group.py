"""Grouping of choices by expert on the GPU, exactly, against a stable sort on the host; and a
router, its grouping, the experts' products and their gradients run together."""
import numpy as np
import pytest
import torch

import rows_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, matrix, same, values

pytestmark = pytest.mark.gpu


def draw(n, experts, how, seed):
    g = np.random.default_rng(seed)
    if how == "even":
        ids = g.integers(0, experts, n)
    elif how == "crowded":
        ids = np.minimum(g.zipf(1.3, n) - 1, experts - 1)
    elif how == "one":
        ids = np.full(n, experts - 1)
    elif how == "none":
        ids = np.full(n, 0xFFFFFFFF)
    elif how == "sorted":
        ids = np.sort(g.integers(0, experts, n))[::-1]
    else:   # a third of them no expert, some only in bits above the tenth
        ids = g.integers(0, experts, n)
        ids = np.where(g.random(n) < 0.2, ids + 1024 * g.integers(1, 1 << 20, n), ids)
        ids = np.where(g.random(n) < 0.2, 0xFFFFFFFF, ids)
        ids = np.where(g.random(n) < 0.1, experts, ids)
    return ids.astype(np.uint32)


def check(ids, experts, align):
    t = torch.from_numpy(ids.view(np.int32)).to(DEV)
    n = ids.size
    room = n + experts * (align - 1)
    out = [torch.full((max(m, 1),), 0x5A5A5A5A, dtype=torch.int32, device=DEV) for m in (room, n, experts + 1, experts)]
    need = rs.rs_group_choices(None, n, experts, align, None, None, None, None, None, 0)
    temp = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    rs.rs_group_choices(t, n, experts, align, *out, temp, need)
    for got, want, what in zip(out, ref.group(ids, experts, align), ("order", "place", "starts", "counts")):
        same(got[: want.size], want, what)
    assert (temp[need:] == 0x5A).all(), "written behind the temp"
    assert np.array_equal(t.cpu().numpy().view(np.uint32), ids), "ids were written"


SIZES = [0, 1, 2, 63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 8191, 8193, 16383, 16384, 16385,
         32769, 100003]


@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("experts", [1, 2, 5, 64, 65, 128, 255, 256, 1000, 1024])
def test_sizes(n, experts):
    for align, how in ((1, "even"), (16, "crowded"), (100, "mixed")):
        print("group n %d experts %d align %d %s" % (n, experts, align, how), flush=True)
        check(draw(n, experts, how, n + experts), experts, align)


@pytest.mark.parametrize("how", ["one", "none", "sorted", "mixed", "crowded"])
@pytest.mark.parametrize("n", [1, 100, 5000, 20000, 131072, 1 << 20, 5_000_011])
def test_distributions(n, how):
    for experts, align in ((128, 128), (1024, 1), (7, 3)):
        print("group n %d experts %d align %d %s" % (n, experts, align, how), flush=True)
        check(draw(n, experts, how, n), experts, align)


def test_wide_padding():
    for n, experts, align in ((10, 3, 1 << 20), (5000, 2, 100001), (0, 1024, 500)):
        print("group n %d experts %d align %d" % (n, experts, align), flush=True)
        check(draw(n, experts, "even", 1), experts, align)


def test_many_choices():
    n, experts = (1 << 28) + 12345, 300
    print("group n = 2^28 + 12345", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    ids = torch.randint(-1, experts, (n,), generator=g, device=DEV, dtype=torch.int32)
    order, place, starts, counts = rs.group_choices(ids, experts, align=64)
    real = ids >= 0
    assert torch.equal(counts.long(), torch.stack([(ids == e).sum() for e in range(experts)]))
    ends = torch.cumsum((counts.long() + 63) // 64 * 64, 0)
    assert torch.equal(starts[1:].long(), ends) and int(starts[0]) == 0
    assert (place[~real] == -1).all()
    at = place[real].long()
    assert torch.equal(order[at].long(), torch.nonzero(real)[:, 0])
    filled = order >= 0
    assert int(filled.sum()) == int(real.sum())
    # in every segment the choices lead, in increasing order, and belong to its expert
    seg = torch.repeat_interleave(torch.arange(experts, device=DEV), (starts[1:] - starts[:-1]).long())
    pos = torch.nonzero(filled)[:, 0]
    assert torch.equal(ids[order[pos].long()].long(), seg[pos])
    assert (pos - starts[seg[pos]] < counts[seg[pos]]).all()
    step = order[pos][1:] > order[pos][:-1]
    assert (step | (seg[pos][1:] != seg[pos][:-1])).all()


def test_streams_and_graphs_with_their_own_temps():
    print("group on two streams, and in two graphs", flush=True)
    a, b = draw(50000, 256, "even", 1), draw(3000, 64, "crowded", 2)
    ta, tb = (torch.from_numpy(i.view(np.int32)).to(DEV) for i in (a, b))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [(rs.group_choices(ta, 256, 16, stream=s[0]), rs.group_choices(tb, 64, 8, stream=s[1])) for _ in range(3)]
    torch.cuda.synchronize()
    for oa, ob in outs:
        for got, want in list(zip(oa, ref.group(a, 256, 16))) + list(zip(ob, ref.group(b, 64, 8))):
            same(got, want, "two streams")
    graphs, held = [], []
    for t, e in ((ta, 256), (tb, 64)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(rs.group_choices(t, e, 4))
        graphs.append(graph)
    for i in range(3):
        ta.copy_(torch.roll(torch.from_numpy(a.view(np.int32)).to(DEV), i * 100))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(held[0], ref.group(np.roll(a, i * 100), 256, 4)):
            same(got, want, "replay %d" % i)
        for got, want in zip(held[1], ref.group(b, 64, 4)):
            same(got, want, "replay %d" % i)
        eager = rs.group_choices(ta, 256, 4)
        assert all(torch.equal(x, y) for x, y in zip(eager, held[0]))


def test_wrapper_shapes_and_refusals():
    ids = torch.zeros(6, 4, dtype=torch.int32, device=DEV)
    order, place, starts, counts = rs.group_choices(ids, 3, align=5)
    assert place.shape == (6, 4) and order.shape == (24 + 12,) and starts.tolist() == [0, 25, 25, 25]
    with pytest.raises(TypeError):
        rs.group_choices(ids.long(), 3)
    with pytest.raises(TypeError):
        rs.group_choices(ids.t(), 3)
    with pytest.raises(rs.RsError):
        rs.group_choices(ids, 0)
    assert rs.group_choices(ids[:0], 3)[3].tolist() == [0, 0, 0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_mixture_layer_together(score):
    """Scores -> choices -> segments -> each expert's product over its segment -> weighted sum, and
    the gradient of the scores back through it, against every token's experts one by one in f64.

    Integers as inputs and experts keep the products exact; the weights are f32, off by U, and the
    sum of k products of size up to 60 * w by k U more; the gradient by its own bound."""
    print("mixture layer", score, flush=True)
    g = np.random.default_rng(11)
    rows, width, experts, k, align = 333, 16, 24, 3, 16
    x = g.integers(-2, 3, (rows, width)).astype(np.float64)
    wts = g.integers(-1, 2, (experts, width, width)).astype(np.float64)
    scores = matrix(g.standard_normal((rows, experts)), "f32")
    up = g.integers(-2, 3, (rows, width)).astype(np.float64)
    ids, w = rs.route_topk(scores, k, score=score)
    order, place, starts, counts = rs.group_choices(ids, experts, align=align)
    tx, tw, tup = (torch.from_numpy(v).float().to(DEV) for v in (x, wts, up))
    tiles = order.view(-1, align) if order.numel() % align == 0 else order[: order.numel() // align * align].view(-1, align)
    of_tile = torch.searchsorted(starts.long(), torch.arange(tiles.shape[0], device=DEV) * align, right=True) - 1
    held = of_tile < experts
    token = (tiles.long() // k).clamp(min=0)
    y = torch.bmm(tx[token] * (tiles >= 0)[..., None], tw[of_tile.clamp(max=experts - 1)].contiguous())
    y = (y * held[:, None, None]).view(-1, width)
    each = y[place.long().view(-1)].view(rows, k, width)
    out = (each * w[..., None]).sum(1)
    dw = (each * tup[:, None]).sum(2)
    ds = rs.route_topk_grad(scores, ids, w, dw.contiguous(), score=score)
    rids, rw, _ = ref.route(values(scores), k, score=score)
    same(ids, rids, "ids")
    reach = np.einsum("rw,rkwv->rkv", x, wts[rids])
    want = (reach * rw[..., None]).sum(1)
    size = (np.abs(reach) * rw[..., None]).sum(1)
    assert (np.abs(values(out) - want) <= (k + 3) * ref.U * size).all()
    rdw = (reach * up[:, None]).sum(2)
    assert np.array_equal(values(dw), rdw)
    rds, bound = ref.route_grad(values(scores), rids, rdw, score=score)
    assert (np.abs(values(ds) - rds) <= bound + ref.U * np.abs(rds)).all()
