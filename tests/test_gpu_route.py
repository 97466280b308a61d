"""Routing and its gradient on the GPU against the definition in 64 bits: sizes, types, strides,
groups, ties, masks, rows of nothing, streams and graphs.

Weights are computed in 64 bits and rounded once, so they may be off by half a step of f32 (and
2^-40 for the 64-bit arithmetic); choices have no tolerance."""
import itertools

import numpy as np
import pytest
import torch

import rows_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, close, matrix, numpy_of, same, values

pytestmark = pytest.mark.gpu


def check(x, k, dtype="f32", pad=0, shift=0, grad=True, **kw):
    t = matrix(x, dtype, pad, shift)
    before = t.clone()
    x = values(t)
    bias = kw.pop("bias", None)
    tb = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(DEV)
    ids, w = rs.route_topk(t, k, bias=tb, **kw)
    rids, rw, _ = ref.route(x, k, bias=None if bias is None else bias.astype(np.float32), **kw)
    same(ids, rids, "ids")
    close(w, rw, np.where(np.isfinite(rw), np.abs(rw), 0) * 2.0 ** -40, "weights")
    assert torch.equal(t.view(torch.int16 if dtype != "f32" else torch.int32),
                       before.view(torch.int16 if dtype != "f32" else torch.int32)), "scores were written"
    if grad:
        gk = {n: kw[n] for n in ("score", "renormalize", "scale") if n in kw}
        dw = np.random.default_rng(k).standard_normal((x.shape[0], k)).astype(np.float32)
        out = matrix(np.zeros_like(x), dtype, pad, shift)
        got = rs.route_topk_grad(t, ids, w, torch.from_numpy(dw).to(DEV), out=out, **gk)
        assert got is out
        dx, bound = ref.route_grad(x, rids, dw.astype(np.float64), **gk)
        close(got, dx, bound, "dscores", dtype)
        around = got.as_strided((x.shape[0], x.shape[1] + pad), (x.shape[1] + pad, 1))[:, x.shape[1]:]
        assert torch.isnan(around).all(), "written between the rows"


EXPERTS = [1, 2, 3, 7, 15, 16, 17, 60, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 511, 512, 513,
           1000, 1023, 1024]


@pytest.mark.parametrize("experts", EXPERTS)
def test_every_size(experts):
    g = np.random.default_rng(experts)
    for i, (score, biased, renorm) in enumerate(itertools.product(("softmax", "sigmoid"), (0, 1), (0, 1))):
        dtype = ("f32", "f16", "bf16")[(i + experts) % 3]
        rows = (1, 3, 5, 66, 130, 2, 17, 33)[i]
        k = min(experts, (1, 8, 2, 64, 6, 10, 4, 5)[(i + experts) % 8])
        print("route experts %d rows %d k %d %s %s bias %d renorm %d" % (experts, rows, k, dtype, score, biased, renorm),
              flush=True)
        x = g.standard_normal((rows, experts)) * 2
        check(x, k, dtype, pad=(0, 3, 8)[i % 3], shift=(0, 1, 4)[i % 3], score=score, renormalize=bool(renorm),
              bias=g.standard_normal(experts) * 0.1 if biased else None, scale=(1.0, 2.5)[i % 2])


@pytest.mark.parametrize("experts,groups,top,best,k", [
    (256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (64, 64, 6, 1, 6), (64, 64, 64, 1, 64), (96, 3, 2, 2, 7), (96, 3, 1, 1, 32),
    (6, 2, 1, 2, 3), (1024, 32, 5, 2, 12), (1000, 10, 3, 2, 64), (160, 8, 3, 2, 6), (1008, 63, 7, 2, 9), (12, 1, 1, 2, 4),
    (24, 24, 3, 1, 3), (130, 13, 1, 2, 10), (257, 1, 1, 1, 9),
])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(experts, groups, top, best, k, score, biased):
    g = np.random.default_rng(experts + groups)
    for rows, dtype in ((1, "f32"), (70, "bf16"), (9, "f16")):
        print("route groups", experts, groups, top, best, k, score, biased, rows, dtype, flush=True)
        check(g.standard_normal((rows, experts)), k, dtype, score=score, groups=groups, top_groups=top,
              group_best=best, bias=g.standard_normal(experts) * 0.1 if biased else None)


@pytest.mark.parametrize("experts", [8, 64, 100, 256, 1000])
def test_ties_go_to_the_lowest_expert(experts):
    g = np.random.default_rng(5)
    x = g.integers(-2, 3, (40, experts)).astype(np.float64)
    x[0] = 0.0
    x[1] = np.where(np.arange(experts) % 2, 0.0, -0.0)
    for kw in (dict(), dict(score="sigmoid"), dict(bias=np.zeros(experts)),
               dict(score="sigmoid", bias=g.integers(0, 2, experts) * 0.25),
               dict(groups=4, top_groups=2, group_best=2), dict(groups=2, top_groups=1, score="sigmoid"),
               dict(groups=4, top_groups=3, group_best=2, bias=np.zeros(experts), score="sigmoid")):
        print("route ties", experts, sorted(kw), flush=True)
        check(x, min(8, experts // 2), **kw)
        check(x, min(64, experts // 2), "bf16", **kw)


def test_scores_next_to_each_other_are_told_apart():
    """Probabilities that f32 cannot tell apart, and that 64 bits can: saturated sigmoids, and a
    bias that leaves differences of 2^-30."""
    experts = 64
    x = np.tile(20.0 + np.arange(experts) % 13 * 0.25, (5, 1))
    x[1] = -x[1]
    x[2:] = np.random.default_rng(6).permuted(np.tile(16 + np.arange(experts) * 0.125, (3, 1)), axis=1)
    for kw in (dict(score="sigmoid", bias=np.zeros(experts)), dict(score="sigmoid", bias=np.full(experts, 0.5)),
               dict(bias=np.full(experts, 1.0)), dict(score="sigmoid", groups=8, top_groups=3, group_best=2)):
        print("route near ties", sorted(kw), flush=True)
        check(x, 12, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kw", [dict(), dict(renormalize=False), dict(groups=4, top_groups=2, group_best=2),
                                dict(groups=4, top_groups=2), dict(biased=True),
                                dict(biased=True, groups=4, top_groups=1, group_best=2, renormalize=False)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_experts(score, kw, dtype):
    kw = dict(kw)
    g = np.random.default_rng(8)
    x = g.standard_normal((64, 80))
    x[g.random(x.shape) < 0.7] = -np.inf
    x[0] = -np.inf                                  # nothing is left
    x[1, 1:] = -np.inf                              # one expert is left
    x[2] = np.finfo(np.float16).min if dtype == "f16" else -3.3e38   # the lowest values, no mask
    x[3, :40] = np.finfo(np.float16).min if dtype == "f16" else -3.3e38
    x[4, :20] = -np.inf                             # a whole group of four
    x[5] = -800.0                                   # probabilities below f32
    x[5, 3] = -801.0
    bias = g.standard_normal(80) * 3 if kw.pop("biased", False) else None
    if bias is not None:
        bias[7] = -np.inf                           # an expert that is switched off
    print("route masks", score, sorted(kw), dtype, flush=True)
    check(x, 9, dtype, score=score, bias=bias, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_nan_and_infinity(score, biased):
    g = np.random.default_rng(9)
    x = g.standard_normal((6, 72))
    x[0, 5] = np.nan
    x[1, 6] = np.inf
    x[2] = np.nan
    x[3, :70] = -np.inf
    x[3, 70] = np.nan
    x[4, 10:12] = np.inf
    bias = g.standard_normal(72) if biased else None
    if biased:
        bias[3] = np.nan
    for kw in (dict(), dict(groups=8, top_groups=3), dict(renormalize=False)):
        print("route NaN", score, biased, sorted(kw), flush=True)
        check(x, 6, score=score, bias=bias, grad=False, **kw)


def test_one_row_repeated_and_many_rows():
    print("route 300001 rows", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(300001, 16, generator=g, device=DEV)
    ids, w = rs.route_topk(x, 2)
    sub = torch.cat([torch.arange(50), torch.arange(262100, 262200), torch.arange(299951, 300001)]).to(DEV)
    rids, rw, _ = ref.route(values(x[sub]), 2)
    same(ids[sub], rids, "ids")
    close(w[sub], rw, rw * 2.0 ** -40, "weights")
    dw = torch.randn(300001, 2, generator=g, device=DEV)
    dx = rs.route_topk_grad(x, ids, w, dw)
    rdx, bound = ref.route_grad(values(x[sub]), rids, values(dw[sub]))
    close(dx[sub], rdx, bound, "dscores")
    one = x[:1].expand(37, 16)
    ids, w = rs.route_topk(one, 3)
    assert (ids == ids[0]).all() and (w == w[0]).all()
    rids, rw, _ = ref.route(values(x[:1]), 3)
    same(ids[:1], rids, "ids of a repeated row")


def test_rows_far_apart_pass_32_bit_offsets():
    stride = (1 << 31) + 8
    print("route rows 2^31 + 8 elements apart", flush=True)
    whole = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device=DEV)
    x = whole.as_strided((3, 256), (stride, 1))
    x.copy_(torch.from_numpy(np.random.default_rng(2).standard_normal((3, 256))).to(DEV))
    rids, rw, _ = ref.route(values(x), 8)
    ids, w = rs.route_topk(x, 8)
    same(ids, rids, "ids")
    close(w, rw, rw * 2.0 ** -40, "weights")


def test_gradient_of_foreign_choices():
    """A choice that is no expert is passed over, and one that stands twice counts twice."""
    print("route gradient, repeated and absent choices", flush=True)
    x = np.random.default_rng(3).standard_normal((2, 20))
    t = matrix(x, "f32")
    ids = torch.tensor([[3, 3, 5], [7, -1, 1000]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.25, 0.25, 0.5], [0.5, 0.25, 0.25]], device=DEV)
    dw = torch.tensor([[1.0, 2.0, -1.0], [1.0, 2.0, 3.0]], device=DEV)
    got = numpy_of(rs.route_topk_grad(t, ids, w, dw))
    want = np.zeros((2, 20))
    d = [(0.25 + 0.5 - 0.5), (0.5 + 0.5 + 0.75)]
    want[0, 3] = 0.25 * (1 - d[0]) + 0.25 * (2 - d[0])
    want[0, 5] = 0.5 * (-1 - d[0])
    want[1, 7] = 0.5 * (1 - d[1])
    assert np.abs(got - want).max() <= 16 * ref.U * 2   # small numbers, every product exact


def test_gradient_against_differences_of_the_forward():
    """Central differences of the library's own weights: h = 2^-6 leaves h^2 / 6 times third
    derivatives (below 1 for one logit of a softmax or sigmoid weight of scale 1) and 2 U / h."""
    x = np.random.default_rng(12).standard_normal((1, 24))
    x[0, [2, 9, 17]] += 4                           # the choice holds under the steps
    h = 2.0 ** -6
    for score, renorm in itertools.product(("softmax", "sigmoid"), (True, False)):
        print("route differences", score, renorm, flush=True)
        steps = matrix(np.concatenate([x + h * np.eye(24), x - h * np.eye(24)]), "f32")
        ids, w = rs.route_topk(steps, 3, score=score, renormalize=renorm)
        base, bw = rs.route_topk(matrix(x, "f32"), 3, score=score, renormalize=renorm)
        assert (ids.sort(1).values == base.sort(1).values).all()
        dw = np.array([[0.7, -1.1, 0.4]])
        at = {e: j for j, e in enumerate(base[0].tolist())}
        pick = np.take(dw[0], np.vectorize(at.get)(ids.cpu().numpy()))
        loss = (values(w) * pick).sum(1)
        want = (loss[:24] - loss[24:]) / (2 * h)
        got = numpy_of(rs.route_topk_grad(matrix(x, "f32"), base, bw, torch.from_numpy(dw).float().to(DEV),
                                          score=score, renormalize=renorm))[0]
        assert np.abs(got - want).max() <= 2.2 * (h * h / 6 + 4 * ref.U / h)


def test_streams_and_a_replayed_graph():
    print("route on a side stream, two streams at once, and in a graph", flush=True)
    g = np.random.default_rng(10)
    xs = [g.standard_normal((n, 256)) for n in (5000, 3001)]
    bias = g.standard_normal(256).astype(np.float32)
    kw = dict(score="sigmoid", groups=8, top_groups=4, group_best=2)
    want = [ref.route(values(matrix(x[:200], "f32")), 8, bias=bias, **kw) for x in xs]
    ts = [matrix(x, "f32") for x in xs]
    tb = torch.from_numpy(bias).to(DEV)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = [rs.route_topk(t, 8, bias=tb, stream=s, **kw) for t, s in zip(ts, streams)]
        torch.cuda.synchronize()
        for (ids, w), (rids, rw, _) in zip(outs, want):
            same(ids[:200], rids, "ids")
            close(w[:200], rw, rw * 2.0 ** -40, "weights")
    x = ts[0].clone()
    dw = torch.ones(5000, 8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = rs.route_topk(x, 8, bias=tb, **kw)
        dx = rs.route_topk_grad(x, ids, w, dw, score="sigmoid")
    for i in range(3):
        x.copy_(torch.roll(ts[0], i, 0))
        dw.fill_(float(i))
        graph.replay()
        torch.cuda.synchronize()
        eids, ew = rs.route_topk(x, 8, bias=tb, **kw)
        assert torch.equal(ids, eids) and torch.equal(w, ew)
        assert torch.equal(dx, rs.route_topk_grad(x, eids, ew, dw, score="sigmoid"))


def test_no_rows():
    x = torch.empty(0, 64, device=DEV)
    ids, w = rs.route_topk(x, 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert rs.route_topk_grad(x, ids, w, w).shape == (0, 64)


def test_wrapper_refusals():
    x = torch.zeros(4, 8, device=DEV)
    for bad in (lambda: rs.route_topk(x.t(), 2), lambda: rs.route_topk(x.double(), 2),
                lambda: rs.route_topk(x[0], 2), lambda: rs.route_topk(x, 2, bias=torch.zeros(7, device=DEV)),
                lambda: rs.route_topk(x, 2, bias=torch.zeros(8, device=DEV).half()),
                lambda: rs.route_topk_grad(x, *([torch.zeros(4, 2, device=DEV)] * 3))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(rs.RsError):
        rs.route_topk(x, 9)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_biases(score):
    """Biases near f32's ends, whose pair sums pass them, and infinite ones, with and without groups."""
    g = np.random.default_rng(20)
    x = g.standard_normal((30, 64))
    for name, bias in (("low", np.where(np.arange(64) % 8 < 6, -3.4e38, 0.1)), ("all low", np.full(64, -3.4e38)),
                       ("high", np.where(np.arange(64) % 16 < 4, 3.4e38, 0.0)), ("inf", np.where(np.arange(64) % 9 == 0, np.inf, 0.0)),
                       ("-inf", np.where(np.arange(64) % 2 == 0, -np.inf, 0.0)), ("tiny", np.full(64, 1e-42)),
                       ("cancelling", -ref.probabilities(x[:1], score)[0])):
        for kw in (dict(), dict(groups=8, top_groups=3, group_best=2), dict(groups=4, top_groups=2)):
            print("route bias", name, score, sorted(kw), flush=True)
            check(x, 8, bias=bias, score=score, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [2, 8, 9])
def test_group_sums_that_cancel(score, size):
    """Large biases of both signs in a group: their sum is small, the roundings of its terms are not."""
    g = np.random.default_rng(21)
    groups = 16
    for big in (1e3, 1e5, 1e8):
        bias = np.where(np.arange(groups * size) % size == 0, big, -big)
        print("route cancelling groups", score, size, big, flush=True)
        check(g.standard_normal((60, groups * size)), 4, score=score, bias=bias, groups=groups, top_groups=5, group_best=2)


@pytest.mark.parametrize("seed", range(40))
def test_random_combinations(seed):
    g = np.random.default_rng(1000 + seed)
    groups = int(g.choice([1, 1, 2, 3, 4, 8, 16, 33, 64]))
    size = int(g.integers(1, max(2, 1024 // groups + 1)))
    experts = groups * size
    top = int(g.integers(1, groups + 1))
    best = int(g.integers(1, min(2, size) + 1))
    k = int(g.integers(1, min(64, top * size) + 1))
    rows = int(g.integers(1, 200))
    kind = seed % 4
    x = g.standard_normal((rows, experts)) * (3.0, 1.0, 0.3, 20.0)[kind]
    if seed % 3 == 0:
        x = np.round(x * 2) / 2                     # ties
    if seed % 5 == 0:
        x[g.random(x.shape) < 0.6] = -np.inf
    kw = dict(score=("softmax", "sigmoid")[seed % 2], renormalize=bool(g.integers(2)), groups=groups, top_groups=top,
              group_best=best, scale=float(g.choice([1.0, 0.5, 2.5])))
    bias = None if g.integers(3) == 0 else np.round(g.standard_normal(experts) * 8) / 64 * g.integers(0, 2)
    dtype = ("f32", "f16", "bf16")[seed % 3]
    print("route random", seed, rows, experts, k, dtype, kw, bias is not None, flush=True)
    check(x, k, dtype, pad=seed % 7, shift=seed % 5, bias=bias, **kw)


@pytest.mark.parametrize("experts", [64, 127, 128, 129, 255, 256, 257, 1024])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gradient_of_plain_weights_at_the_borders_of_its_lanes(experts, dtype):
    g = np.random.default_rng(experts)
    for k in (1, 16, 17, 32, 33, 64):
        print("route gradient of plain weights", experts, k, dtype, flush=True)
        check(g.standard_normal((9, experts)) * 2, k, dtype, pad=k % 3, renormalize=False, scale=1.5)
