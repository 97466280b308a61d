"""Calls on rows of scores, on the CPU: what they refuse before anything is launched, their size
queries, and the reference's gradients against differences."""
import ctypes

import numpy as np
import pytest

import rows_reference as ref
import sorting_lsd_radix_amd as rs

# never-dereferenced addresses: every case fails a host check first
A, B, C, D, E, F, T = (0x10000000 * i for i in range(1, 8))
G, H, I, J = (0x100000000 * i for i in range(1, 5))


def refused(status, call, *args, **kw):
    with pytest.raises(rs.RsError) as ei:
        call(*args, **kw)
    assert ei.value.status == status, (args, ei.value)


def route(et=0, scores=A, stride=256, bias=B, rows=16, experts=256, k=8, fn=1, groups=8, top_groups=4,
          best=2, renorm=1, scale=1.0, ids=C, weights=D):
    rs.rs_route_topk(et, scores, stride, bias, rows, experts, k, fn, groups, top_groups, best, renorm,
                     scale, ids, weights, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(et=3), rs.RS_ERR_INVALID_VALUE), (dict(et=-1), rs.RS_ERR_INVALID_VALUE),
    (dict(fn=2), rs.RS_ERR_INVALID_VALUE),
    (dict(experts=0), rs.RS_ERR_INVALID_VALUE),
    (dict(experts=1025), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(rows=1 << 30), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(k=65), rs.RS_ERR_UNSUPPORTED_SIZE), (dict(k=0), rs.RS_ERR_INVALID_VALUE),
    (dict(k=33, top_groups=1), rs.RS_ERR_INVALID_VALUE),        # a group holds 32
    (dict(groups=0), rs.RS_ERR_INVALID_VALUE), (dict(groups=3), rs.RS_ERR_INVALID_VALUE),
    (dict(groups=128), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(top_groups=0), rs.RS_ERR_INVALID_VALUE), (dict(top_groups=9), rs.RS_ERR_INVALID_VALUE),
    (dict(best=0), rs.RS_ERR_INVALID_VALUE), (dict(best=3), rs.RS_ERR_INVALID_VALUE),
    (dict(experts=8, groups=8, best=2, k=1), rs.RS_ERR_INVALID_VALUE),   # groups of one expert
    (dict(scale=0.0), rs.RS_ERR_INVALID_VALUE), (dict(scale=-1.0), rs.RS_ERR_INVALID_VALUE),
    (dict(scale=float("nan")), rs.RS_ERR_INVALID_VALUE), (dict(scale=float("inf")), rs.RS_ERR_INVALID_VALUE),
    (dict(scores=None), rs.RS_ERR_INVALID_VALUE), (dict(ids=None), rs.RS_ERR_INVALID_VALUE),
    (dict(weights=None), rs.RS_ERR_INVALID_VALUE),
    (dict(scores=A + 2), rs.RS_ERR_MISALIGNED), (dict(et=1, scores=A + 1), rs.RS_ERR_MISALIGNED),
    (dict(bias=B + 2), rs.RS_ERR_MISALIGNED), (dict(ids=C + 2), rs.RS_ERR_MISALIGNED),
    (dict(weights=D + 1), rs.RS_ERR_MISALIGNED),
    (dict(ids=A + 64), rs.RS_ERR_OVERLAP), (dict(weights=C + 4), rs.RS_ERR_OVERLAP),
    (dict(weights=B + 1020), rs.RS_ERR_OVERLAP),
    (dict(stride=1 << 62), rs.RS_ERR_INVALID_VALUE),
])
def test_route_refusals(kw, status):
    refused(status, route, **kw)


def test_route_of_no_rows_launches_nothing():
    route(rows=0, scores=None, ids=None, weights=None)


def route_grad(et=0, scores=A, stride=256, ids=B, weights=C, dweights=D, rows=16, experts=256, k=8, fn=0,
               renorm=1, scale=1.0, dscores=E, dstride=256):
    rs.rs_route_topk_grad(et, scores, stride, ids, weights, dweights, rows, experts, k, fn, renorm, scale,
                          dscores, dstride, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(et=7), rs.RS_ERR_INVALID_VALUE), (dict(fn=-1), rs.RS_ERR_INVALID_VALUE),
    (dict(experts=2000), rs.RS_ERR_UNSUPPORTED_SIZE), (dict(k=65), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(rows=1 << 31), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(experts=4), rs.RS_ERR_INVALID_VALUE), (dict(k=0), rs.RS_ERR_INVALID_VALUE),
    (dict(scale=0.0), rs.RS_ERR_INVALID_VALUE), (dict(dstride=255), rs.RS_ERR_INVALID_VALUE),
    (dict(dscores=None), rs.RS_ERR_INVALID_VALUE), (dict(dweights=None), rs.RS_ERR_INVALID_VALUE),
    (dict(dscores=E + 2), rs.RS_ERR_MISALIGNED), (dict(weights=C + 2), rs.RS_ERR_MISALIGNED),
    (dict(dscores=A), rs.RS_ERR_OVERLAP), (dict(dscores=B - 256), rs.RS_ERR_OVERLAP),
    (dict(dscores=C), rs.RS_ERR_OVERLAP), (dict(dscores=D), rs.RS_ERR_OVERLAP),
])
def test_route_grad_refusals(kw, status):
    refused(status, route_grad, **kw)


def group(ids=A, n=1000, experts=64, align=16, order=B, place=C, starts=D, counts=E, temp=T, size=1 << 20):
    return rs.rs_group_choices(ids, n, experts, align, order, place, starts, counts, temp, size, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(experts=0), rs.RS_ERR_INVALID_VALUE), (dict(experts=1025), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(align=0), rs.RS_ERR_INVALID_VALUE), (dict(align=1 << 25), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(n=1 << 30), rs.RS_ERR_UNSUPPORTED_SIZE), (dict(n=(1 << 30) - 64 * 15), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(ids=None), rs.RS_ERR_INVALID_VALUE), (dict(order=None), rs.RS_ERR_INVALID_VALUE),
    (dict(place=None), rs.RS_ERR_INVALID_VALUE), (dict(starts=None), rs.RS_ERR_INVALID_VALUE),
    (dict(counts=None), rs.RS_ERR_INVALID_VALUE),
    (dict(ids=A + 4), rs.RS_ERR_MISALIGNED), (dict(order=B + 8), rs.RS_ERR_MISALIGNED),
    (dict(place=C + 4), rs.RS_ERR_MISALIGNED), (dict(starts=D + 2), rs.RS_ERR_MISALIGNED),
    (dict(temp=T + 4), rs.RS_ERR_MISALIGNED), (dict(size=3), rs.RS_ERR_TEMP_TOO_SMALL),
    (dict(place=A), rs.RS_ERR_OVERLAP), (dict(order=A + 2000), rs.RS_ERR_OVERLAP),
    (dict(starts=E - 4), rs.RS_ERR_OVERLAP), (dict(temp=B + 64), rs.RS_ERR_OVERLAP),
])
def test_group_refusals(kw, status):
    refused(status, group, **kw)


def test_group_size_query():
    q = rs.rs_group_choices(None, 1 << 20, 256, 128, None, None, None, None, None, 0)
    assert 0 < q <= 4 << 20
    assert q == rs.rs_group_choices(None, 1 << 20, 256, 1, None, None, None, None, None, 0)
    assert rs.rs_group_choices(None, 0, 1, 1, None, None, None, None, None, 0) > 0
    refused(rs.RS_ERR_UNSUPPORTED_SIZE, rs.rs_group_choices, None, 1 << 30, 256, 1, None, None, None, None,
            None, 0)


def logprobs(et=2, logits=G, stride=1000, targets=A, rows=8, vocab=1000, scale=1.0, k=5, stats=B, lse=C,
             entropy=D, logprob=E, rank=F, top_ids=H, top_lp=I, temp=J, size=1 << 24):
    rs.rs_token_logprobs(et, logits, stride, targets, rows, vocab, scale, k, stats, lse, entropy, logprob,
                         rank, top_ids, top_lp, temp, size, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(et=3), rs.RS_ERR_INVALID_VALUE), (dict(vocab=0), rs.RS_ERR_INVALID_VALUE),
    (dict(vocab=4), rs.RS_ERR_INVALID_VALUE),                    # fewer logits than alternatives
    (dict(vocab=1 << 30), rs.RS_ERR_UNSUPPORTED_SIZE), (dict(rows=1 << 30), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(k=65), rs.RS_ERR_UNSUPPORTED_SIZE),
    (dict(scale=0.0), rs.RS_ERR_INVALID_VALUE), (dict(scale=-2.0), rs.RS_ERR_INVALID_VALUE),
    (dict(scale=float("nan")), rs.RS_ERR_INVALID_VALUE), (dict(scale=float("inf")), rs.RS_ERR_INVALID_VALUE),
    (dict(scale=1e-30), rs.RS_ERR_INVALID_VALUE),
    (dict(logits=None), rs.RS_ERR_INVALID_VALUE), (dict(stats=None), rs.RS_ERR_INVALID_VALUE),
    (dict(targets=None), rs.RS_ERR_INVALID_VALUE),
    (dict(targets=None, logprob=None), rs.RS_ERR_INVALID_VALUE),
    (dict(top_ids=None), rs.RS_ERR_INVALID_VALUE), (dict(top_lp=None), rs.RS_ERR_INVALID_VALUE),
    (dict(k=0), rs.RS_ERR_INVALID_VALUE),                        # alternatives' arrays without any
    (dict(logits=G + 1), rs.RS_ERR_MISALIGNED), (dict(et=0, logits=G + 2), rs.RS_ERR_MISALIGNED),
    (dict(stats=B + 2), rs.RS_ERR_MISALIGNED), (dict(temp=J + 8), rs.RS_ERR_MISALIGNED),
    (dict(vocab=1 << 20, stride=1 << 20, size=16), rs.RS_ERR_TEMP_TOO_SMALL),
    (dict(lse=G + 100), rs.RS_ERR_OVERLAP), (dict(rank=E), rs.RS_ERR_OVERLAP),
    (dict(top_ids=A + 4), rs.RS_ERR_OVERLAP),
    (dict(stride=1 << 62), rs.RS_ERR_INVALID_VALUE),
])
def test_logprobs_refusals(kw, status):
    refused(status, logprobs, **kw)


def test_logprobs_of_no_rows_launches_nothing():
    logprobs(rows=0, logits=None, stats=None)


def logprobs_grad(et=2, logits=G, stride=1000, targets=A, stats=B, entropy=C, rows=8, vocab=1000, scale=1.0,
                  dlp=D, dh=E, dlse=F, dlogits=H, dstride=1000):
    rs.rs_token_logprobs_grad(et, logits, stride, targets, stats, entropy, rows, vocab, scale, dlp, dh, dlse,
                              dlogits, dstride, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(et=3), rs.RS_ERR_INVALID_VALUE), (dict(vocab=0), rs.RS_ERR_INVALID_VALUE),
    (dict(rows=1 << 30), rs.RS_ERR_UNSUPPORTED_SIZE), (dict(dstride=999), rs.RS_ERR_INVALID_VALUE),
    (dict(scale=0.0), rs.RS_ERR_INVALID_VALUE),
    (dict(dlp=None, dh=None, dlse=None), rs.RS_ERR_INVALID_VALUE),
    (dict(targets=None), rs.RS_ERR_INVALID_VALUE), (dict(entropy=None), rs.RS_ERR_INVALID_VALUE),
    (dict(stats=None), rs.RS_ERR_INVALID_VALUE), (dict(dlogits=None), rs.RS_ERR_INVALID_VALUE),
    (dict(dlogits=H + 1), rs.RS_ERR_MISALIGNED), (dict(dlp=D + 1), rs.RS_ERR_MISALIGNED),
    (dict(dlogits=G + 2000), rs.RS_ERR_OVERLAP),
    (dict(dlogits=G, dstride=1001), rs.RS_ERR_OVERLAP),          # in place only with the same stride
    (dict(dlogits=B), rs.RS_ERR_OVERLAP),
])
def test_logprobs_grad_refusals(kw, status):
    refused(status, logprobs_grad, **kw)


def test_wrappers_refuse_what_is_no_matrix_on_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    for call in (lambda: rs.route_topk(x, 2), lambda: rs.token_logprobs(x),
                 lambda: rs.group_choices(torch.zeros(4, dtype=torch.int32), 8),
                 lambda: rs.token_logprobs_grad(x, torch.zeros(4, 2), dlse=torch.zeros(4)),
                 lambda: rs.route_topk_grad(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2),
                                            torch.zeros(4, 2))):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("call,counts", [
    (route, ("experts", "k", "groups", "top_groups", "best")), (route_grad, ("experts", "k")),
    (group, ("experts", "align")), (logprobs, ("vocab", "k")), (logprobs_grad, ("vocab",))])
def test_counts_past_32_bits_are_refused_as_what_they_are(call, counts):
    """The C interface has 32 bits for each of these; 2^32 + 8 is not 8, and -1 is no count."""
    for name in counts:
        for more in (1 << 32, (1 << 32) + 8, (1 << 33) + 1, 1 << 64, -1, -(1 << 32) + 4):
            refused(rs.RS_ERR_UNSUPPORTED_SIZE, call, **{name: more})


class StreamOf:
    """As much of a torch stream as is looked at before it is used."""

    def __init__(self, device):
        self.device = device


def test_a_stream_of_another_device_is_refused():
    torch = pytest.importorskip("torch")
    rs._load_torch()
    with pytest.raises(TypeError, match="cuda:1"):
        rs._run_on(1, StreamOf(torch.device("cuda:0")), lambda on: pytest.fail("called"))


def test_a_temp_that_is_not_the_devices_own_memory_is_refused():
    torch = pytest.importorskip("torch")
    size = ctypes.c_size_t(64)
    for temp in (torch.empty(64, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8).expand(64)):
        with pytest.raises(TypeError, match="temp"):
            rs._temp_arg(temp, size, torch.device("cuda:0"))


# --- the reference -----------------------------------------------------------------------------------

def differences(f, x, h=1e-5):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        out[i] = (f(up) - f(down)) / (2 * h)
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_formula_against_differences(score, renormalize):
    g = np.random.default_rng(3)
    x, dw = g.standard_normal((4, 9)), g.standard_normal((4, 3))
    kw = dict(score=score, renormalize=renormalize, scale=1.7)
    ids, _, _ = ref.route(x, 3, **kw)

    def loss(y):   # the choice held fixed
        p = ref.probabilities(y, score)[np.arange(4)[:, None], ids]
        w = 1.7 * (p / p.sum(1, keepdims=True) if renormalize else p)
        return (w * dw).sum()

    dx, bound = ref.route_grad(x, ids, dw, **kw)
    # central differences at h = 1e-5: h^2 / 6 of third derivatives below 100, and 2e-16 * 20 / h
    assert np.allclose(dx, differences(loss, x), rtol=0, atol=1e-8)
    assert (bound >= 0).all()


def test_logprob_gradient_formula_against_differences():
    g = np.random.default_rng(4)
    x = g.standard_normal((3, 11)) * 2
    t = np.array([4, 11, 0])
    a, h, q = g.standard_normal((3, 3))

    def loss(y):
        o, _ = ref.logprobs(y, t, 0, 0.8)
        return (a * o["logprob"] + h * o["entropy"] + q * o["lse"]).sum()

    dx, _ = ref.logprobs_grad(x, t, 0.8, a, h, q)
    assert np.allclose(dx, differences(loss, x), rtol=0, atol=1e-8)


def test_reference_on_small_cases_by_hand():
    ids, w, _ = ref.route(np.array([[0.0, 1.0, 1.0, -0.0]]), 4)
    assert ids.tolist() == [[1, 2, 0, 3]] and abs(w.sum() - 1) < 1e-15
    ids, w, _ = ref.route(np.full((1, 4), -np.inf), 2)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]
    # two groups of two: the sums 5 and 6 of the best two, though the largest is in the first
    b = np.array([5.0, 0.0, 3.0, 3.0], np.float32)
    ids, _, _ = ref.route(np.zeros((1, 4)), 2, bias=b, groups=2, top_groups=1, group_best=2)
    assert ids.tolist() == [[2, 3]]
    order, place, starts, counts = ref.group(np.array([2, 0, 2, 7], np.uint32), 3, 4)
    assert order.tolist() == [1, -1, -1, -1, 0, 2, -1, -1, -1, -1, -1, -1, -1]
    assert place.tolist() == [4, 0, 5, -1] and starts.tolist() == [0, 4, 4, 8] and counts.tolist() == [1, 0, 2]
    o, _ = ref.logprobs(np.array([[0.0, np.log(3.0), 0.0]]), np.array([2]), 2, 1.0)
    assert np.allclose(o["logprob"], np.log(0.2)) and o["rank"].tolist() == [2]
    assert o["top_ids"].tolist() == [[1, 0]]
    assert np.allclose(o["entropy"], -(0.6 * np.log(0.6) + 0.4 * np.log(0.2)))
