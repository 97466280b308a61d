"""How the tensor wrappers of the calls on rows of scores treat streams, memory and sizes."""
import numpy as np
import pytest
import torch

import rows_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, same

pytestmark = pytest.mark.gpu


def busy(stream=None):
    """Some fifty milliseconds of copies on a stream."""
    a = torch.empty(1 << 28, device=DEV)
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        for _ in range(120):
            b.copy_(a)
    return a, b


def test_address_0_is_the_default_stream():
    """An address is of the stream that it names, 0 of the default one: the calls run behind what
    that stream has to do before."""
    print("streams by address", flush=True)
    side = torch.cuda.Stream()
    rs.route_topk(torch.zeros(4, 8, device=DEV), 2)
    for on, address in ((torch.cuda.default_stream(), 0), (side, side.cuda_stream)):
        assert on.cuda_stream == address
        assert rs._run_on(0, address, lambda s: s) == address
        ids = torch.zeros(1000, dtype=torch.int32, device=DEV)
        late = torch.arange(1000, dtype=torch.int32, device=DEV) % 7
        held = busy(on)
        with torch.cuda.stream(on):
            ids.copy_(late)
        got = rs.group_choices(ids, 7, stream=address)
        torch.cuda.synchronize()
        for g, want in zip(got, ref.group(np.arange(1000) % 7, 7, 1)):
            same(g, want, "stream %d" % address)
        del held


def calls(stream, rows=4096, cols=512):
    """Every wrapper on `stream`, each as (tensors given to it alone, call on them)."""
    x = torch.randn(rows, cols, device=DEV)
    b = torch.randn(cols, device=DEV)
    i = torch.zeros(rows, 8, dtype=torch.int32, device=DEV)
    w = torch.rand(rows, 8, device=DEV)
    t = torch.zeros(rows, dtype=torch.int32, device=DEV)
    r = [torch.rand(rows, device=DEV) for _ in range(4)]
    st = torch.ones(rows, 2, device=DEV)

    def temp(n):
        return torch.empty(n, dtype=torch.uint8, device=DEV)

    return [
        ("route", lambda: ([x.clone(), b.clone()], lambda x, b: rs.route_topk(x, 8, bias=b, stream=stream))),
        ("route grad", lambda: ([x.clone(), i.clone(), w.clone(), w.clone(), torch.empty_like(x)],
                                lambda x, i, w, d, o: rs.route_topk_grad(x, i, w, d, out=o, stream=stream))),
        ("group", lambda: ([i.clone(), temp(1 << 20)],
                           lambda i, m: rs.group_choices(i, 64, temp=m, stream=stream))),
        ("logprobs", lambda: ([x.clone(), t.clone(), temp(1 << 20)],
                              lambda x, t, m: rs.token_logprobs(x, t, top_k=3, temp=m, stream=stream))),
        ("logprobs grad", lambda: ([x.clone(), st.clone(), t.clone(), *(v.clone() for v in r), torch.empty_like(x)],
                                   lambda x, s, t, a, e, h, q, o: rs.token_logprobs_grad(
                                       x, s, t, dlogprob=a, entropy=e, dentropy=h, dlse=q, out=o, stream=stream))),
    ]


@pytest.mark.parametrize("by", ["stream", "address"])
def test_what_a_call_was_given_may_be_dropped_at_once(by):
    """While the call waits on another stream, its inputs, `out` and `temp` do not go to the next
    allocations of their own stream."""
    side = torch.cuda.Stream()
    busy(side)
    torch.cuda.synchronize()
    for name, make in calls(side if by == "stream" else side.cuda_stream):
        print("dropped inputs:", name, flush=True)
        tensors, call = make()
        torch.cuda.synchronize()
        held = busy(side)
        sizes = [(t.numel() * t.element_size(), t.data_ptr()) for t in tensors]
        result = call(*tensors)
        del tensors, result, call
        again = [torch.empty(n, dtype=torch.uint8, device=DEV) for n, _ in sizes for _ in range(2)]
        assert not side.query(), "the copies in front were to take longer than this"
        assert not {t.data_ptr() for t in again} & {p for _, p in sizes}, name
        torch.cuda.synchronize()
        del held, again


def test_captured_calls_on_a_given_stream():
    """The stream that captures, given by name, is the current one in all but name."""
    print("capture on a given stream", flush=True)
    x = torch.randn(300, 64, device=DEV)
    want = rs.route_topk(x, 4)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ids, w = rs.route_topk(x + 0.0, 4, stream=side)
    for _ in range(3):
        ids.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
        torch.empty(1 << 22, device=DEV).normal_()
        torch.cuda.synchronize()


def test_temps():
    """A temp is memory of the tensors' device, all of it, and as much as the call asks for."""
    print("temps", flush=True)
    ids = torch.arange(50000, dtype=torch.int32, device=DEV) % 9
    x = torch.randn(2, 70000, device=DEV)
    for call, need in ((lambda m: rs.group_choices(ids, 9, temp=m),
                        rs.rs_group_choices(None, 50000, 9, 1, *([None] * 5), 0)),
                       (lambda m: rs.token_logprobs(x, top_k=4, temp=m),
                        rs.rs_token_logprobs(0, None, 70000, None, 2, 70000, 1.0, 4, *([None] * 8), 0))):
        assert need > rs.RS_NO_TEMP
        for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device=DEV).expand(need),
                    torch.empty(need, 2, dtype=torch.uint8, device=DEV)[:, 0]):
            with pytest.raises(TypeError):
                call(bad)
        with pytest.raises(rs.RsError) as e:
            call(torch.empty(need - 1, dtype=torch.uint8, device=DEV))
        assert e.value.status == rs.RS_ERR_TEMP_TOO_SMALL
        whole = torch.full((need // 4 + 4,), -7, dtype=torch.int32, device=DEV)   # any type, by its bytes
        for got, want in zip(call(whole[:-4]), call(None)):
            assert got is want is None or torch.equal(got, want)
        assert (whole[-4:] == -7).all()


def test_rows_and_counts_past_32_bits():
    print("counts past 2^32", flush=True)
    long = torch.empty(1, (1 << 32) + 100, dtype=torch.float16, device=DEV)
    x = torch.zeros(4, 64, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    one = torch.zeros(1, device=DEV)
    stats = torch.ones(1, 2, device=DEV)
    for call in (lambda: rs.token_logprobs(long), lambda: rs.token_logprobs_grad(long, stats, dlse=one),
                 lambda: rs.route_topk(long, 8), lambda: rs.route_topk_grad(long, ids[:1], w[:1], w[:1]),
                 lambda: rs.route_topk(x, (1 << 32) + 2), lambda: rs.route_topk(x, -1),
                 lambda: rs.route_topk(x, 2, groups=(1 << 32) + 1), lambda: rs.token_logprobs(x, top_k=1 << 32),
                 lambda: rs.group_choices(ids, (1 << 32) + 8), lambda: rs.group_choices(ids, 8, align=(1 << 32) + 1)):
        with pytest.raises(rs.RsError) as e:
            call()
        assert e.value.status == rs.RS_ERR_UNSUPPORTED_SIZE


@pytest.mark.parametrize("top_k", [1, 2, 3, 5, 6])
def test_groups_of_a_slice_of_a_batch(top_k):
    """The ids of some rows of a batch begin anywhere, on a given stream and in a graph as well."""
    print("slices of ids, top_k", top_k, flush=True)
    whole = np.random.default_rng(top_k).integers(-1, 40, (700, top_k)).astype(np.int32)
    ids = torch.from_numpy(whole).to(DEV)
    side = torch.cuda.Stream()
    for first, rows in ((1, 5), (2, 697), (3, 1), (7, 0), (699, 1)):
        want = ref.group(whole[first:first + rows], 40, 8)
        torch.cuda.synchronize()
        for stream in (None, side):
            got = rs.group_choices(ids[first:first + rows], 40, align=8, stream=stream)
            torch.cuda.synchronize()
            assert got[1].shape == (rows, top_k)
            for g, w in zip(got, want):
                same(g.reshape(-1), w, "from row %d" % first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rs.group_choices(ids[1:], 40, align=8)
    for i in range(4):
        now = np.roll(whole, i, 0)
        ids.copy_(torch.from_numpy(now))
        graph.replay()
        torch.cuda.synchronize()
        for g, w, e in zip(got, ref.group(now[1:], 40, 8), rs.group_choices(ids[1:], 40, align=8)):
            same(g.reshape(-1), w, "replay %d" % i)
            assert torch.equal(g, e)
