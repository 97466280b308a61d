"""The calls that move rows by index and adjust logits as a model's step makes them: one after the
other with their gradients, on other streams, in graphs, with given memory."""
import numpy as np
import pytest
import torch

import sorting_lsd_radix_amd as rs
from rows_helpers import DEV
from test_gpu_rows_calls import busy

pytestmark = pytest.mark.gpu

VOCAB, WIDTH, ROWS, EXPERTS, TOP_K, SCALE = 500, 96, 64, 8, 2, 3.0


def model(seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, by=1.0):
        return torch.randn(*shape, generator=g) * by
    return {"table": normal(VOCAB, WIDTH), "router": normal(WIDTH, EXPERTS, by=WIDTH ** -0.5),
            "experts": normal(EXPERTS, WIDTH, WIDTH, by=WIDTH ** -0.5), "head": normal(WIDTH, VOCAB, by=WIDTH ** -0.5),
            "ids": torch.randint(0, VOCAB, (ROWS,), generator=g).int(),
            "targets": torch.randint(0, VOCAB, (ROWS,), generator=g).int(), "dlogprob": normal(ROWS)}


def step(m, dtype):
    """Outputs and gradients of a step through a router's experts, with the calls."""
    t = {k: v.to(DEV) for k, v in m.items()}
    x = rs.embed_tokens(t["table"].to(dtype), t["ids"], scale=SCALE)
    scores = x.float() @ t["router"]
    chosen, w = rs.route_topk(scores, TOP_K)
    order, place, starts, _ = rs.group_choices(chosen, EXPERTS, align=16)
    y = rs.gather_choices(x, order, place)
    edges = starts.tolist()
    z, dy = torch.zeros_like(y), torch.zeros_like(y)
    for e in range(EXPERTS):
        part = slice(edges[e], edges[e + 1])
        z[part] = (y[part].float() @ t["experts"][e]).to(dtype)
    out = rs.combine_choices(z, place, weights=w)
    logits = out.float() @ t["head"]
    lp = rs.token_logprobs(logits, t["targets"])
    dlogits = rs.token_logprobs_grad(logits, lp.stats, t["targets"], dlogprob=t["dlogprob"])
    dout = (dlogits @ t["head"].T).to(dtype)
    dz, dw = rs.combine_choices_grad(dout, z, order, place, w)
    for e in range(EXPERTS):
        part = slice(edges[e], edges[e + 1])
        dy[part] = (dz[part].float() @ t["experts"][e].T).to(dtype)
    dx = rs.combine_choices(dy, place)
    dscores = rs.route_topk_grad(scores, chosen, w, dw)
    dx = (dx.float() + dscores @ t["router"].T).to(dtype)
    dtable = rs.embed_tokens_grad(dx, t["ids"], VOCAB, scale=SCALE, dtype=torch.float32)
    return {"chosen": chosen, "w": w, "out": out, "logprob": lp.logprob, "dtable": dtable, "dscores": dscores}


def reference(m, chosen):
    """The same in 64 bits by torch's autograd, with the given choices."""
    t = {k: v.double() if v.is_floating_point() else v.long() for k, v in m.items()}
    table = t["table"].requires_grad_()
    x = table[t["ids"]] * SCALE
    scores = x @ t["router"]
    scores.retain_grad()
    p = scores.softmax(1).gather(1, chosen)
    w = p / p.sum(1, keepdim=True)
    rows = torch.stack([torch.stack([x[i] @ t["experts"][e] for e in chosen[i]]) for i in range(ROWS)])
    out = (w[:, :, None] * rows).sum(1)
    lp = (out @ t["head"]).log_softmax(1).gather(1, t["targets"][:, None])[:, 0]
    (lp * t["dlogprob"]).sum().backward()
    return {"w": w, "out": out, "logprob": lp, "dtable": table.grad, "dscores": scores.grad}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_step_through_the_experts(dtype):
    """Some twenty sums of at most 96 products follow each other, forward and back.  In f32 each is off by
    at most 98 * 2^-24 of the sum of its terms' sizes, which for normal entries is some ten times the
    sum's own scale: 20 * 98 * 2^-24 * 10 = 1.2e-3 at most.  Rows kept in bf16 are rounded ten times on the
    way, by 2^-8 of each element; a sum of their products averages them, but a softmax's share of two
    experts may double them: 20 * 2^-8 = 0.08 of the largest entry."""
    print("step", dtype, flush=True)
    for seed in range(3):
        m = model(seed)
        if dtype == torch.bfloat16:
            m["table"] = m["table"].bfloat16().float()
        got = step(m, dtype)
        want = reference(m, got["chosen"].cpu().long())
        room = 1.2e-3 if dtype == torch.float32 else 20 * 2.0 ** -8
        for name, w in want.items():
            off = (got[name].double().cpu() - w.detach()).abs().max()
            assert off <= room * w.abs().max(), (name, float(off), float(w.abs().max()))
        again = step(m, dtype)
        assert all(torch.equal(got[name], again[name]) for name in want), "equal calls give equal bits"


def test_a_step_of_sampling():
    """Embedded, projected, adjusted and scored: what is masked has no probability, and the others' are those
    of the adjusted logits; a row of which nothing is left has none at all."""
    print("sampling", flush=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    table = torch.randn(VOCAB, WIDTH, generator=g, device=DEV)
    history = torch.randint(0, VOCAB, (8, 40), generator=g, device=DEV).int()
    x = rs.embed_tokens(table, history[:, -1].contiguous(), scale=0.1)
    logits = x @ table.T
    allowed = torch.rand(8, VOCAB, generator=g, device=DEV) < 0.5
    allowed[3] = False
    bits = torch.zeros(8, 512, dtype=torch.int64, device=DEV)
    bits[:, :VOCAB] = allowed
    words = (bits.view(8, 16, 32) << torch.arange(32, device=DEV)).sum(2)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    by = torch.full((8,), 1.3, device=DEV)
    adjusted = rs.adjust_logits(logits, history=history, repetition=by, presence=by, mask=words)
    lp = rs.token_logprobs(adjusted, top_k=4)
    seen = torch.zeros(8, VOCAB, dtype=torch.bool, device=DEV).scatter_(1, history.long(), True)
    l = logits.double()
    l = torch.where(seen, torch.where(l > 0, l / by.double()[:, None], l * by.double()[:, None]) - by.double()[:, None], l)
    l[~allowed] = -torch.inf
    want = l.log_softmax(1).sort(dim=1, descending=True, stable=True)
    live = [r for r in range(8) if r != 3]
    assert torch.equal(lp.top_ids[live].long(), want.indices[live, :4])
    # each adjusted logit is off by 5 roundings of at most 2^-24 of some tens, the log of the sum by as much
    assert float((lp.top_logprobs[live].double() - want.values[live, :4]).abs().max()) < 1e-4
    assert (lp.top_logprobs[3] == -torch.inf).all() and float(lp.entropy[3]) == 0.0


def calls(stream, rows=4096, width=512, k=4):
    """Every wrapper on `stream`, each as (tensors given to it alone, call on them)."""
    f = torch.randn(rows, width, device=DEV)
    ids = torch.randint(0, 32, (rows, k), device=DEV).int()
    order, place, _, _ = rs.group_choices(ids, 32)
    y = torch.randn(rows * k, width, device=DEV)
    w = torch.rand(rows, k, device=DEV)
    token = torch.randint(0, rows, (rows,), device=DEV).int()
    one = torch.rand(rows, device=DEV)
    history = torch.randint(0, width, (rows, 64), device=DEV).int()
    mask = torch.full((rows, width // 32), 0x0F0F0F0F, dtype=torch.int32, device=DEV)
    temp = rs.rs_embed_tokens_grad(0, None, 0, None, rows, rows, width, 1.0, 0, 0, None, 0, None, 0)

    def c(*tensors):
        return [t.clone() for t in tensors]
    return [
        ("gather", lambda: (c(f, order, place, w, y), lambda x, o, p, w, out: rs.gather_choices(
            x, o, p, weights=w, out=out, stream=stream))),
        ("gather grad", lambda: (c(y, f, place, w, f), lambda d, x, p, w, out: rs.gather_choices_grad(
            d, x, p, w, out=out, stream=stream))),
        ("combine", lambda: (c(y, place, w, f), lambda y, p, w, out: rs.combine_choices(
            y, p, weights=w, out=out, stream=stream))),
        ("combine grad", lambda: (c(f, y, order, place, w, y), lambda d, y, o, p, w, out: rs.combine_choices_grad(
            d, y, o, p, w, out=out, stream=stream))),
        ("embed", lambda: (c(f, token, f), lambda t, i, out: rs.embed_tokens(t, i, out=out, stream=stream))),
        ("embed grad", lambda: (c(f, token, f) + [torch.empty(temp, dtype=torch.uint8, device=DEV)],
                                lambda d, i, out, m: rs.embed_tokens_grad(d, i, rows, out=out, temp=m, stream=stream))),
        ("adjust", lambda: (c(f, history, one, mask, f, token % 64, token % 9, history, f[:, :64].contiguous()),
                            lambda x, h, one, m, out, n, q, i, b: rs.adjust_logits(
                                x, history=h, lengths=n, prompt_lengths=q, repetition=one, presence=one, frequency=one,
                                bias_ids=i, bias=b, mask=m, out=out, stream=stream))),
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


def test_two_streams_at_once():
    """Calls of the same kind side by side, each with its own memory, give what they give alone."""
    print("two streams", flush=True)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    made = [[(name, make()) for name, make in calls(s)] for s in sides]
    alone = []
    torch.cuda.synchronize()
    for k in range(2):
        for name, (tensors, call) in made[k]:
            got = call(*tensors)
            torch.cuda.synchronize()
            alone.append([t.clone() for t in (got if isinstance(got, tuple) else (got,))])
    torch.cuda.synchronize()
    together = [[], []]
    for a, b in zip(*made):
        for k, (name, (tensors, call)) in enumerate((a, b)):
            together[k].append(call(*tensors))
    torch.cuda.synchronize()
    for want, (got, name) in zip(alone, [(g, m[0]) for k in range(2) for g, m in zip(together[k], made[k])]):
        for g, w in zip(got if isinstance(got, tuple) else (got,), want):
            assert torch.equal(g, w), name


def test_captured_calls_on_a_given_stream():
    """In a graph on a stream given by name, replayed with the program's own work between."""
    print("capture on a given stream", flush=True)
    side = torch.cuda.Stream()
    made = [(name, make()) for name, make in calls(side)]
    torch.cuda.synchronize()
    eager = {name: call(*tensors) for name, (tensors, call) in made}
    torch.cuda.synchronize()   # the copies are made on another stream
    want = {name: [t.clone() for t in (r if isinstance(r, tuple) else (r,))] for name, r in eager.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = {name: call(*tensors) for name, (tensors, call) in made}
    for i in range(4):
        for r in got.values():
            for t in r if isinstance(r, tuple) else (r,):
                t.fill_(-3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, r in got.items():
            for g, w in zip(r if isinstance(r, tuple) else (r,), want[name]):
                assert torch.equal(g, w), (i, name)
        torch.empty(1 << 22, device=DEV).normal_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("n,vocab", [(300, 50), (300, 5000), (20000, 900), (600000, 900)])
def test_temps(n, vocab):
    """A temp is memory of the tensors' device, all of it, as much as the call asks for and no more."""
    print("temps", n, vocab, flush=True)
    x = torch.randn(n, 40, device=DEV).half()
    ids = torch.randint(-1, vocab, (n,), device=DEV).int()

    def call(m):
        return rs.embed_tokens_grad(x, ids, vocab, temp=m)
    need = rs.rs_embed_tokens_grad(1, None, 0, None, n, vocab, 40, 1.0, 0, 1, None, 0, None, 0)
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device=DEV).expand(need),
                torch.empty(need, 2, dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(TypeError):
            call(bad)
    with pytest.raises(rs.RsError) as e:
        call(torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == rs.RS_ERR_TEMP_TOO_SMALL
    want = call(None)
    for garbage in (-1, 0x55555555):
        whole = torch.full((need // 4 + 4,), garbage, dtype=torch.int32, device=DEV)   # any type, by its bytes
        assert torch.equal(call(whole[:-4]), want)
        assert (whole[-4:] == garbage).all()


def test_counts_past_32_bits():
    print("counts past 2^32", flush=True)
    long = torch.empty(1, (1 << 32) + 100, dtype=torch.float16, device=DEV)
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    w = torch.zeros(1, 1, device=DEV)
    x = torch.zeros(1, 8, device=DEV)
    for call in (lambda: rs.gather_choices(long, i, p), lambda: rs.combine_choices(long, p),
                 lambda: rs.gather_choices_grad(long, long, p, w), lambda: rs.combine_choices_grad(long, long, i, p, w),
                 lambda: rs.embed_tokens(long, i), lambda: rs.embed_tokens_grad(long, i, 8),
                 lambda: rs.embed_tokens_grad(x, i, (1 << 32) + 8), lambda: rs.adjust_logits(long),
                 lambda: rs.embed_tokens_grad(x, i, -1)):
        with pytest.raises(rs.RsError) as e:
            call()
        assert e.value.status == rs.RS_ERR_UNSUPPORTED_SIZE


def test_what_the_wrappers_refuse():
    print("refusals", flush=True)
    x = torch.zeros(4, 8, device=DEV)
    i = torch.zeros(8, dtype=torch.int32, device=DEV)
    p = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    y = torch.zeros(8, 8, device=DEV)
    f = torch.zeros(4, device=DEV)
    for call in (
            lambda: rs.gather_choices(x.T, i, p), lambda: rs.gather_choices(x, i.long(), p),
            lambda: rs.gather_choices(x, i, p.view(-1)), lambda: rs.gather_choices(x, i, p[:3]),
            lambda: rs.gather_choices(x, i.view(2, 4), p), lambda: rs.gather_choices(x, i, p, weights=w.half()),
            lambda: rs.gather_choices(x, i, p, out=y.half()), lambda: rs.gather_choices(x, i, p, out=y[:7]),
            lambda: rs.gather_choices(x.double(), i, p), lambda: rs.gather_choices(x, i[::2], p),
            lambda: rs.combine_choices(y, p, weights=w[:3]), lambda: rs.combine_choices(y, p.float()),
            lambda: rs.combine_choices(y, i), lambda: rs.gather_choices_grad(y.half(), x, p, w),
            lambda: rs.gather_choices_grad(y[:, :7], x, p, w), lambda: rs.gather_choices_grad(y, x, p, None),
            lambda: rs.combine_choices_grad(x[:, :7], y, i, p, w), lambda: rs.combine_choices_grad(x, y, i[:7], p, w),
            lambda: rs.embed_tokens(x, i.long()), lambda: rs.embed_tokens(x, i[::2]),
            lambda: rs.embed_tokens(x, i, out=y.view(2, 4, 8)), lambda: rs.embed_tokens_grad(x, i, 5),
            lambda: rs.embed_tokens_grad(y, i, 5, accumulate=True), lambda: rs.embed_tokens_grad(y, i, 5, dtype=torch.float16),
            lambda: rs.embed_tokens_grad(y, i, 5, out=x), lambda: rs.adjust_logits(x, bias=w),
            lambda: rs.adjust_logits(x, repetition=f), lambda: rs.adjust_logits(x, history=p[:3]),
            lambda: rs.adjust_logits(x, history=p, lengths=f), lambda: rs.adjust_logits(x, history=p, repetition=f.double()),
            lambda: rs.adjust_logits(x, mask=p), lambda: rs.adjust_logits(x, bias_ids=p, bias=w[:, :1]),
            lambda: rs.adjust_logits(x, dtype=torch.float16), lambda: rs.adjust_logits(x, out=y[:4, :7]),
            lambda: rs.adjust_logits(x, history=p.cpu()), lambda: rs.adjust_logits(x, history=p.T.contiguous().T)):
        with pytest.raises((TypeError, AttributeError)):
            call()
    for call in (lambda: rs.gather_choices(x, i, p, out=torch.zeros(1, 8, device=DEV).expand(8, 8)),
                 lambda: rs.embed_tokens(y, i, scale=float("nan"))):
        with pytest.raises(rs.RsError) as e:
            call()
        assert e.value.status == rs.RS_ERR_INVALID_VALUE
    for call in (lambda: rs.gather_choices(y[:4], i, p, out=y), lambda: rs.combine_choices(y, p, out=y[:4]),
                 lambda: rs.embed_tokens(y, i, out=y), lambda: rs.embed_tokens_grad(y, i, 8, out=y),
                 lambda: rs.adjust_logits(y[:, :6], out=y[:, 1:7])):
        with pytest.raises(rs.RsError) as e:
            call()
        assert e.value.status == rs.RS_ERR_OVERLAP
