"""Penalties, biases and masks on logits against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import moves_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, DTYPES, close, matrix, values

pytestmark = pytest.mark.gpu


def on(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rules(rng, rows, vocab, history=0, biases=0, masked=None):
    """Arguments of the reference, by name."""
    r = {}
    if history:
        h = np.minimum(rng.zipf(1.4, (rows, history)) - 1, vocab - 1).astype(np.int32)
        h = rng.permutation(vocab).astype(np.int32)[h]
        odd = rng.random((rows, history)) < 0.05
        h[odd] = rng.choice([-1, vocab, 2 ** 31 - 1], odd.sum())
        lengths = rng.integers(0, history + 1, rows).astype(np.int32)
        lengths[0] = history
        lengths[-1] = rng.choice([-5, 0, history + 3])
        r.update(history=h, lengths=lengths, prompts=rng.integers(-1, history + 2, rows).astype(np.int32),
                 repetition=(0.5 + rng.random(rows)).astype(np.float32),
                 presence=rng.standard_normal(rows).astype(np.float32),
                 frequency=rng.standard_normal(rows).astype(np.float32))
    if biases:
        ids = rng.integers(-2, vocab + 2, (rows, biases)).astype(np.int32)
        ids[:, -1] = ids[:, 0]   # the last of two counts
        r.update(bias_ids=ids, bias=(rng.standard_normal((rows, biases)) * 9).astype(np.float32))
    if masked is not None:
        r["allowed"] = rng.random((rows, vocab)) >= masked
    return r


def call(x, r, **kw):
    mask = None if "allowed" not in r else on(ref.mask_words(r["allowed"]))
    args = {k: on(v) for k, v in r.items() if k not in ("allowed", "prompts")}
    return rs.adjust_logits(x, mask=mask, prompt_lengths=on(r.get("prompts")), **args, **kw)


# rows, vocabulary, tokens of history, bias entries, share masked, elements between rows, before the first
SHAPES = [
    (1, 1, 1, 1, 0.5, 0, 0), (2, 31, 5, 3, 0.5, 0, 0), (3, 32, 40, 0, None, 1, 1), (4, 33, 0, 7, None, 0, 3),
    (5, 1000, 200, 30, 0.9, 0, 0), (3, 8191, 300, 0, 0.3, 8, 0), (2, 8193, 3000, 300, None, 0, 0),
    (7, 20011, 0, 0, 0.99, 5, 2), (2, 40000, 1000, 300, 0.5, 0, 0), (3, 700, 0, 0, None, 0, 1),
    (1, 131072, 40000, 10, 0.5, 0, 0), (2, 9000, 10, 70000, None, 0, 0),
]


@pytest.mark.parametrize("dtype,to", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("shape", SHAPES)
def test_adjust(shape, dtype, to):
    print("adjust", shape, dtype, to, flush=True)
    rows, vocab, history, biases, masked, pad, shift = shape
    rng = np.random.default_rng(rows + vocab)
    x = rng.standard_normal((rows, vocab)) * 4
    x[rng.random((rows, vocab)) < 0.05] = 0.0
    x = matrix(x, dtype, pad, shift)
    before = values(x)
    r = rules(rng, rows, vocab, history, biases, masked)
    want, bound = ref.adjust(before, **r)
    got = call(x, r, dtype=DTYPES[to])
    assert got.dtype == DTYPES[to] and got.is_contiguous()
    close(got, want, bound, "logits", to)
    assert np.array_equal(values(x), before)
    whole = torch.full((rows, vocab + pad), 7.0, dtype=DTYPES[to], device=DEV)
    out = whole[:, :vocab]
    assert call(x, r, out=out) is out
    assert torch.equal(out, got) and (whole[:, vocab:] == 7.0).all()
    if dtype == to:
        assert call(x, r, out=x) is x   # in place
        assert torch.equal(x, got)


@pytest.mark.parametrize("dtype,rows", [("f32", 40), ("bf16", 70)])
@pytest.mark.parametrize("history,biases", [(0, 0), (600, 20), (17000, 20), (600, 600)])
def test_many_rows(history, biases, dtype, rows):
    """So many logits that a thread takes two vectors, with every kind of lists."""
    print("many rows", history, biases, dtype, flush=True)
    rng = np.random.default_rng(rows + history + biases)
    vocab = 131072
    x = matrix(rng.standard_normal((rows, vocab)), dtype)
    r = rules(rng, rows, vocab, history, biases, 0.5)
    got = call(x, r)
    close(got, *ref.adjust(values(x), **r), "logits", dtype)
    assert torch.equal(call(x, r, out=x), got)


@pytest.mark.parametrize("only", ["history", "lengths", "prompts", "repetition", "presence", "frequency"])
def test_each_rule_alone(only):
    """Whatever of the lists and penalties is given, the others have their neutral value."""
    print("alone:", only, flush=True)
    rng = np.random.default_rng(len(only))
    r = rules(rng, 5, 3000, 500)
    r = {k: v for k, v in r.items() if k in ("history", only)}
    if only in ("lengths", "prompts"):
        r["frequency"] = np.ones(5, np.float32)
    x = matrix(rng.standard_normal((5, 3000)), "f32")
    close(call(x, r), *ref.adjust(values(x), **r), only)


def test_extreme_values():
    """Infinities and NaN of allowed tokens follow the formula; a masked one is -inf whatever it was;
    a row of which nothing is left is -inf throughout."""
    print("extreme values", flush=True)
    rng = np.random.default_rng(2)
    vocab = 600
    for dtype in ("f32", "f16", "bf16"):
        top = torch.finfo(DTYPES[dtype])
        x = rng.standard_normal((4, vocab))
        x[:, ::7] = np.resize([np.nan, np.inf, -np.inf, top.max, top.min, -0.0], x[:, ::7].shape)
        x = matrix(x, dtype)
        r = rules(rng, 4, vocab, 2000, 40, 0.5)
        r["allowed"][1] = False
        r["repetition"][2] = 1.0
        r["bias"][3, ::2] = -np.inf
        close(call(x, r), *ref.adjust(values(x), **r), "extremes", dtype)


def test_extreme_penalties():
    """Repetition penalties whose inverse is none, or no exact one, and infinite others."""
    print("extreme penalties", flush=True)
    by = np.array([1e-39, 2e-45, 1e-30, 2.0 ** -100, 2.0 ** -101, 1e30, 2.0 ** 100, 2.0 ** 127, 3e38, np.inf, 0.0, -2.0,
                   np.nan, 1.0], np.float32)
    rows, vocab = len(by), 400
    x = np.tile(np.array([1e-37, 3e-39, 1.5, 3e38, -1.5, -3e-39, -3e38, 0.0, -0.0, np.inf, -np.inf, np.nan], np.float32), (rows, 40))
    x = matrix(x[:, :vocab], "f32")
    h = np.tile(np.arange(0, vocab, 2, dtype=np.int32), (rows, 1))
    r = {"history": h, "prompts": np.full(rows, 1000, np.int32), "repetition": by}
    close(call(x, r), *ref.adjust(values(x), **r), "penalties")
    r = {"history": h, "presence": by, "frequency": by[::-1].copy()}
    close(call(x, r), *ref.adjust(values(x), **r), "penalties behind the prompt")


@pytest.mark.parametrize("count", [16383, 16384, 16385, 32766, 32767, 32768, 65536, 70001])
def test_counts_of_one_token(count):
    """One token fills a history, behind and in the prompt: every occurrence counts."""
    print("one token", count, flush=True)
    vocab = 9001
    h = np.full((2, count), 8200, np.int32)
    r = {"history": h, "prompts": np.array([0, count - 5], np.int32),
         "frequency": np.array([0.5, 0.5], np.float32), "repetition": np.array([1, 2], np.float32)}
    x = matrix(np.ones((2, vocab)), "f32")
    got = call(x, r).cpu().numpy()
    assert got[0, 8200] == 1 - 0.5 * count and got[1, 8200] == 0.5 - 2.5
    got[:, 8200] = 1
    assert (got == 1).all()


@pytest.mark.parametrize("entries", [1, 2, 511, 512, 513, 65534, 65535, 65536, 70000])
def test_last_entry_of_a_token(entries):
    print("entries", entries, flush=True)
    ids = np.full((1, entries), 8500, np.int32)
    b = np.arange(entries, dtype=np.float32)[None]
    x = torch.zeros(1, 9000, device=DEV)
    got = rs.adjust_logits(x, bias_ids=on(ids), bias=on(b))
    assert got[0, 8500] == entries - 1
    assert (got != 0).sum() == (entries > 1)


@pytest.mark.parametrize("history", [0, 700, 20000])
def test_biases_whose_tokens_share_low_bits(history):
    """Entries of one token and of tokens a power of two apart, in any order."""
    print("biases that collide", history, flush=True)
    rng = np.random.default_rng(history)
    rows, vocab, n = 3, 9000, 512
    ids = (rng.integers(0, 4, (rows, n)) * 1024 + rng.integers(0, 40, (rows, n)) + rng.integers(0, 2, (rows, n)) * 4096).astype(np.int32)
    ids[rng.random((rows, n)) < 0.1] = -1
    r = rules(rng, rows, vocab, history)
    if history:
        r["history"][:, :100] = ids[:, :100]   # tokens with both
    r.update(bias_ids=ids, bias=rng.standard_normal((rows, n)).astype(np.float32))
    x = matrix(rng.standard_normal((rows, vocab)), "f32")
    close(call(x, r), *ref.adjust(values(x), **r), "colliding biases")


def test_strides_of_lists():
    """Lists that are parts of larger buffers, and one list for all rows."""
    print("strides of lists", flush=True)
    rng = np.random.default_rng(12)
    rows, vocab = 6, 5000
    r = rules(rng, rows, vocab, 300, 20, 0.5)
    x = matrix(rng.standard_normal((rows, vocab)), "bf16")
    words = on(ref.mask_words(r["allowed"]))
    want = call(x, r)

    def wide(t):
        whole = torch.full((rows, t.shape[1] + 9), 3, dtype=t.dtype, device=DEV)
        whole[:, 4:4 + t.shape[1]] = t
        return whole[:, 4:4 + t.shape[1]]

    args = {k: on(v) for k, v in r.items() if k not in ("allowed", "prompts")}
    for name in ("history", "bias_ids", "bias"):
        args[name] = wide(args[name])
    got = rs.adjust_logits(x, mask=wide(words), prompt_lengths=on(r["prompts"]), **args)
    assert torch.equal(got, want)
    one = {k: np.repeat(v[:1], rows, 0) for k, v in r.items()}
    want = call(x, one)
    args = {k: on(v) for k, v in one.items() if k not in ("allowed", "prompts")}
    for name in ("history", "bias_ids", "bias"):
        args[name] = args[name][:1].expand(rows, -1)
    got = rs.adjust_logits(x, mask=on(ref.mask_words(one["allowed"][:1])).expand(rows, -1),
                           prompt_lengths=on(one["prompts"]), **args)
    assert torch.equal(got, want)


def test_nothing():
    print("nothing", flush=True)
    x = torch.randn(3, 100, device=DEV)
    assert torch.equal(rs.adjust_logits(x), x)
    assert rs.adjust_logits(x[:0]).shape == (0, 100)
    none = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    f = torch.ones(3, device=DEV)
    got = rs.adjust_logits(x, history=none, repetition=f * 2, presence=f, frequency=f, bias_ids=none,
                           bias=torch.empty(3, 0, device=DEV))
    assert torch.equal(got, x)


def test_replays_of_a_graph():
    """Adjusted, scored, and the history grown, in a graph."""
    print("graph", flush=True)
    rng = np.random.default_rng(4)
    r = rules(rng, 4, 10000, 600, 10, 0.5)
    x = matrix(rng.standard_normal((4, 10000)), "bf16")
    t = {k: on(v) for k, v in r.items() if k not in ("allowed", "prompts")}
    mask, prompts = on(ref.mask_words(r["allowed"])), on(r["prompts"])

    def step():
        y = rs.adjust_logits(x, mask=mask, prompt_lengths=prompts, dtype=torch.float32, **t)
        return y, rs.token_logprobs(y, top_k=3).top_logprobs

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        x.normal_()
        t["history"].copy_(torch.randint(0, 10000, (4, 600), device=DEV))
        t["lengths"].copy_(torch.randint(0, 600, (4,), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        for g, want in zip(got, step()):
            assert torch.equal(g, want)
        torch.cuda.synchronize()
