"""Rows of an embedding table by token, and the table's gradient, against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import moves_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, DTYPES, close, matrix, values

pytestmark = pytest.mark.gpu

# tokens, rows of the table, width, elements between rows, elements before the first
SHAPES = [
    (1, 1, 1, 0, 0), (1, 1000, 64, 0, 0), (4, 300, 4096, 0, 0), (15, 3, 7, 3, 1), (16, 2, 33, 0, 0),
    (17, 1, 40, 0, 0), (33, 50, 513, 1, 3), (100, 1000, 129, 8, 0), (1000, 37, 96, 0, 0), (1500, 5, 20, 2, 1),
    (700, 4000, 48, 0, 0), (64, 65, 2051, 0, 2),
]


def tokens(rng, n, vocab):
    """By a power law; some outside the table."""
    ids = np.minimum(rng.zipf(1.3, n) - 1, vocab - 1).astype(np.int32)
    ids = rng.permutation(vocab).astype(np.int32)[ids]
    out = rng.random(n) < 0.1
    ids[out] = rng.choice([-1, vocab, vocab + 1, 2 ** 31 - 1, -2 ** 31], out.sum())
    return ids


def on(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [1.0, -3.7])
@pytest.mark.parametrize("shape", SHAPES)
def test_embed(shape, scale, dtype):
    print("embed", shape, scale, dtype, flush=True)
    n, vocab, width, pad, shift = shape
    rng = np.random.default_rng(n + width)
    table = matrix(rng.standard_normal((vocab, width)), dtype, pad, shift)
    ids = tokens(rng, n, vocab)
    want, bound = ref.embed(values(table), ids, float(np.float32(scale)))
    got = rs.embed_tokens(table, on(ids), scale=scale)
    assert got.shape == (n, width) and got.dtype == table.dtype
    close(got, want, bound, "rows", dtype)
    whole = torch.full((n, width + 5), 7.0, dtype=table.dtype, device=DEV)
    out = whole[:, :width]
    assert rs.embed_tokens(table, on(ids).view(torch.uint32), scale=scale, out=out) is out
    assert torch.equal(out, got) and (whole[:, width:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_embed_many(scale, dtype):
    """So many rows that a wave takes several vectors of one, with an end off their borders."""
    print("embed many", scale, dtype, flush=True)
    rng = np.random.default_rng(7)
    table = matrix(rng.standard_normal((200, 1003)), dtype, 2, 1)
    ids = tokens(rng, 5000, 200)
    close(rs.embed_tokens(table, on(ids), scale=scale), *ref.embed(values(table), ids, float(np.float32(scale))), "rows", dtype)


@pytest.mark.parametrize("dtype,to", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("scale", [1.0, -3.7])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient(shape, scale, dtype, to):
    print("gradient", shape, scale, dtype, to, flush=True)
    n, vocab, width, pad, shift = shape
    rng = np.random.default_rng(n + width + 1)
    dout = matrix(rng.standard_normal((n, width)), dtype, pad, shift)
    ids = tokens(rng, n, vocab)
    s = float(np.float32(scale))
    want, bound = ref.embed_grad(values(dout), ids, vocab, s)
    got = rs.embed_tokens_grad(dout, on(ids), vocab, scale=scale, dtype=DTYPES[to])
    assert got.shape == (vocab, width) and got.dtype == DTYPES[to]
    close(got, want, bound, "gradient", to)
    assert torch.equal(got, rs.embed_tokens_grad(dout, on(ids), vocab, scale=scale, dtype=DTYPES[to]))
    # into given rows, which others lie between; then added to what they hold
    whole = torch.full((vocab, width + pad), 7.0, dtype=DTYPES[to], device=DEV)
    out = whole[:, :width]
    assert rs.embed_tokens_grad(dout, on(ids), vocab, scale=scale, out=out) is out
    assert torch.equal(out, got) and (whole[:, width:] == 7.0).all()
    old = rng.standard_normal((vocab, width))
    out.copy_(on(old))
    old = values(out)
    want, bound = ref.embed_grad(values(dout), ids, vocab, s, old)
    rs.embed_tokens_grad(dout, on(ids), vocab, scale=scale, out=out, accumulate=True)
    close(out, want, bound, "accumulated", to)
    gone = np.setdiff1d(np.arange(vocab), ids)
    assert np.array_equal(values(out)[gone], old[gone])
    assert (whole[:, width:] == 7.0).all()


@pytest.mark.parametrize("n", [1, 16, 17, 1024, 16384, 16385, 40000])
@pytest.mark.parametrize("kind", ["one", "each", "two", "runs", "outside"])
def test_counts_of_tokens(n, kind):
    """Whole sums of whole numbers, exact in f32: one token, every token once, tokens over borders of
    every size, none at all."""
    print("counts", n, kind, flush=True)
    rng = np.random.default_rng(n)
    vocab = {"one": 70000, "each": n, "two": 3, "runs": n, "outside": 9}[kind]
    ids = {"one": np.full(n, 69999), "each": rng.permutation(n), "two": rng.integers(0, 2, n) * 2,
           "runs": np.repeat(np.arange(n), rng.integers(0, 300, n))[:n] if n > 1 else np.zeros(1, int),
           "outside": np.full(n, -1)}[kind]
    ids = np.resize(ids, n) if len(ids) else np.zeros(n, int)
    ids = rng.permutation(ids).astype(np.int32)
    x = rng.integers(-8, 9, (n, 12)).astype(np.float32)
    want = np.zeros((vocab + 1, 12))
    np.add.at(want, np.where((ids >= 0) & (ids < vocab), ids, vocab), x)
    got = rs.embed_tokens_grad(on(x).bfloat16(), on(ids), vocab, dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy(), want[:vocab])


def test_shapes_of_ids():
    print("shapes of ids", flush=True)
    rng = np.random.default_rng(2)
    table = matrix(rng.standard_normal((50, 24)), "f16")
    ids = on(rng.integers(0, 50, (3, 4, 5)).astype(np.int32))
    rows = rs.embed_tokens(table, ids)
    assert rows.shape == (3, 4, 5, 24)
    assert torch.equal(rows, table[ids.long()])
    flat = rs.embed_tokens_grad(rows.view(60, 24), ids, 50)
    assert torch.equal(flat, rs.embed_tokens_grad(rows, ids, 50))
    assert torch.equal(flat, rs.embed_tokens_grad(rows.view(60, 24), ids.view(-1), 50))
    one = rs.embed_tokens(table, ids[0, 0, 0])
    assert one.shape == (24,) and torch.equal(one, table[ids[0, 0, 0].long()])
    assert torch.equal(rs.embed_tokens_grad(one, ids[0, 0, 0], 50)[ids[0, 0, 0].long()], one)
    wide = torch.zeros(3, 4, 5, 30, dtype=torch.float16, device=DEV)
    wide[..., :24] = rows
    assert torch.equal(flat, rs.embed_tokens_grad(wide[..., :24], ids, 50))   # one stride for all rows
    with pytest.raises(TypeError):
        rs.embed_tokens_grad(torch.zeros(3, 5, 4, 24, device=DEV).transpose(1, 2), ids, 50)


def test_strides():
    """One gradient for all tokens (stride 0), as a sum's; one row for the whole table."""
    print("strides", flush=True)
    rng = np.random.default_rng(4)
    ids = tokens(rng, 300, 40)
    one = matrix(rng.standard_normal((1, 100)), "bf16")
    dout = one.expand(300, 100)
    want, bound = ref.embed_grad(values(dout), ids, 40, 1.0)
    close(rs.embed_tokens_grad(dout, on(ids), 40), want, bound, "gradient", "bf16")
    table = one.expand(40, 100)
    close(rs.embed_tokens(table, on(ids)), *ref.embed(values(table), ids, 1.0), "rows", "bf16")


def test_nothing():
    print("nothing", flush=True)
    ids = torch.empty(0, dtype=torch.int32, device=DEV)
    table = torch.ones(9, 40, device=DEV)
    assert rs.embed_tokens(table, ids).shape == (0, 40)
    assert (rs.embed_tokens_grad(table[:0], ids, 9) == 0).all()
    out = torch.ones(9, 40, device=DEV)
    rs.embed_tokens_grad(table[:0], ids, 9, out=out, accumulate=True)
    assert (out == 1).all()


def test_special_values():
    """A copy keeps every bit; NaN and infinities stay in their own rows."""
    print("special values", flush=True)
    rng = np.random.default_rng(3)
    bits = on(rng.integers(-2 ** 15, 2 ** 15, (60, 70)).astype(np.int16))
    ids = on(rng.integers(0, 60, 200).astype(np.int32))
    for dtype in ("f16", "bf16"):
        assert torch.equal(rs.embed_tokens(bits.view(DTYPES[dtype]), ids).view(torch.int16), bits[ids.long()])
    x = torch.ones(200, 70, device=DEV)
    x[5], x[6, 1] = float("nan"), float("inf")
    g = rs.embed_tokens_grad(x, ids, 60)
    odd = torch.zeros(60, dtype=torch.bool, device=DEV)
    odd[ids[5].long()] = True
    assert torch.isnan(g[odd]).all() and not torch.isnan(g[~odd]).any()
    if ids[5] != ids[6]:
        assert torch.isinf(g[ids[6].long(), 1]) and not torch.isinf(g[ids[6].long(), 0])


def test_offsets_past_32_bits():
    print("large table", flush=True)
    vocab, width = 3000, 1 << 20   # 6 GB of bf16
    table = torch.empty(vocab, width, dtype=torch.bfloat16, device=DEV)
    table.copy_(torch.arange(vocab, device=DEV)[:, None] % 251)
    ids = torch.tensor([0, 2999, 2100, 2047, 2048, 2999, -1], dtype=torch.int32, device=DEV)
    rows = rs.embed_tokens(table, ids)
    want = torch.where(ids >= 0, ids % 251, 0).to(torch.bfloat16)
    assert torch.equal(rows[:, 0], want) and torch.equal(rows[:, -1], want)
    table.fill_(9)
    rs.embed_tokens_grad(rows, ids, vocab, out=table)
    total = torch.zeros(vocab, device=DEV)
    total.index_add_(0, ids[:-1].long(), want[:-1].float())
    assert torch.equal(table[:, 0].float(), total) and torch.equal(table[:, -1].float(), total)


@pytest.mark.parametrize("n", [900, 20000])
def test_replays_of_a_graph(n):
    print("graph", n, flush=True)
    x = torch.randn(n, 72, device=DEV)
    ids = torch.randint(0, 500, (n,), device=DEV).to(torch.int32)
    rs.embed_tokens_grad(x, ids, 500)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rs.embed_tokens_grad(x, ids, 500, scale=2.0)
        rows = rs.embed_tokens(got, ids)
    for i in range(4):
        x.normal_()
        ids.copy_(torch.randint(-1, 500, (n,), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = rs.embed_tokens_grad(x, ids, 500, scale=2.0)
        assert torch.equal(got, want), i
        assert torch.equal(rows, rs.embed_tokens(want, ids))
        torch.cuda.synchronize()


@pytest.mark.parametrize("n,vocab", [(131072, 1000), (131073, 5000), (300000, 1 << 20), (524289, 70000), (2097152, 300), (2097153, 1500)])
def test_many_tokens(n, vocab):
    """Every size of the sort: whole numbers, whose sums are exact in f32."""
    print("many tokens", n, vocab, flush=True)
    rng = np.random.default_rng(n)
    ids = np.minimum(rng.zipf(1.2, n) - 2, vocab).astype(np.int32)   # -1 and `vocab` among them
    x = rng.integers(-8, 9, (n, 3)).astype(np.float32)
    want = np.zeros((vocab + 1, 3))
    np.add.at(want, np.where((ids >= 0) & (ids < vocab), ids, vocab), x)
    got = rs.embed_tokens_grad(on(x).half(), on(ids), vocab, dtype=torch.float32)
    assert np.abs(want).max() < 2 ** 24
    assert np.array_equal(got.cpu().numpy(), want[:vocab])


@pytest.mark.parametrize("vocab,width", [(200000, 300), (1 << 20, 33), (3, 1 << 21)])
def test_large_tables(vocab, width):
    """Rows filled beside the sort, with and without tokens, and behind it."""
    print("large tables", vocab, width, flush=True)
    rng = np.random.default_rng(vocab)
    n = 2000 if width < 1000 else 5
    ids = np.concatenate([rng.integers(0, vocab, n - 3), [0, vocab - 1, -1]]).astype(np.int32)
    x = torch.randint(-8, 9, (n, width), device=DEV).bfloat16()
    got = torch.full((vocab, width), float("nan"), dtype=torch.bfloat16, device=DEV)
    rs.embed_tokens_grad(x, on(ids), vocab, out=got)
    want = torch.zeros(vocab, width, device=DEV)
    want.index_add_(0, on(ids[:-1]).long(), x[:-1].float())
    assert torch.equal(got, want.bfloat16())


@pytest.mark.parametrize("n", [1, 100, 1000, 5000])
@pytest.mark.parametrize("vocab", [7, 1000, 1500, 8000, 8007, 40001, 1 << 21])
@pytest.mark.parametrize("width", [3, 40])
def test_rows_without_tokens(n, vocab, width):
    """Few and many tokens for a table's rows, one to three passes of the sort: every row without one is
    zeros, every other its sum."""
    print("rows without tokens", n, vocab, width, flush=True)
    rng = np.random.default_rng(n + vocab)
    ids = rng.integers(-1, vocab, n).astype(np.int32)
    x = rng.integers(-8, 9, (n, width)).astype(np.float32)
    out = torch.full((vocab, width), float("nan"), dtype=torch.bfloat16, device=DEV)
    rs.embed_tokens_grad(on(x).bfloat16(), on(ids), vocab, out=out)
    want = torch.zeros(vocab + 1, width, device=DEV)
    want.index_add_(0, on(np.where(ids < 0, vocab, ids)).long(), on(x))
    assert torch.equal(out, want[:vocab].bfloat16())


@pytest.mark.parametrize("n", [1025, 2048, 7000, 16384, 16385])
@pytest.mark.parametrize("vocab", [5, 1000, 1025, 3000])
@pytest.mark.parametrize("skew", [0.0, 1.0, 100.0])
def test_tiles_that_count_for_themselves(n, vocab, skew):
    """Several tiles, one and two passes, tokens evenly spread, by a power law, and all the same but a few."""
    print("tiles", n, vocab, skew, flush=True)
    rng = np.random.default_rng(n + vocab)
    law = np.arange(1, vocab + 1, dtype=np.float64) ** -skew
    ids = rng.permutation(vocab)[rng.choice(vocab, n, p=law / law.sum())].astype(np.int32)
    ids[rng.integers(0, n, 5)] = [-1, vocab, 0, vocab - 1, 2]
    x = rng.integers(-8, 9, (n, 6)).astype(np.float32)
    out = torch.full((vocab, 6), float("nan"), dtype=torch.float32, device=DEV)
    rs.embed_tokens_grad(on(x).bfloat16(), on(ids), vocab, out=out)
    want = np.zeros((vocab + 1, 6))
    np.add.at(want, np.where((ids >= 0) & (ids < vocab), ids, vocab), x)
    assert np.array_equal(out.cpu().numpy(), want[:vocab])
