"""The calls that move rows by index at sizes where their launches or forms change."""
import gc

import numpy as np
import pytest
import torch

import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, DTYPES

pytestmark = pytest.mark.gpu


def test_table_past_one_grid():
    """A table of more 16-byte vectors than a grid dimension has work items, filled beside one launch and
    by another: every row without a token is zeros, every other its gradient, at both ends and between."""
    print("66 GB table", flush=True)
    vocab, width = 520, (1 << 26) - 5
    free, _ = torch.cuda.mem_get_info()
    if free < 90 << 30:
        pytest.skip("needs 90 GB of the card's memory")
    ids = torch.tensor([519, 511, 0, 300, 519], dtype=torch.int32, device=DEV)
    x = torch.arange(1, 6, device=DEV, dtype=torch.bfloat16)[:, None].expand(5, width)
    x = x.clone()
    out = torch.full((vocab, width), 7.0, dtype=torch.bfloat16, device=DEV)
    rs.embed_tokens_grad(x, ids, vocab, out=out)
    want = {519: 6.0, 511: 2.0, 0: 3.0, 300: 4.0}
    for v in range(vocab):
        low, high = torch.aminmax(out[v])
        assert float(low) == want.get(v, 0.0) == float(high), v
    del out, x
    gc.collect()
    torch.cuda.empty_cache()


def some_tokens(kind, n, vocab, seed):
    """"law": by a power law; "one": three quarters of them the same; "runs": each some hundred times.  All with a
    twentieth outside the table."""
    rng = np.random.default_rng(seed)
    ids = np.minimum(rng.zipf(1.3, n) - 1, vocab - 1) if kind == "law" else rng.integers(0, max(1, min(vocab, n // 300)), n)
    if kind == "one":
        ids = np.where(rng.random(n) < 0.75, vocab - 1, rng.integers(0, vocab, n))
    ids = rng.permutation(vocab)[ids].astype(np.int32)
    out = rng.random(n) < 0.05
    ids[out] = rng.choice([-1, vocab, 2 ** 31 - 1], out.sum())
    return torch.from_numpy(ids).to(DEV)


# tokens, rows, width, dtype, elements between rows; a wave takes 64 vectors of 16 bytes of 8, 16, 32 or 64 positions
WIDE = [
    (3001, 900, 1031, "bf16", 1), (6000, 70, 515, "f32", 0), (16400, 5000, 2051, "f16", 0), (20003, 100000, 2048, "bf16", 8),
    (16400, 300, 4099, "bf16", 0), (40000, 32003, 1001, "f32", 0), (50021, 3000, 1501, "f32", 3), (140000, 20000, 1040, "f16", 0),
    (524290, 4000, 522, "bf16", 2),
]


@pytest.mark.parametrize("kind", ["law", "one", "runs"])
@pytest.mark.parametrize("shape", WIDE)
def test_wide_rows_of_tokens_in_many_pieces(shape, kind):
    """Whole numbers, whose sums are exact in f32, in rows of several waves: tokens of one piece and of
    hundreds, pieces of every length, every size of the sort; into both types, given and added to."""
    print("wide rows", shape, kind, flush=True)
    n, vocab, width, dtype, pad = shape
    ids = some_tokens(kind, n, vocab, n + vocab)
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randint(-4, 5, (n, width + pad), generator=g, device=DEV, dtype=torch.int8).to(DTYPES[dtype])[:, :width]
    inside = (ids >= 0) & (ids < vocab)
    want = torch.zeros(vocab + 1, width, device=DEV)
    want.index_add_(0, torch.where(inside, ids, vocab).long(), x.float())
    want = want[:vocab] * -2
    assert float(want.abs().max()) < 2 ** 23
    for to in {DTYPES[dtype], torch.float32}:
        whole = torch.full((vocab, width + pad), float("nan"), dtype=to, device=DEV)
        out = whole[:, :width]
        rs.embed_tokens_grad(x, ids, vocab, scale=-2.0, out=out)
        assert torch.equal(out, want.to(to)), to
        old = torch.randint(-100, 101, (vocab, width), generator=g, device=DEV, dtype=torch.int8).to(to)
        out.copy_(old)
        rs.embed_tokens_grad(x, ids, vocab, scale=-2.0, out=out, accumulate=True)
        assert torch.equal(out, (old.float() + want).to(to)), to
        assert whole[:, width:].isnan().all()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("rows,top_k,width,dtype", [(8400, 3, 2051, "bf16"), (9000, 12, 520, "f16"), (5100, 5, 1001, "f32")])
def test_combining_past_the_caches(rows, top_k, width, dtype, weighted):
    """So many rows that they are read around the caches; whole numbers times powers of two, whose sums are exact."""
    print("combine past the caches", rows, top_k, width, dtype, weighted, flush=True)
    assert rows * top_k * width * (4 if dtype == "f32" else 2) > 96 << 20
    g = torch.Generator(device=DEV).manual_seed(rows)
    ids = torch.randint(-1, 40, (rows, top_k), generator=g, device=DEV).int()
    order, place, _, _ = rs.group_choices(ids, 40, align=16)
    y = torch.randint(-4, 5, (order.numel(), width), generator=g, device=DEV, dtype=torch.int8).to(DTYPES[dtype])
    w = 2.0 ** torch.randint(-2, 3, (rows, top_k), generator=g, device=DEV).float() if weighted else None
    y[order < 0] = float("nan")   # padding: not read
    want = torch.zeros(rows, width, device=DEV)
    for j in range(top_k):
        p = place[:, j].long()
        part = torch.where((p >= 0)[:, None], y[p.clamp(min=0)].float(), 0.0)
        want += part if w is None else part * w[:, j:j + 1]
    assert torch.equal(rs.combine_choices(y, place, weights=w), want.to(DTYPES[dtype]))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,width", [(600000, 3000, 24), (20000, 200000, 520)])
def test_replays_of_each_sort(n, vocab, width, accumulate):
    """The gradient of more tokens than its own sort takes, and of few for a large table, in a graph that is
    replayed with other work between: whole numbers, exact."""
    print("replays", n, vocab, width, accumulate, flush=True)
    x = torch.zeros(n, width, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(n, dtype=torch.int32, device=DEV)
    out = torch.zeros(vocab, width, device=DEV)
    size = rs.rs_embed_tokens_grad(rs.RS_ELEM_BF16, None, 0, None, n, vocab, width, 1.0, 0, rs.RS_ELEM_F32, None, 0, None, 0)
    temp = torch.empty(size, dtype=torch.uint8, device=DEV)

    def call():
        rs.embed_tokens_grad(x, ids, vocab, out=out, accumulate=accumulate, temp=temp)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        x.copy_(torch.randint(-8, 9, (n, width), device=DEV))
        ids.copy_(torch.randint(-1, vocab, (n,), device=DEV))
        temp.fill_(255 - i)
        out.fill_(3.0)
        want = torch.full((vocab + 1, width), 3.0 if accumulate else 0.0, device=DEV)
        want.index_add_(0, torch.where(ids < 0, vocab, ids).long(), x.float())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[:vocab]), i
