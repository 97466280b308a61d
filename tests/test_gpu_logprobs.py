"""Log probabilities, entropies, ranks and top alternatives, and their gradient, on the GPU against
the definition in 64 bits, with bounds that count f32's roundings (rows_reference.py)."""
import numpy as np
import pytest
import torch

import rows_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, DTYPES, close, matrix, numpy_of, same, values

pytestmark = pytest.mark.gpu


def ids32(t):
    return torch.from_numpy(np.asarray(t, np.int64).astype(np.uint32).view(np.int32)).to(DEV)


def check(x, targets, k=0, dtype="f32", scale=1.0, pad=0, shift=0, grad=True):
    t = matrix(x, dtype, pad, shift)
    x = values(t)
    rows, vocab = x.shape
    targets = None if targets is None else np.asarray(targets, np.int64)
    tt = None if targets is None else ids32(np.where(targets < 0, 0xFFFFFFFF, targets))
    rt = None if targets is None else np.where(targets < 0, vocab, targets)
    got = rs.token_logprobs(t, tt, top_k=k, scale=scale)
    want, off = ref.logprobs(x, rt, k, np.float32(scale))
    for name in ("rank", "top_ids"):
        if name in want:
            same(getattr(got, name), want[name], name)
    for name in ("stats", "lse", "entropy", "logprob", "top_logprobs"):
        if name in want:
            close(getattr(got, name), want[name], np.broadcast_to(off[name], want[name].shape), name)
    if targets is None:
        assert got.logprob is None and got.rank is None
    if not grad:
        return
    g = np.random.default_rng(vocab)
    a, h, q = (g.standard_normal(rows).astype(np.float32) for _ in range(3))
    sets = [(a, h, None), (None, None, q), (a, None, None), (None, h, q), (a, h, q)]
    if targets is None:
        sets = [(None, h, None), (None, h, q)]
    for a_, h_, q_ in sets[vocab % 2::2]:
        dev = [None if v is None else torch.from_numpy(v).to(DEV) for v in (a_, h_, q_)]
        out = matrix(np.zeros_like(x), dtype, pad, shift)
        rs.token_logprobs_grad(t, got.stats, tt, dlogprob=dev[0], entropy=got.entropy, dentropy=dev[1],
                               dlse=dev[2], scale=scale, out=out)
        dx, bound = ref.logprobs_grad(x, rt, np.float32(scale),
                                      *(None if v is None else v.astype(np.float64) for v in (a_, h_, q_)))
        close(out, dx, bound, "dlogits", dtype)
        around = out.as_strided((rows, vocab + pad), (vocab + pad, 1))[:, vocab:]
        assert torch.isnan(around).all(), "written between the rows"
    return got


VOCABS = [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 31, 63, 64, 65, 100, 255, 256, 257, 511, 513, 1000, 1023, 1025, 2047,
          2048, 2049, 4095, 4097, 8191, 8192, 8193, 10007, 16385, 32000, 32003, 50021, 65536, 65537, 131072, 262147]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_every_size(vocab, dtype):
    g = np.random.default_rng(vocab)
    for i, rows in enumerate((1, 3, 40) if vocab < 20000 else (1, 5)):
        k = min(vocab, (0, 1, 5, 20, 64)[(i + vocab) % 5])
        print("logprobs vocab %d rows %d k %d %s" % (vocab, rows, k, dtype), flush=True)
        x = g.standard_normal((rows, vocab)) * 3
        t = g.integers(-1, vocab, rows)
        t[0] = (0, vocab - 1, vocab // 2)[i]
        check(x, t, k, dtype, scale=(1.0, 0.7, 1.3)[i], pad=(0, 1, 8)[i], shift=(0, 3, 8)[i])


@pytest.mark.parametrize("rows", [2, 7, 17, 100, 300, 1500])
def test_numbers_of_rows(rows):
    for vocab, k, dtype in ((9000, 10, "bf16"), (40009, 64, "f32") if rows < 200 else (300, 64, "f32")):
        print("logprobs rows %d vocab %d k %d" % (rows, vocab, k), flush=True)
        g = np.random.default_rng(rows)
        check(g.standard_normal((rows, vocab)) * 3, g.integers(0, vocab, rows), k, dtype, grad=rows < 200)


@pytest.mark.parametrize("vocab", [40, 700, 5000, 70001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_lowest_index(vocab, dtype):
    g = np.random.default_rng(7)
    x = g.integers(-3, 4, (6, vocab)).astype(np.float64)
    x[1] = 0.0
    x[2] = np.where(np.arange(vocab) % 3, 0.0, -0.0)
    x[3] = -5.0
    x[3, vocab // 2:] = 2.0                        # ties only in the second half
    x[4, -7:] = 9.0
    for k in (1, 7, 20, 40):
        print("logprobs ties vocab %d k %d" % (vocab, k), flush=True)
        check(x, [vocab - 1, vocab // 2, vocab // 2, vocab // 2 + 3, vocab - 3, 0], k, dtype)


@pytest.mark.parametrize("vocab", [50, 3000, 66000])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masks(vocab, dtype):
    g = np.random.default_rng(8)
    lowest = float(torch.finfo(DTYPES[dtype]).min)
    x = g.standard_normal((12, vocab)) * 4
    t = g.integers(0, vocab, 12)
    x[0] = -np.inf                                  # nothing is left
    x[1] = -np.inf
    x[1, vocab - 1] = 3.0                           # one token is left, and is the target
    t[1] = vocab - 1
    x[2] = -np.inf
    x[2, vocab // 3] = -50.0                        # one is left, the target is masked
    t[2] = 0
    x[3] = lowest                                   # the type's lowest value everywhere
    x[4] = lowest
    x[4, 5:9] = [1.0, 2.0, 1.0, -3.0]
    x[5, g.random(vocab) < 0.9] = -np.inf
    x[6, g.random(vocab) < 0.9] = lowest
    x[7] = -np.inf
    x[7, -3:] = lowest                              # lowest values among masked ones
    x[8] = -300.0                                   # far below the sums' first reference
    x[8, 3] = -290.0
    x[9, : vocab // 2] = -np.inf                    # a mask longer than any part of a row
    x[10] = np.where(np.arange(vocab) < vocab // 2, -1000.0, 1000.0)
    x[11, ::2] = -np.inf
    t[9] = 0
    for k, scale in ((5, 1.0), (40, 0.25), (0, 3.0)):
        print("logprobs masks vocab %d k %d scale %g %s" % (vocab, k, scale, dtype), flush=True)
        check(x, t, k, dtype, scale=scale, pad=3, shift=1)


@pytest.mark.parametrize("vocab", [60, 9000])
def test_nan_and_infinity(vocab):
    g = np.random.default_rng(9)
    x = g.standard_normal((8, vocab))
    x[0, 5] = np.nan
    x[1, 6] = np.inf
    x[2] = np.nan
    x[3] = -np.inf
    x[3, 7] = np.nan
    x[4, 10:12] = np.inf
    x[5, 11] = np.nan
    x[6, : vocab // 2] = np.nan
    t = [4, 6, 8, 3, 11, 11, vocab - 1, 2]
    for k in (0, 3, 30, 60):
        print("logprobs NaN vocab %d k %d" % (vocab, k), flush=True)
        check(x, t, k, grad=False)
    # the gradient of a row with NaN or +inf is NaN, of the others as ever
    lt = matrix(x, "f32")
    got = rs.token_logprobs(lt, ids32(t))
    dx = numpy_of(rs.token_logprobs_grad(lt, got.stats, ids32(t), dlogprob=torch.ones(8, device=DEV)))
    assert np.isnan(dx[:7]).all()
    rdx, bound = ref.logprobs_grad(values(lt)[7:], np.array(t[7:]), 1.0, np.ones(1))
    close(torch.from_numpy(dx[7:]).float(), rdx, bound, "dlogits")


def test_peaked_and_crowded_rows():
    """Rows whose best logits sit in one thread's share or in one vector, and rows with far more
    good logits than alternatives: whatever a threshold lets through, the list is exact."""
    g = np.random.default_rng(10)
    vocab = 60000
    x = np.tile(g.standard_normal(vocab), (7, 1))
    x[0, :64] += 50
    x[1, ::2048] += 50
    x[2, 1000:3000] += 50
    x[3] = np.arange(vocab) * 1e-3
    x[4] = -np.arange(vocab) * 1e-3
    x[5, 8::256 * 4] += 30
    x[6, 30000:] = 5.0
    for dtype in ("f32", "bf16"):
        for k in (1, 20, 64):
            print("logprobs peaks k %d %s" % (k, dtype), flush=True)
            check(x, [63, 2048, 1500, 59999, 59999, 8, 45000], k, dtype, grad=False)
            check(np.tile(x, (50, 1)), [1] * 350, k, dtype, grad=False) if k == 20 else None


def test_more_than_2_to_31_logits():
    rows, vocab = 17000, 131072
    print("logprobs %d x %d" % (rows, vocab), flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.empty(rows, vocab, dtype=torch.bfloat16, device=DEV)
    for r in range(0, rows, 1000):
        x[r:r + 1000] = (torch.randn(min(1000, rows - r), vocab, generator=g, device=DEV) * 3).bfloat16()
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV, dtype=torch.int32)
    a = torch.randn(rows, generator=g, device=DEV)
    got = rs.token_logprobs(x, t, top_k=4)
    dx = rs.token_logprobs_grad(x, got.stats, t, dlogprob=a)
    for r in (0, 16383, 16384, rows - 1):
        rt = t[r:r + 1].cpu().numpy().astype(np.int64)
        want, off = ref.logprobs(values(x[r:r + 1]), rt, 4, 1.0)
        same(got.top_ids[r:r + 1], want["top_ids"], "top_ids")
        same(got.rank[r:r + 1], want["rank"], "rank")
        close(got.logprob[r:r + 1], want["logprob"], off["logprob"], "logprob")
        rdx, bound = ref.logprobs_grad(values(x[r:r + 1]), rt, 1.0, values(a[r:r + 1]))
        close(dx[r:r + 1], rdx, bound, "dlogits", "bf16")
    # in place, the same bits
    rs.token_logprobs_grad(x, got.stats, t, dlogprob=a, out=x)
    assert torch.equal(x.view(torch.int16), dx.view(torch.int16))


def test_many_short_rows_and_a_repeated_row():
    print("logprobs 70001 x 40", flush=True)
    g = np.random.default_rng(13)
    check(g.standard_normal((70001, 40)), g.integers(-1, 40, 70001), 3, "f16")
    one = matrix(g.standard_normal((1, 5000)), "f32")
    got = rs.token_logprobs(one.expand(9, 5000), ids32(np.arange(9)), top_k=2)
    want, off = ref.logprobs(np.tile(values(one), (9, 1)), np.arange(9), 2, 1.0)
    same(got.rank, want["rank"], "rank")
    close(got.logprob, want["logprob"], off["logprob"], "logprob")


def test_rows_far_apart_pass_32_bit_offsets():
    stride = (1 << 31) + 8
    print("logprobs rows 2^31 + 8 elements apart", flush=True)
    whole = torch.empty(2 * stride + 5000, dtype=torch.bfloat16, device=DEV)
    x = whole.as_strided((3, 5000), (stride, 1))
    x.copy_(torch.from_numpy(np.random.default_rng(2).standard_normal((3, 5000))).to(DEV))
    t = np.array([0, 7, 4999])
    got = rs.token_logprobs(x, ids32(t), top_k=6)
    want, off = ref.logprobs(values(x), t, 6, 1.0)
    same(got.top_ids, want["top_ids"], "top_ids")
    close(got.logprob, want["logprob"], off["logprob"], "logprob")
    before = values(x)
    rs.token_logprobs_grad(x, got.stats, ids32(t), dlogprob=torch.ones(3, device=DEV), out=x)
    dx, bound = ref.logprobs_grad(before, t, 1.0, np.ones(3))
    close(x, dx, bound, "dlogits", "bf16")


def test_outputs_on_their_own():
    """Through the C ABI: any output left out leaves the others as they are."""
    print("logprobs, outputs left out", flush=True)
    rows, vocab = 6, 9000
    x = matrix(np.random.default_rng(1).standard_normal((rows, vocab)), "f32")
    t = ids32(np.arange(rows))
    full = rs.token_logprobs(x, t, top_k=3)
    need = rs.rs_token_logprobs(0, None, vocab, None, rows, vocab, 1.0, 0, *([None] * 8), 0)
    temp = torch.empty(need, dtype=torch.uint8, device=DEV)
    for left in range(4):
        outs = [torch.full((rows,), 7.0, device=DEV), torch.full((rows,), 7.0, device=DEV),
                torch.full((rows,), 7.0, device=DEV), torch.full((rows,), 7, dtype=torch.int32, device=DEV)]
        stats = torch.empty(rows, 2, device=DEV)
        given = [o if i != left else None for i, o in enumerate(outs)]
        rs.rs_token_logprobs(0, x, vocab, t, rows, vocab, 1.0, 0, stats, *given, None, None, temp, need)
        assert torch.equal(stats, full.stats)
        for i, (o, f) in enumerate(zip(outs, (full.lse, full.entropy, full.logprob, full.rank))):
            assert (o == 7).all() if i == left else torch.equal(o, f)


def test_gradient_against_differences_of_the_forward():
    """h = 2^-5 leaves h^2 / 6 times third derivatives (below 2 for these rows: entropy's are at most
    p (|ln p| + 3)) and the forward's own error of about 40 U over h."""
    print("logprobs differences", flush=True)
    vocab, h = 30, 2.0 ** -5
    x = np.random.default_rng(12).standard_normal((1, vocab))
    steps = matrix(np.concatenate([x + h * np.eye(vocab), x - h * np.eye(vocab)]), "f32")
    t = np.full(2 * vocab, 4)
    o = rs.token_logprobs(steps, ids32(t))
    loss = 0.8 * values(o.logprob[:, None])[:, 0] - 0.6 * values(o.entropy[:, None])[:, 0] + \
        0.3 * values(o.lse[:, None])[:, 0]
    want = (loss[:vocab] - loss[vocab:]) / (2 * h)
    base = matrix(x, "f32")
    b = rs.token_logprobs(base, ids32([4]))
    full = [torch.tensor([v], device=DEV) for v in (0.8, -0.6, 0.3)]
    got = rs.token_logprobs_grad(base, b.stats, ids32([4]), dlogprob=full[0], entropy=b.entropy, dentropy=full[1],
                                 dlse=full[2])
    assert np.abs(numpy_of(got)[0] - want).max() <= 2 * h * h / 6 * 1.7 + 2 * 80 * ref.U / h


@pytest.mark.parametrize("rows,vocab", [(3, 60000), (1100, 3000)])
def test_streams_and_a_replayed_graph(rows, vocab):
    print("logprobs on two streams and in graphs", rows, vocab, flush=True)
    g = np.random.default_rng(14)
    x = matrix(g.standard_normal((rows, vocab)), "bf16")
    y = matrix(g.standard_normal((rows, vocab)), "bf16")
    t = ids32(g.integers(0, vocab, rows))
    a = torch.ones(rows, device=DEV)
    plain = [rs.token_logprobs(v, t, top_k=8, scale=0.9) for v in (x, y)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[rs.token_logprobs(v, t, top_k=8, scale=0.9, stream=st) for v, st in zip((x, y), s)] for _ in range(3)]
    torch.cuda.synchronize()
    for pair in outs:
        for got, want in zip(pair, plain):
            assert all(torch.equal(p, q) for p, q in zip(got, want))
    held, graphs = [], []
    live = x.clone()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = rs.token_logprobs(live, t, top_k=8, scale=0.9)
            d = rs.token_logprobs_grad(live, o.stats, t, dlogprob=a, entropy=o.entropy, dentropy=a, scale=0.9)
        held.append((o, d))
        graphs.append(graph)
    for i in range(4):
        live.copy_((x, y)[i % 2])
        graphs[i // 2].replay()
        torch.cuda.synchronize()
        o, d = held[i // 2]
        want = plain[i % 2]
        assert all(torch.equal(p, q) for p, q in zip(o, want))
        assert torch.equal(d, rs.token_logprobs_grad(live, want.stats, t, dlogprob=a, entropy=want.entropy,
                                                     dentropy=a, scale=0.9))


def test_no_rows_and_refusals():
    x = torch.empty(0, 50, device=DEV)
    got = rs.token_logprobs(x, torch.empty(0, dtype=torch.int32, device=DEV), top_k=3)
    assert got.top_ids.shape == (0, 3) and got.logprob.shape == (0,)
    assert rs.token_logprobs_grad(x, got.stats, dlse=got.lse).shape == (0, 50)
    x = torch.zeros(4, 50, device=DEV)
    t = torch.zeros(4, dtype=torch.int32, device=DEV)
    got = rs.token_logprobs(x, t)
    for bad in (lambda: rs.token_logprobs(x, t.long()), lambda: rs.token_logprobs(x, t[:3]),
                lambda: rs.token_logprobs(x.t()), lambda: rs.token_logprobs(x.double()),
                lambda: rs.token_logprobs_grad(x, got.stats[:, 0], t, dlogprob=got.lse),
                lambda: rs.token_logprobs_grad(x, got.stats, t, dlogprob=got.lse, out=x[:, :49]),
                lambda: rs.token_logprobs_grad(x, got.stats, t, dlogprob=got.lse.half())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(rs.RsError):
        rs.token_logprobs(x, t, top_k=51)
    with pytest.raises(rs.RsError):
        rs.token_logprobs(x, t, scale=0.0)


@pytest.mark.parametrize("scale", [2.0 ** -60, 1e-4, 300.0, 1e6, 2.0 ** 60])
@pytest.mark.parametrize("vocab", [50, 9000])
def test_extreme_scales(scale, vocab):
    print("logprobs scale %g vocab %d" % (scale, vocab), flush=True)
    g = np.random.default_rng(15)
    x = g.standard_normal((5, vocab)) * 3
    x[1] += 100.0
    x[2] -= 1000.0
    x[3, ::3] = -np.inf
    check(x, [0, 1, 2, 4, vocab - 1], 5, "f32", scale=scale, grad=False)


@pytest.mark.parametrize("far", [1e4, 7.2e5, 7.268e5, 7.27e5, 1.4e6, 1.5e6, 1e9, 1e35])
def test_logits_far_from_zero(far):
    """Offsets around every limit at which a sum's reference is taken another way (2^20 and 2^21
    in powers of two are 7.27e5 and 1.45e6); a quarter of the logits lie just past the limit."""
    print("logprobs around %g" % far, flush=True)
    g = np.random.default_rng(16)
    step = np.float64(np.spacing(np.float32(far)))
    x = np.round(g.standard_normal((6, 20000)) * max(3.0, 2 * step) / step) * step
    x[0::2] += far
    x[1::2] -= far
    x[4, ::4] -= far / 2
    x[5, ::4] -= far
    check(x, [3, 30, 300, 3000, 5, 8], 4, "f32", grad=False)


def test_one_long_row():
    vocab = (1 << 28) + 5
    print("logprobs 2 x (2^28 + 5)", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    x = torch.randn(2, vocab, generator=g, device=DEV)
    x[0, -1] = 9.0
    x[1, 1 << 27] = 9.0
    t = ids32([vocab - 1, 1 << 27])
    got = rs.token_logprobs(x, t, top_k=3)
    for r in range(2):
        y = x[r].double()
        lse = torch.logsumexp(y, 0)
        # 2^28 / 64 / 256 terms a thread, and the bound of rows_reference.logprobs at W = 28
        es = ref.U * (vocab / 64 / 256 + 8 + 100 + 3 * (28 + 34))
        assert abs(float(got.lse[r]) - float(lse)) <= es + 4 * ref.U * (abs(float(lse)) + 30)
        assert abs(float(got.logprob[r]) - float(9.0 - lse)) <= es + 4 * ref.U * (float(lse) + 60)
        assert int(got.rank[r]) == 0 and int(got.top_ids[r, 0]) == int(t[r])
        assert got.top_ids[r].tolist() == torch.topk(y, 3).indices.tolist()
        del y


@pytest.mark.parametrize("seed", range(40))
def test_random_combinations(seed):
    g = np.random.default_rng(2000 + seed)
    vocab = int(np.exp(g.uniform(0, np.log(60000))))
    rows = int(g.integers(1, max(2, min(60, 400000 // vocab))))
    k = int(min(vocab, g.integers(0, 65)))
    x = g.standard_normal((rows, vocab)) * (3.0, 0.5, 10.0)[seed % 3]
    if seed % 4 == 0:
        x = np.round(x)                             # ties, past any list of candidates
    if seed % 5 == 0:
        x[g.random(x.shape) < g.choice([0.5, 0.99, 0.9999])] = -np.inf
    if seed % 7 == 0:
        x[:, : vocab // 3] += 30.0                  # the best crowd in front
    t = g.integers(-1, vocab, rows)
    dtype = ("f32", "f16", "bf16")[seed % 3]
    print("logprobs random", seed, rows, vocab, k, dtype, flush=True)
    check(x, t if seed % 6 else None, k, dtype, scale=float(g.choice([1.0, 0.7, 1.5, 0.01])), pad=seed % 9, shift=seed % 5)
