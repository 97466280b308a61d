"""The sums behind the log probabilities on the GPU where a loose bound would hide them: rows with
one or a few tokens left, peaked rows, and threads whose reference moves far from zero."""
import numpy as np
import pytest
import torch

import rows_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, close, matrix, numpy_of, same, values

pytestmark = pytest.mark.gpu


def ids32(t):
    return torch.from_numpy(np.asarray(t, np.int64).astype(np.uint32).view(np.int32)).to(DEV)


# A thread takes 16 logits a step, its block 4096: with whole steps of one value each, every thread
# sees the values in turn.  Its reference is the first value while the largest is within 16 powers
# of two of it (11.09 at scale 1), and moves with the third value.  (With 1100 rows none is split.)
STEP = 4096


@pytest.mark.parametrize("far", [0.0, 37.0, 611.0, 9973.0, -9973.0, 99991.0, -99991.0, 499979.0, 700001.0, -700001.0])
def test_terms_of_an_earlier_reference_keep_their_weight(far):
    """Bound.  No term's distance to the largest is over 11.25 (16.3 powers of two), and x and x - m
    are exact.  A term's exponent: the factor a is off by 2 U, so 33 U; d, its own rounding, at
    most 17 U; the move's and the last shift's difference of references 17 U each; two exp2 of 2 U,
    three products and the joins of 30 U: 117 U.  The chains of three steps of 16: 24 U more."""
    print("logprobs reference moves at %g" % far, flush=True)
    x = np.repeat(np.array([[0.0, 11.0, 11.25], [0.0, 10.75, 11.25]]), STEP, axis=1) + far
    rows = matrix(np.tile(x, (550, 1)), "f32")
    assert np.array_equal(values(rows[:2]), x)
    at = np.array([STEP, 2 * STEP + 5])
    got = rs.token_logprobs(rows, ids32(np.tile(at, 550)), top_k=3)
    d = x - x.max(1, keepdims=True)
    s = np.exp(d).sum(1)
    entropy = np.log(s) - (np.exp(d) * d).sum(1) / s
    off = 141 * ref.U
    stats = np.tile(np.stack([x.max(1), s], 1), (550, 1))
    close(got.stats, stats, stats * [0, off], "stats")
    ln_p = d[np.arange(2), at] - np.log(s)
    close(got.logprob, np.tile(ln_p, 550), np.tile(off + 4 * ref.U * (np.abs(ln_p) + 2 * np.log(s)), 550), "logprob")
    close(got.entropy, np.tile(entropy, 550), np.tile(off * 8 + 8 * ref.U * (np.log(s) + 1), 550), "entropy")


LEFT = [(1, "f32", 200), (3, "bf16", 200), (700, "f32", 300), (700, "f16", 300), (9000, "bf16", 300),
        (9000, "f32", 300), (40009, "f32", 40), (70001, "bf16", 12)]


@pytest.mark.parametrize("vocab,dtype,rows", LEFT)
@pytest.mark.parametrize("spread", [4.0, 11.0, 300.0, 3e4])
def test_one_token_left(vocab, dtype, rows, spread):
    """A row with one token left knows its answer: probability 1, no entropy, no gradient, exactly."""
    g = np.random.default_rng(vocab)
    x = np.full((rows, vocab), -np.inf)
    at = g.integers(0, vocab, rows)
    x[np.arange(rows), at] = g.uniform(-spread, spread, rows)
    t = matrix(x, dtype)
    x = values(t)
    for scale in (1.0, 0.7, 3.0):
        print("logprobs one left", vocab, dtype, spread, scale, flush=True)
        c = np.float64(np.float32(scale))
        got = rs.token_logprobs(t, ids32(at), top_k=1, scale=scale)
        same(got.logprob, np.zeros(rows), "logprob")
        same(got.entropy, np.zeros(rows), "entropy")
        same(got.top_logprobs, np.zeros((rows, 1)), "top_logprobs")
        same(got.top_ids, at[:, None], "top_ids")
        same(got.rank, np.zeros(rows), "rank")
        m = x[np.arange(rows), at]
        same(got.stats, np.stack([m, np.ones(rows)], 1), "stats")
        close(got.lse, m * c, 0 * m, "lse")                 # the product, rounded once
        one = torch.full((rows,), 0.7, device=DEV)
        dx = rs.token_logprobs_grad(t, got.stats, ids32(at), dlogprob=one, entropy=got.entropy, dentropy=one,
                                    scale=scale)
        same(dx, np.zeros((rows, vocab)), "dlogits")


@pytest.mark.parametrize("vocab,rows", [(2, 500), (33, 500), (5000, 300), (50021, 40)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_no_probability_is_above_one(vocab, rows, dtype):
    g = np.random.default_rng(vocab + 1)
    x = g.standard_normal((rows, vocab)) * 3
    at = g.integers(0, vocab, rows)
    x[np.arange(rows), at] += g.uniform(0, 60, rows)        # from flat rows to rows of one token
    t = matrix(x, dtype, pad=1)
    for scale in (1.0, 0.3, 2.7):
        print("logprobs at most 1", vocab, dtype, scale, flush=True)
        got = rs.token_logprobs(t, ids32(at), top_k=min(vocab, 8), scale=scale)
        assert (got.stats[:, 1] >= 1).all()
        assert (got.logprob <= 0).all() and (got.top_logprobs <= 0).all()
        assert (got.entropy >= 0).all()
        m = got.stats[:, 0].double() * float(np.float32(scale))
        assert (got.lse.double() >= m - m.abs() * ref.U).all()


@pytest.mark.parametrize("vocab,dtype", [(60, "f32"), (3000, "bf16"), (9000, "f32"), (66000, "f16")])
def test_few_tokens_left(vocab, dtype):
    """Bound.  The largest logit's term is 1 exactly.  Another, w powers of two below it: the factor
    a is off by 2 U, d by its rounding of at most w + 16, the reference's distance by 16, a move by
    w + 32 (the term is then within 16 of the old reference), exp2 twice or, after a move, three
    times 2 U, four products, a join's w and exp2 in each of at most 30 joins that it passes, of
    which only those that it moves in round (at most 5 live logits: 5), the rest exact: U (ln 2 (9 w
    + 64) + 30) of it.  The sum of L terms rounds L - 1 times, in a thread before its reference's
    distance is taken off, and the largest is taken out of it: L + 2 times U s."""
    g = np.random.default_rng(vocab + 2)
    rows = 400
    x = np.full((rows, vocab), -np.inf)
    live = g.integers(2, 7, rows)
    for r in range(rows):
        where = g.choice(vocab, live[r], replace=False) if r % 3 else np.arange(live[r]) + g.integers(0, vocab - 6)
        x[r, where] = g.uniform(-12, 12, live[r])
    t = matrix(x, dtype)
    x = values(t)
    at = x.argmax(1)
    print("logprobs few left", vocab, dtype, flush=True)
    got = rs.token_logprobs(t, ids32(at), top_k=2)
    d = x - x.max(1, keepdims=True)
    e = np.exp(d)
    with np.errstate(invalid="ignore"):
        w = np.where(e > 0, -d / np.log(2), 0.0)
    s = e.sum(1)
    rest = np.where(d < 0, e, 0.0)
    off = ref.U * ((rest * (np.log(2) * (9 * w + 64) + 30)).sum(1) + (live + 2) * s)
    close(got.stats, np.stack([x.max(1), s], 1), np.stack([0 * s, off], 1), "stats")
    close(got.logprob, -np.log(s), off / s + 4 * ref.U * np.log(s), "logprob")
    m = x.max(1)
    close(got.lse, m + np.log(s), off / s + 2 * ref.U * (np.abs(m) + np.log(s)), "lse")


def gradients(x, targets, scale):
    t = matrix(x, "f32")
    x = values(t)
    rows = x.shape[0]
    got = rs.token_logprobs(t, ids32(targets), scale=scale)
    g = np.random.default_rng(rows)
    a, h, q = (g.standard_normal(rows).astype(np.float32) for _ in range(3))
    for a_, h_, q_ in ((a, None, None), (None, None, q), (a, h, q)):
        dev = [None if v is None else torch.from_numpy(v).to(DEV) for v in (a_, h_, q_)]
        dx = rs.token_logprobs_grad(t, got.stats, ids32(targets), dlogprob=dev[0], entropy=got.entropy,
                                    dentropy=dev[1], dlse=dev[2], scale=scale)
        want, bound = ref.logprobs_grad(x, np.asarray(targets), np.float32(scale),
                                        *(None if v is None else v.astype(np.float64) for v in (a_, h_, q_)))
        close(dx, want, bound, "dlogits")


@pytest.mark.parametrize("scale", [2.0 ** -60, 1e-4, 300.0, 1e6, 2.0 ** 60])
@pytest.mark.parametrize("vocab", [50, 9000])
def test_gradient_at_extreme_scales(scale, vocab):
    print("logprobs gradient scale %g vocab %d" % (scale, vocab), flush=True)
    g = np.random.default_rng(25)
    x = g.standard_normal((5, vocab)) * 3
    x[1] += 100.0
    x[2] -= 1000.0
    x[3, ::3] = -np.inf
    gradients(x, [0, 1, 2, 4, vocab - 1], scale)


@pytest.mark.parametrize("far", [1e4, 7.2e5, 7.27e5, 1.5e6, 1e9, 1e35, 3.4e38])
def test_gradient_far_from_zero(far):
    print("logprobs gradient around %g" % far, flush=True)
    g = np.random.default_rng(26)
    step = np.float64(np.spacing(np.float32(far)))
    x = np.round(g.standard_normal((4, 9000)) * max(3.0, 2 * step) / step) * step
    x[0::2] += far
    x[1::2] -= far
    x = np.clip(x, -3.4028234663852886e38, 3.4028234663852886e38)
    x[2, ::4] -= far / 2
    gradients(x, [3, 30, 300, 3000], 1.0)


def test_a_masked_target_has_its_own_term():
    """A target of -inf among other logits: p = 0, but logprob's derivative is c there."""
    print("logprobs gradient of a masked target", flush=True)
    x = np.array([[1.0, -np.inf, 2.0, -np.inf], [-np.inf] * 4])
    t = matrix(x, "f32")
    got = rs.token_logprobs(t, ids32([1, 1]), scale=0.5)
    same(got.logprob, np.array([-np.inf, -np.inf]), "logprob")
    dx = rs.token_logprobs_grad(t, got.stats, ids32([1, 1]), dlogprob=torch.tensor([3.0, 3.0], device=DEV), scale=0.5)
    p = np.exp([0.5, 0, 1.0, 0]) * [1, 0, 1, 0]
    want = np.stack([1.5 * (np.array([0, 1, 0, 0]) - p / p.sum()), np.zeros(4)])
    close(dx, want, np.abs(want) * 64 * ref.U, "dlogits")
