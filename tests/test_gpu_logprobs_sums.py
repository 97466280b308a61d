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
