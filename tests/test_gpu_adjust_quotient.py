"""The quotient of a positive logit and its repetition penalty, to half a step of f32."""
import numpy as np
import pytest
import torch

import sorting_lsd_radix_amd as rs
from rows_helpers import DEV

pytestmark = pytest.mark.gpu


def quotients(l, by):
    """The adjusted logits l [rows, n] > 0, every one a token of its row's prompt, with penalties by [rows]."""
    rows, n = l.shape
    history = torch.arange(n, dtype=torch.int32, device=DEV).expand(rows, -1)
    prompts = torch.full((rows,), n, dtype=torch.int32, device=DEV)
    return rs.adjust_logits(torch.from_numpy(l).to(DEV), history=history, prompt_lengths=prompts,
                            repetition=torch.from_numpy(by).to(DEV)).cpu().numpy()


def close_to_half_a_step(got, l, by):
    """With y the rounded 1 / r, q the rounded l y and d the rounded l - q r, the result is the rounded q + d y.
    q is off the quotient by 2^-23 of it at most, and y r is 1 to 2^-24, so that what is rounded last
    is off by 2^-47 of the quotient, and by less than that again for d's rounding: less than 2^-22 of a
    step.  Where results are subnormal the step is theirs, and so are q's errors."""
    with np.errstate(over="ignore"):
        want = l.astype(np.float64) / by.astype(np.float64)[:, None]
        step = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64)
    top = float(np.finfo(np.float32).max)
    # between the largest number and half a step above it the larger step of infinity does not count
    step = np.where(np.abs(want) >= 2.0 ** 127, 2.0 ** 104, step)
    large = np.abs(want) >= top + 2.0 ** 103
    assert np.array_equal(got[large], np.copysign(np.inf, want[large]))
    off = np.abs(got.astype(np.float64) - want)
    bad = ~large & ~(off <= 0.5 * step * (1 + 2.0 ** -20))
    assert not bad.any(), "%d of %d, the furthest by %.3f steps" % (bad.sum(), bad.size, (off / step)[bad].max())


@pytest.mark.parametrize("n", [1000, 131072])
def test_usual_penalties(n):
    print("usual penalties", n, flush=True)
    rng = np.random.default_rng(n)
    by = np.concatenate([1 + rng.random(40), [1.0, 1.1, 1.2, 1.3, 1.5, 2.0, 3.0, 0.7, -1.3, np.nextafter(np.float32(2), np.float32(1)),
                                              np.nextafter(np.float32(1), np.float32(2))]]).astype(np.float32)
    l = np.abs(rng.standard_normal((len(by), n)) * 8).astype(np.float32) + np.float32(2.0 ** -30)
    close_to_half_a_step(quotients(l, by), l, by)


def test_all_magnitudes():
    """Logits from 2^-100 on and penalties of any size: subnormal quotients, and those past the largest."""
    print("all magnitudes", flush=True)
    rng = np.random.default_rng(5)
    by = (2.0 ** rng.uniform(-99.9, 99.9, 200) * rng.choice([-1, 1], 200)).astype(np.float32)
    by[:6] = [0.5, 0.25, 2.0 ** -100, 2.0 ** 100, 0.75, 1.0]
    l = (2.0 ** rng.uniform(-100, 127.99, (200, 3000))).astype(np.float32)
    l[:, -1], l[:, -2] = np.finfo(np.float32).max, np.inf
    got = quotients(l, by)
    assert np.array_equal(got[:, -2], np.copysign(np.float32(np.inf), by))
    l, got = np.delete(l, -2, 1), np.delete(got, -2, 1)
    close_to_half_a_step(got, l, by)


def test_outside_the_usual_range():
    """Penalties that are 0, infinite, none or without an exact inverse."""
    print("outside the usual range", flush=True)
    by = np.array([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-39, 2e-45, 2.0 ** -101, 2.0 ** 101, 3e38], np.float32)
    l = np.tile(np.array([2e-45, 1e-39, 1e-30, 1.0, 1.5, 3e38, np.inf], np.float32), (len(by), 1))
    with np.errstate(all="ignore"):
        want = l / by[:, None]
    assert np.array_equal(quotients(l, by), want, equal_nan=True)
