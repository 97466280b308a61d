"""Tensors and comparisons of the GPU tests of the calls on rows of scores."""
import numpy as np
import torch

import rows_reference as ref

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def matrix(x, dtype, pad=0, shift=0):
    """x as a [rows, cols] view of `dtype` rows that are cols + pad apart, `shift` elements behind
    an allocation's start; what lies around the rows is NaN."""
    rows, cols = x.shape
    whole = torch.full((shift + rows * (cols + pad) + 8,), float("nan"), dtype=DTYPES[dtype], device=DEV)
    t = whole[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x)).to(DEV))
    return t


def values(t):
    """A matrix's values, exactly, in f64."""
    return t.double().cpu().numpy()


def numpy_of(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def close(got, want, bound, what, dtype="f32"):
    """|got - want| <= bound + half a step of the stored type; where want is no number, the same."""
    got = numpy_of(got)
    assert got.shape == want.shape, what
    # a value past the stored type's largest by half a step or more has no nearer one than infinity
    # (three times f32's lowest logit is -1.02e39, f32 ends at 3.4e38)
    top = torch.finfo(DTYPES[dtype])
    want = np.where(np.abs(want) >= top.max * (1 + top.eps / 4), np.copysign(np.inf, want), want)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN in other places"
    odd = ~fine & ~np.isnan(want)
    assert np.array_equal(got[odd], want[odd]), what + ": infinities"
    room = bound + ref.HALF_STEP[dtype] * np.abs(want) * (1 + 2.0 ** -7) + ref.SMALLEST[dtype]
    bad = fine & (np.abs(got - np.where(fine, want, 0)) > np.where(fine, room, 0))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d too far off, the first at %s: %r, not %r (bound %.3g)"
                             % (what, bad.sum(), bad.size, i, got[i], want[i], np.broadcast_to(room, want.shape)[i]))


def same(got, want, what):
    got = numpy_of(got)
    assert got.shape == want.shape, "%s: shape %s, not %s" % (what, got.shape, want.shape)
    bad = got != want
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d differ, the first at %s: %r, not %r"
                             % (what, bad.sum(), bad.size, i, got[i], want[i]))
