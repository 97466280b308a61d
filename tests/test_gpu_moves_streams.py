"""Calls that move rows by index and adjust logits, side by side on two streams."""
import pytest
import torch

from test_gpu_moves_calls import calls

pytestmark = pytest.mark.gpu


def test_two_streams_at_once_write_everything():
    """Each call has its own memory, which holds none of the results when the calls begin: what they give
    side by side is all that they give alone."""
    print("two streams, cleared outputs", flush=True)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    made = [[(name, *make()) for name, make in calls(s)] for s in sides]
    torch.cuda.synchronize()

    def results(r):
        return r if isinstance(r, tuple) else (r,)

    alone = []
    for a, b in zip(*made):
        for name, tensors, call in (a, b):
            got = results(call(*tensors))
            torch.cuda.synchronize()
            alone.append([t.clone() for t in got])
            torch.cuda.synchronize()
            given = {t.data_ptr() for t in tensors}
            assert got[0].data_ptr() in given, name   # `out`, which is written again
            for t in got:
                t.fill_(float("nan"))
            torch.cuda.synchronize()
    together = [(name, results(call(*tensors))) for a, b in zip(*made) for name, tensors, call in (a, b)]
    torch.cuda.synchronize()
    for want, (name, got) in zip(alone, together):
        for g, w in zip(got, want):
            assert torch.equal(g, w), name
