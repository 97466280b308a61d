"""How the tensor wrappers of the calls on rows of scores treat streams, memory and sizes."""
import numpy as np
import pytest
import torch

import rows_reference as ref
import sorting_lsd_radix_amd as rs
from rows_helpers import DEV, same

pytestmark = pytest.mark.gpu


def busy(stream=None):
    """Some milliseconds of copies on a stream."""
    a = torch.empty(1 << 28, device=DEV)
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        for _ in range(12):
            b.copy_(a)
    return a, b


def test_address_0_is_the_default_stream():
    """An address is of the stream that it names, 0 of the default one: the calls run behind what
    that stream has to do before."""
    print("streams by address", flush=True)
    side = torch.cuda.Stream()
    rs.route_topk(torch.zeros(4, 8, device=DEV), 2)
    for on, address in ((torch.cuda.default_stream(), 0), (side, side.cuda_stream)):
        assert on.cuda_stream == address
        assert rs._run_on(0, address, lambda s: s) == address
        ids = torch.zeros(1000, dtype=torch.int32, device=DEV)
        late = torch.arange(1000, dtype=torch.int32, device=DEV) % 7
        held = busy(on)
        with torch.cuda.stream(on):
            ids.copy_(late)
        got = rs.group_choices(ids, 7, stream=address)
        torch.cuda.synchronize()
        for g, want in zip(got, ref.group(np.arange(1000) % 7, 7, 1)):
            same(g, want, "stream %d" % address)
        del held
