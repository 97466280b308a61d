"""The calls that move rows by index at sizes where their launches or forms change."""
import gc

import pytest
import torch

import sorting_lsd_radix_amd as rs
from rows_helpers import DEV

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
