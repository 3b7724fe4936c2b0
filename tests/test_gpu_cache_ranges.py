"""Attention over caches whose lengths, queries or grids leave the usual range: every legal finite
input is within the bound of oracle.attend_bound."""
import numpy as np
import pytest
import torch

from cache_util import DEV, HostCache, check_attend, dev
from post_weight_quantization_12_b200 import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("news,ratio", [(3, 2), (20, 3)])
@pytest.mark.parametrize("over", [1, 2, 15, 1000])
def test_rows_at_positions_past_the_page_table(news, ratio, over):
    """A length past the table: the positions past it are left out, those before it stay where they
    are, also for the rows whose own position lies before the table's end."""
    host = HostCache(4, 2, 16, 64, 8, 64, seed=6)
    table = np.array([[2, 0, 3]], np.int32)
    lengths, starts = np.array([48 + over], np.int32), np.array([0, news], np.int32)
    g = torch.Generator().manual_seed(7)
    q = torch.randn(news, 2 * ratio, 64, generator=g).to(torch.bfloat16)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(table), dev(lengths), dev(starts))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == _lib.GPTQ_INFO_BAD_PAGE
    for i in range(news):
        limit = min(48 + over - news + i + 1, 48)
        check_attend(out[i:i + 1], host, table, [limit], [0, 1], q[i:i + 1], 0.125)
