"""Calls on the 8-bit cache that its other tests do not make: attentions that run at the
same time, and tables without a column."""

import numpy as np
import pytest
import torch

from cache_utils import dev, make_pool, to_cache
from hstu_sequential_transduction_b200 import ops

pytestmark = pytest.mark.gpu


def test_evict_with_tables_of_no_pages(cuda_device):
    """No room for a cached token: nothing moves; a length says otherwise and is flagged."""
    pool, _, _, _ = make_pool(np.random.default_rng(3), [70], 2, 64)
    cache = to_cache(pool, cuda_device)
    none = torch.zeros(2, 0, dtype=torch.int32, device=cuda_device)
    kw = dict(keep=4, max_cache_len=100)
    ws = ops.alloc_workspace(ops.hstu_cache_evict_workspace_size(cache, none, **kw), cuda_device)
    for lens, flag in (([0, 0], (0, 0)), ([0, 5], (5, 64))):
        table, new_lens, kept = ops.hstu_cache_evict(cache, none, dev(lens, cuda_device, torch.int32), none,
                                                     workspace=ws, **kw)
        assert ops.hstu_check_device_flag(ws) == flag
        assert new_lens.tolist() == lens and kept.tolist() == [[-1] * 4] * 2 and table.shape == (2, 0)
