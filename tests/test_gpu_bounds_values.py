"""Block bounds whose keys differ by more than fp32's range of products with the unit."""
import numpy as np
import pytest
import torch

from test_gpu_sparse import Cache, check_bounds, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("large", [float("inf"), float("nan"), 3e38, 1e20, -2e38])
def test_tiny_keys_beside_large_ones(kvc, D, large):
    """A key above zero counts as one unit at least in the upper bound, one below zero in the lower, however small it is
    against the unit."""
    c = Cache(kvc, [16 * 3], H_KV=2, D=D)
    try:
        small = [1e-20, -1e-20, 1e-38, -1e-38, 9.2e-41, -9.2e-41, 0.0, -0.0]   # the smallest bf16, and no key at all
        row = torch.tensor([large] + [small[i % 8] for i in range(D - 1)]).to(torch.bfloat16)
        for place in range(16):
            c.patch(int(c.table[0, 1]), 1, 0, place, row)
            c.patch(int(c.table[0, 2]), 0, 0, place, row if place == 5 else torch.zeros(D, dtype=torch.bfloat16))
        slots = c.slots([(0, 0, 48)])
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
        check_bounds(c, slots)
        codes, _ = c.kvc.kvc_block_bounds_views(c.pool, 0, c.bounds)
        hi, lo = codes[int(c.table[0, 1]), 1].tolist()
        assert hi[1:9] == [1, 0, 1, 0, 1, 0, 0, 0] and lo[1:9] == [0, -1, 0, -1, 0, -1, 0, 0]
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["fp8", "int4"])
def test_tiny_scales_beside_large_ones(kvc, dtype):
    """The same through a quantised pool's scales, whose products with the codes are the keys."""
    c = Cache(kvc, [40], H_KV=2, dtype=dtype)
    try:
        c.scales[0, :, ::2], c.scales[0, :, 1::2] = 1e-30, 1e34
        sc = torch.from_numpy(c.scales).cuda()
        kvc.kvc_pool_set_scales(c.pool, 0, sc[0].contiguous(), sc[1].contiguous())
        slots = c.slots([(0, 0, 40)])
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
        check_bounds(c, slots)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()
