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


def test_blocks_that_other_calls_wrote(kvc):
    """Writes by table and copies leave bounds as they were; one row for each block, its last filled place, renews them."""
    c = Cache(kvc, [100, 30], H_KV=2, D=64)
    try:
        slots = c.slots([(0, 0, 100), (1, 0, 30)])
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
        check_bounds(c, slots)
        old = c.bounds.clone()
        r = np.random.default_rng(0)
        new = lambda n: torch.from_numpy(r.standard_normal((n, 2, 64)).astype(np.float32) * 30).bfloat16().cuda()
        # sequence 0: five tokens from position 95 on, which end in a block of their own; sequence 1: one at position 30
        c.kvc.kvc_write_tokens(c.pool, 0, dev(c.table), dev([95, 30]), dev([0, 5, 5]), new(5), new(5))
        c.kvc.kvc_append(c.pool, 0, dev(c.table[1:]), dev([30]), new(1), new(1))
        free = [b for b in range(c.N) if b not in c.table][0]
        c.kvc.kvc_copy_blocks(c.pool, dev([[int(c.table[0, 2]), free]]))
        assert torch.equal(c.bounds, old)
        last = [c.table[0, 5] * 16 + 15, c.table[0, 6] * 16 + 3, c.table[1, 1] * 16 + 14, free * 16 + 15]
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(last))
        check_bounds(c, list(slots) + last)
        assert not torch.equal(c.bounds, old)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()
