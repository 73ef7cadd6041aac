"""Rows scored together on the tensor cores: what the first products, every group size and long tables depend on."""
import numpy as np
import pytest
import torch

from mod_reference import bf16
from test_gpu_sparse import Cache, check_select, random_bounds, select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,g,H_KV", [(64, 1, 2), (64, 4, 2), (128, 4, 1), (128, 5, 1), (128, 8, 2), (128, 2, 2)])
def test_the_first_products_take_the_queries_of_the_call(kvc, D, g, H_KV):
    """A sequence of one tile: its product follows the queries' stores at once.  Every row is checked, and calls after
    one another have other queries, so that what an earlier one left is no answer."""
    c = Cache(kvc, [16 * 100], H_KV=H_KV, D=D)
    try:
        codes, units = random_bounds(c, D + g)
        n = -(-10500 // (H_KV * max(g, 4)))   # enough rows for any group size, see rows_together
        rows = [(0, 16 * 100 - 1 - i % 400) for i in range(n)]
        r = np.random.default_rng(g)
        for call in range(6):
            q = bf16(r.standard_normal((n, g * H_KV, D)) * 2).cuda()
            got = select(c, q, rows, 9, 1, 1)
            keep = list(range(call, n, 6))
            check_select(c, q[keep], [rows[i] for i in keep], codes, units, got[keep], 9, 1, 1)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


@pytest.mark.parametrize("D,g", [(128, 4), (64, 5)])
@pytest.mark.parametrize("from_tile", [1, 3, 7])
def test_expired_waits(kvc, monkeypatch, D, g, from_tile):
    """The first wait that runs out ends the call, with no product on its way: before any tile, within a walk, within the
    second walk.  Rows whose lists are not finished list nothing, padding is left as it is, and the next call is right."""
    c = Cache(kvc, [16 * 600, 16 * 550], H_KV=1, D=D, width=700)   # five tiles a walk
    try:
        codes, units = random_bounds(c, g)
        n = -(-10500 // g)
        rows = [(0, 16 * 600 - 1 - i % 500) for i in range(n)] + [(-1, 4)] + [(1, 16 * 550 - 1)] * 4
        q = bf16(np.random.default_rng(g).standard_normal((len(rows), g, D)) * 2).cuda()
        want = select(c, q, rows, 20, 1, 1)
        monkeypatch.setenv("KVC_TEST_STALL", str(from_tile))
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        got = select(c, q, rows, 20, 1, 1)
        end.record()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_TIMEOUT
        assert begin.elapsed_time(end) < 10e3   # one limit of 2 s, another where a warp was a tile ahead
        live = torch.tensor([s >= 0 for s, _ in rows], device="cuda")
        assert torch.all(got[live] == -1) and torch.all(got[~live] == -77)
        monkeypatch.delenv("KVC_TEST_STALL")
        got = select(c, q, rows, 20, 1, 1)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        assert torch.equal(got, want)
        keep = [0, 1, 700, n - 1, n, n + 1, n + 4]
        check_select(c, q[keep], [rows[i] for i in keep], codes, units, got[keep], 20, 1, 1)
    finally:
        c.close()
