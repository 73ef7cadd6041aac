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


@pytest.mark.parametrize("D,g,H_KV", [(64, 8, 1), (128, 8, 2), (128, 2, 2), (64, 2, 1), (128, 16, 1)])
def test_every_group_size(kvc, D, g, H_KV):
    """Sizes that have an instance of their own, and one that has not: tiles of rows that end inside sequences, chunks
    and single rows side by side, blocks that end inside tiles, table entries outside the pool."""
    c = Cache(kvc, [16 * 130 + 5, 700, 16 * 700], H_KV=H_KV, D=D, width=900)
    try:
        codes, units = random_bounds(c, g)
        rows = [(0, p) for p in range(2040, 2085)] + [(1, p) for p in range(640, 700, 3)] + [(-1, -1)] * 2
        rows += [(2, p) for p in range(11187, 11200)] + [(1, 5), (0, 2000), (2, 9000)]
        few = len(rows)
        rows += [(2, p) for p in range(1000, 1000 + 10000 // (H_KV * max(g, 4)))]
        q = bf16(np.random.default_rng(2).standard_normal((len(rows), g * H_KV, D)) * 2).cuda()
        for top_k, sink, recent in [(3, 1, 1), (40, 2, 2), (128, 0, 1)]:
            got = select(c, q, rows, top_k, sink, recent)
            check_select(c, q[:few], rows[:few], codes, units, got[:few], top_k, sink, recent)
            check_select(c, q[-3:], rows[-3:], codes, units, got[-3:], top_k, sink, recent)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        c.table[1, 7], c.table[2, 600] = -1, c.N
        got = select(c, q, rows, 40, 1, 1)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        check_select(c, q[:few], rows[:few], codes, units, got[:few], 40, 1, 1)
    finally:
        c.close()


@pytest.mark.parametrize("width", [32768, 32769, 40000])
def test_many_rows_of_tables_of_any_width(kvc, width):
    """The widest table whose rows are scored together, and wider ones, whose rows go alone; long and short sequences."""
    c = Cache(kvc, [2 * 32768, 2 * 300], H_KV=1, D=64, bs=2, width=width)
    try:
        codes, units = random_bounds(c, 5)
        rows = [(0, 2 * 32768 - 1 - i) for i in range(40)] + [(1, 2 * 300 - 1 - i % 300) for i in range(1200)]
        q = bf16(np.random.default_rng(2).standard_normal((len(rows), 4, 64)) * 2).cuda()
        keep = [0, 31, 39, 40, 41, 700, len(rows) - 1]
        for top_k in (50, 128):
            got = select(c, q, rows, top_k, 1, 1)
            check_select(c, q[keep], [rows[i] for i in keep], codes, units, got[keep], top_k, 1, 1)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()
