"""Block bounds, block selection and attention over lists of blocks."""
import numpy as np
import pytest
import torch

import mod_reference
from mod_reference import Mod, attend, bf16, f64, pool_values
from sparse_reference import block_scores, bounds_of, choose

pytestmark = pytest.mark.gpu

DT = {"bf16": 0, "fp8": 1, "int4": 2}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Cache:
    """A pool of random bytes' worth of keys and values, tables of distinct blocks, and sequences of given lengths."""

    def __init__(self, kvc, lens, H_KV=2, D=128, dtype="bf16", bs=16, seed=0, layers=1, layer=0, width=None, size=1.0):
        r = np.random.default_rng(seed)
        self.kvc, self.lens, self.H_KV, self.D, self.dtype, self.bs, self.layer = kvc, lens, H_KV, D, dtype, bs, layer
        need = [-(-n // bs) for n in lens]
        self.N = sum(need) + 3
        width = width or max(1, max(need, default=1))
        ids = r.permutation(self.N).astype(np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.pool = kvc.kvc_pool_create(self.N, bs, layers, H_KV, D, DT[dtype])
        self.scales = None
        if dtype == "bf16":
            x = torch.from_numpy((r.standard_normal(self.N * H_KV * 2 * bs * D) * size).astype(np.float32)).to(torch.bfloat16)
            raw = x.view(torch.uint8).numpy()
        elif dtype == "fp8":
            x = torch.from_numpy((r.standard_normal(self.N * H_KV * 2 * bs * D) * 96).astype(np.float32)).clamp(-448, 448)
            raw = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        else:
            raw = r.integers(0, 256, self.N * H_KV * bs * D, dtype=np.uint8)
        if dtype != "bf16":
            self.scales = (0.5 + r.random((2, H_KV, D))).astype(np.float32) / (96 if dtype == "fp8" else 3)
            sc = torch.from_numpy(self.scales).cuda()
            kvc.kvc_pool_set_scales(self.pool, layer, sc[0].contiguous(), sc[1].contiguous())
        self.pool.bytes_view().view(layers, -1)[layer].copy_(torch.from_numpy(raw))
        self.bounds = kvc.kvc_block_bounds(self.pool)

    def values(self):
        """[N, H_KV, 2, bs, D] fp64: code times scale, one fp32 product."""
        raw = self.pool.bytes_view().cpu().numpy().reshape(self.pool.num_layers, -1)[self.layer]
        v = pool_values(raw, self.dtype, self.N, self.H_KV, self.bs, self.D)
        if self.scales is None:
            return v
        return (v.astype(np.float32) * self.scales.transpose(1, 0, 2)[None, :, :, None]).astype(np.float64)

    def patch(self, block, head, kind, place, row):
        """Overwrite a bf16 row."""
        x = self.pool.bytes_view().view(torch.bfloat16).view(self.pool.num_layers, self.N, self.H_KV, 2, self.bs, self.D)
        x[self.layer, block, head, kind, place] = row.cuda() if isinstance(row, torch.Tensor) else row

    def slots(self, runs):
        """Slot map of tokens start .. end - 1 of sequences."""
        return np.concatenate([[self.table[b, t // self.bs] * self.bs + t % self.bs for t in range(a, z)] for b, a, z in runs]
                              ).astype(np.int32)

    def rows(self, rows):
        """(sequence, position) pairs -> device seq_ids, positions."""
        return dev([s for s, _ in rows]), dev([p for _, p in rows])

    def close(self):
        self.pool.close()


# ------------------------------------------------------------------ bounds
def check_bounds(c, slots, got=None):
    codes, units = (x.cpu().numpy() for x in c.kvc.kvc_block_bounds_views(c.pool, c.layer, c.bounds))
    want_c, want_u = np.zeros_like(codes), np.zeros_like(units)
    fill = {}
    for s in slots:
        if s >= 0:
            fill[int(s) // c.bs] = int(s) % c.bs + 1
    keys = c.values()[:, :, 0]
    for blk, n in fill.items():
        for h in range(c.H_KV):
            want_c[blk, h], want_u[blk, h] = bounds_of(keys[blk, h, :n])
    assert np.array_equal(codes, want_c) and np.array_equal(units, want_u)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp8", 128), ("int4", 128)])
@pytest.mark.parametrize("bs", [1, 5, 16, 64])
def test_bounds(kvc, dtype, D, bs):
    c = Cache(kvc, [300, 0, 17, 64, 1], D=D, dtype=dtype, bs=bs, H_KV=3, layers=3, layer=1)
    try:
        # prompts, a continued one, single tokens, padding between and behind
        slots = np.concatenate([c.slots([(0, 3, 211), (3, 63, 64)]), [-1, -1], c.slots([(2, 0, 17), (4, 0, 1)]), [-1]]).astype(np.int32)
        c.kvc.kvc_update_bounds(c.pool, c.layer, c.bounds, dev(slots))
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        check_bounds(c, slots)
        other = [kvc.kvc_block_bounds_views(c.pool, i, c.bounds)[0] for i in (0, 2)]
        assert not any(x.any() for x in other)
    finally:
        c.close()


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 255, 256, 257, 5000])
def test_bounds_of_many_rows(kvc, rows):
    """Chunk borders of the grid, both chunk sizes."""
    for H_KV in (1, 16):
        c = Cache(kvc, [rows], H_KV=H_KV, D=64)
        try:
            slots = c.slots([(0, 0, rows)])
            c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
            check_bounds(c, slots)
        finally:
            c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("H_KV", [7, 9, 20, 33])
def test_bounds_of_many_heads(kvc, dtype, H_KV):
    """A CTA takes eight heads, the last one of a row of CTAs what is left; decoding rows and a prompt over many blocks."""
    c = Cache(kvc, [700, 33, 1], H_KV=H_KV, dtype=dtype)
    try:
        slots = np.concatenate([c.slots([(0, 0, 700), (1, 32, 33), (2, 0, 1)]), [-1]]).astype(np.int32)
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        check_bounds(c, slots)
    finally:
        c.close()


@pytest.mark.parametrize("H_KV", [1, 2, 3])
def test_bounds_of_rows_that_skip_places(kvc, H_KV):
    """The rows of a block ascend but need not follow one another, and one may come twice: the last counts."""
    c = Cache(kvc, [16 * 3000], H_KV=H_KV, D=64)
    try:
        slots = np.concatenate([b * 16 + np.array([0, 3, 9, 9, 14]) for b in c.table[0]]).astype(np.int32)
        for _ in range(5):
            c.bounds.zero_()
            c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
            check_bounds(c, slots)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


def test_bounds_of_unusual_keys(kvc):
    """Zeros, subnormals, the largest values, infinities, NaN; what stands behind the last token is not read."""
    big = torch.finfo(torch.bfloat16).max
    c = Cache(kvc, [16 * 9], H_KV=1, D=64)
    try:
        t = c.table[0]
        for j, v in enumerate([0.0, 1e-40, -1e-38, 127.0, 127.5, big, float("inf"), float("-inf"), float("nan")]):
            for place in range(16):
                c.patch(int(t[j]), 0, 0, place, 0.0)
            c.patch(int(t[j]), 0, 0, 3, v)
        slots = c.slots([(0, 0, 16 * 8 + 4)])
        for place in range(4, 16):
            c.patch(int(t[8]), 0, 0, place, float("inf"))   # past the last token
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
        check_bounds(c, slots)
        codes, units = kvc.kvc_block_bounds_views(c.pool, 0, c.bounds)
        assert units[int(t[0])].item() == 2.0 ** -100 and units[int(t[6])].item() == 2.0 ** 100
        assert codes[int(t[8]), 0].tolist() == [[127] * 64, [-127] * 64]
    finally:
        c.close()


def test_bounds_hold_every_key(kvc):
    """No product of a query with a key is above its block's bound."""
    c = Cache(kvc, [800], H_KV=2, D=128)
    try:
        slots = c.slots([(0, 0, 800)])
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(slots))
        codes, units = (x.cpu().numpy().astype(np.float64) for x in kvc.kvc_block_bounds_views(c.pool, 0, c.bounds))
        k = c.values()[:, :, 0]
        used = c.table[0]
        hi, lo = codes[used, :, 0] * units[used, :, None], codes[used, :, 1] * units[used, :, None]
        assert np.all(k[used] <= hi[:, :, None]) and np.all(k[used] >= lo[:, :, None])
    finally:
        c.close()


def test_bad_slots_are_recorded(kvc):
    c = Cache(kvc, [40])
    try:
        slots = c.slots([(0, 0, 40)])
        c.kvc.kvc_update_bounds(c.pool, 0, c.bounds, dev(np.concatenate([slots, [c.N * 16, -2]])))
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        check_bounds(c, slots)
    finally:
        c.close()


# ------------------------------------------------------------------ selection
def random_bounds(c, seed, spread=6):
    """Bounds of their own: the selection reads nothing else."""
    r = np.random.default_rng(seed)
    x = np.sort(np.clip(np.rint(r.standard_normal((c.N, c.H_KV, 2, c.D)) * 40), -127, 127), axis=2)[:, :, ::-1]
    u = 2.0 ** r.integers(-spread, spread + 1, (c.N, c.H_KV))
    codes, units = c.kvc.kvc_block_bounds_views(c.pool, c.layer, c.bounds)
    codes.copy_(torch.from_numpy(x.astype(np.int8).copy()))
    units.copy_(torch.from_numpy(u.astype(np.float32)))
    return x.astype(np.int8), u.astype(np.float32)


def select(c, q, rows, top_k, sink, recent, seq=True, **how):
    seqs, pos = c.rows(rows)
    out = torch.full((len(rows), c.H_KV, top_k), -77, dtype=torch.int32, device="cuda")
    c.kvc.kvc_select_blocks(c.pool, c.layer, c.bounds, q, dev(c.table), pos, out, seq_ids=seqs if seq else None, sink=sink,
                            recent=recent, **how)
    return out


def check_select(c, q, rows, codes, units, got, top_k, sink, recent):
    got, q = got.cpu().numpy(), f64(q)
    g = q.shape[1] // c.H_KV
    for i, (s, p) in enumerate(rows):
        if s == -1 or p == -1:
            assert np.all(got[i] == -77)
            continue
        nb = p // c.bs + 1
        ids = c.table[s, :nb]
        ok = (ids >= 0) & (ids < c.N)
        safe = np.where(ok, ids, 0)
        for h in range(c.H_KV):
            score = block_scores(q[i, h * g:(h + 1) * g], codes[safe, h], units[safe, h])
            want = choose(score, ok, top_k, sink, recent)
            assert np.array_equal(got[i, h], want), (i, h, got[i, h], want)


@pytest.mark.parametrize("D,g,H_KV", [(64, 1, 3), (64, 4, 2), (128, 1, 2), (128, 3, 2), (128, 8, 1), (128, 13, 1), (128, 32, 1),
                                      (64, 32, 1)])
@pytest.mark.parametrize("bs", [16, 4])
def test_selection(kvc, D, g, H_KV, bs):
    lens = [1, bs, bs + 1, 37 * bs, 0, 33 * bs - 1, 300 * bs, 700 * bs + 3]
    c = Cache(kvc, lens, D=D, H_KV=H_KV, bs=bs, width=800)
    try:
        codes, units = random_bounds(c, D + g)
        r = np.random.default_rng(1)
        q = bf16(r.standard_normal((len(lens), g * H_KV, D)) * 3).cuda()
        rows = [(b, n - 1) for b, n in enumerate(lens)]
        for top_k, sink, recent in [(1, 0, 1), (2, 1, 1), (8, 2, 3), (33, 1, 1), (299, 0, 5), (800, 3, 2)]:
            got = select(c, q, rows, top_k, sink, recent, seq=False)
            check_select(c, q, rows, codes, units, got, top_k, sink, recent)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


@pytest.mark.parametrize("bs,H_KV,B,n_rows,long", [(16, 8, 64, 64, 300), (4, 4, 97, 90, 1100), (1, 2, 512, 512, 400),
                                                   (4, 8, 33, 33, 2500), (1, 8, 20, 20, 4500)])
def test_selection_of_batches_of_different_lengths(kvc, bs, H_KV, B, n_rows, long):
    """Decoding batches that fill the GPU once or a few times, whose rows are taken in an order of their own: up to `long`
    blocks, equal lengths, one token, padding, positions out of range, rows that are not the sequences in order."""
    r = np.random.default_rng(n_rows + bs)
    lens = [int(n) for n in bs * long * r.random(B) ** 4 + 1]
    lens[:6] = [1, bs, bs + 1, bs * long, bs * long, bs * long - 1]
    c = Cache(kvc, lens, H_KV=H_KV, D=64, bs=bs)
    try:
        codes, units = random_bounds(c, 3)
        order = [int(b) for b in r.permutation(B)[:n_rows]]
        rows = [(b, lens[b] - 1) for b in order]
        rows[3] = rows[n_rows - 1] = (-1, -1)
        rows[5], rows[6] = (order[5], 2 ** 31 - 1), (order[6], -7)
        q = bf16(r.standard_normal((n_rows, 2 * H_KV, 64))).cuda()
        got = select(c, q, rows, 24, 1, 2)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        assert torch.all(got[5:7] == -1)
        fine = [i for i in range(n_rows) if i not in (5, 6)]
        check_select(c, q[fine], [rows[i] for i in fine], codes, units, got[fine], 24, 1, 2)
    finally:
        c.close()


@pytest.mark.parametrize("n_q", [3, 40, 333])
def test_selection_of_chunks_and_padding(kvc, n_q):
    c = Cache(kvc, [2000, 3100, 60], H_KV=2, D=64)
    try:
        codes, units = random_bounds(c, 9)
        rows = [(1, p) for p in range(3100 - n_q, 3100)] + [(-1, -1)] * 3 + [(2, p) for p in range(50, 60)] + [(0, 1999), (-1, 5), (0, -1)]
        q = bf16(np.random.default_rng(2).standard_normal((len(rows), 8, 64))).cuda()
        got = select(c, q, rows, 17, 1, 2)
        check_select(c, q, rows, codes, units, got, 17, 1, 2)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


@pytest.mark.parametrize("D,g,H_KV", [(64, 1, 2), (64, 4, 1), (128, 1, 1), (128, 3, 2), (128, 4, 2), (128, 5, 1), (128, 32, 1),
                                      (64, 17, 1)])
def test_selection_of_long_chunks(kvc, D, g, H_KV):
    """Rows scored together (there are enough of them: most only stand in line, a few of each kind are checked): tiles of
    rows and blocks that end anywhere, several sequences in one tile."""
    c = Cache(kvc, [16 * 130 + 5, 700, 16 * 700], H_KV=H_KV, D=D, width=900)
    try:
        codes, units = random_bounds(c, g)
        rows = [(0, p) for p in range(2040, 2085)] + [(1, p) for p in range(640, 700, 3)] + [(-1, -1)] * 2 + [(2, p) for p in range(11187, 11200)]
        rows += [(1, 5), (0, 2000), (2, 9000)]
        few = len(rows)
        rows += [(2, p) for p in range(1000, 1000 + 10000 // (H_KV * max(g, 4)))]
        q = bf16(np.random.default_rng(2).standard_normal((len(rows), g * H_KV, D)) * 2).cuda()
        for top_k, sink, recent in [(3, 1, 1), (40, 2, 2), (128, 0, 1), (200, 0, 1)]:
            got = select(c, q, rows, top_k, sink, recent)
            check_select(c, q[:few], rows[:few], codes, units, got[:few], top_k, sink, recent)
            check_select(c, q[-3:], rows[-3:], codes, units, got[-3:], top_k, sink, recent)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        c.table[1, 7], c.table[2, 600] = -1, c.N
        got = select(c, q, rows, 40, 1, 1)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        check_select(c, q[:few], rows[:few], codes, units, got[:few], 40, 1, 1)
        rows[3], rows[50] = (7, 3), (1, -9)
        got = select(c, q, rows, 40, 1, 1)
        kvc.kvc_pool_sync_status(c.pool)
        assert torch.all(got[3] == -1) and torch.all(got[50] == -1)
    finally:
        c.close()


@pytest.mark.parametrize("blocks", [4000, 9000, 30000])
def test_chunks_of_very_long_sequences(kvc, blocks):
    """Fewer rows to a tile, and the rows' own kernel where a tile has no room."""
    c = Cache(kvc, [blocks * 2], H_KV=1, D=64, bs=2)
    try:
        codes, units = random_bounds(c, 1)
        rows = [(0, p) for p in range(blocks * 2 - 1100, blocks * 2)]
        q = bf16(np.random.default_rng(2).standard_normal((len(rows), 4, 64)) * 2).cuda()
        got = select(c, q, rows, 100, 1, 1)
        keep = [0, 7, 1099]
        check_select(c, q[keep], [rows[i] for i in keep], codes, units, got[keep], 100, 1, 1)
        alone = torch.cat([select(c, q[i:i + 1], rows[i:i + 1], 100, 1, 1) for i in range(0, len(rows), 25)])
        assert torch.equal(got[::25], alone)
    finally:
        c.close()


@pytest.mark.parametrize("blocks", [1000, 20000])
@pytest.mark.parametrize("n_q", [1, 9, 1100])
def test_equal_scores_go_to_the_lower_block(kvc, blocks, n_q):
    """Few distinct scores: the list's border lies inside a run of equals; also all equal, and all zero."""
    c = Cache(kvc, [blocks * 4], H_KV=1, D=64, bs=4)
    try:
        r = np.random.default_rng(3)
        kinds = np.sort(r.integers(-127, 128, (5, 1, 2, 64)), axis=2)[:, :, ::-1].astype(np.int8)
        for which in (r.integers(0, 5, c.N), np.zeros(c.N, int)):
            codes, units = kinds[which], np.ones((c.N, 1), np.float32)
            cv, uv = kvc.kvc_block_bounds_views(c.pool, 0, c.bounds)
            cv.copy_(torch.from_numpy(codes.copy())), uv.copy_(torch.from_numpy(units))
            for scale in (1.0, 0.0):
                q = bf16(r.standard_normal((n_q, 2, 64)) * scale).cuda()
                rows = [(0, blocks * 4 - 1 - i) for i in range(n_q)]
                keep = list(range(0, n_q, 200)) + [n_q - 1]
                for top_k in (7, 100, 512):
                    got = select(c, q, rows, top_k, 1, 1)
                    check_select(c, q[keep], [rows[i] for i in keep], codes, units, got[keep], top_k, 1, 1)
    finally:
        c.close()


def test_selection_of_unusual_queries(kvc):
    big = float(torch.finfo(torch.bfloat16).max)
    c = Cache(kvc, [16 * 90], H_KV=1, D=64)
    try:
        codes, units = random_bounds(c, 4, spread=100)   # units from 2^-100 to 2^100
        q = bf16(np.random.default_rng(5).standard_normal((7, 2, 64)))
        q[0, 0, 3], q[1, 0, 3], q[2, 1, 3], q[3] = float("nan"), float("inf"), float("-inf"), float("nan")
        q[4, 0, 0], q[5], q[6] = big, q[5] * 1e-38, q[6] * 1e-30
        rows = [(0, 1439)] * 7
        got = select(c, q.cuda(), rows, 20, 1, 1)
        check_select(c, q, rows, codes, units, got, 20, 1, 1)
        got = select(c, q.repeat(200, 1, 1).cuda(), rows * 200, 20, 1, 1)   # scored together
        check_select(c, q.repeat(2, 1, 1), rows * 2, codes, units, got[:14], 20, 1, 1)
        assert torch.equal(got[:7].repeat(200, 1, 1), got)
    finally:
        c.close()


def test_selection_in_error(kvc):
    c = Cache(kvc, [400, 640], H_KV=2, D=64)
    try:
        codes, units = random_bounds(c, 6)
        q = bf16(np.random.default_rng(7).standard_normal((6, 4, 64))).cuda()
        c.table[0, 3], c.table[0, 24], c.table[0, 9] = -1, -1, c.N   # one of them the query's own block
        rows = [(0, 399), (1, 639)] * 3
        got = select(c, q, rows, 12, 1, 1)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        check_select(c, q, rows, codes, units, got, 12, 1, 1)
        for bad in [(2, 5), (-2, 5), (0, -2), (0, 640), (1, 2 ** 31 - 1)]:
            got = select(c, q, [(1, 639), bad] + [(-1, -1)] * 4, 12, 1, 1)
            assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
            assert torch.all(got[1] == -1) and torch.all(got[2:] == -77)
            check_select(c, q[:1], [(1, 639)], codes, units, got[:1], 12, 1, 1)
    finally:
        c.close()


@pytest.mark.parametrize("n_rows", [1, 1100])
@pytest.mark.parametrize("unit", [float("inf"), float("nan"), 3e38, -1.0])
def test_bounds_that_are_none_stay_inside_the_lists(kvc, n_rows, unit):
    """A buffer that was never filled may hold any units: the lists are then of any blocks, but still lists."""
    c = Cache(kvc, [16 * 700], H_KV=2, D=64)
    try:
        codes, units = random_bounds(c, 3)
        kvc.kvc_block_bounds_views(c.pool, 0, c.bounds)[1][:] = unit
        q = bf16(np.random.default_rng(2).standard_normal((n_rows, 8, 64))).cuda()
        rows = [(0, 16 * 700 - 1 - i) for i in range(n_rows)]
        seqs, pos = c.rows(rows)
        for top_k in (5, 60, 128, 400):
            room = torch.full((n_rows + 4, 2, top_k), -77, dtype=torch.int32, device="cuda")
            kvc.kvc_select_blocks(c.pool, 0, c.bounds, q, dev(c.table), pos, room[:n_rows], seq_ids=seqs, sink=1, recent=1)
            torch.cuda.synchronize()
            assert torch.all(room[n_rows:] == -77)
            got = room[:n_rows].cpu().numpy()
            for i in (0, n_rows // 2, n_rows - 1):
                for h in range(2):
                    used = got[i, h][got[i, h] >= 0]
                    assert np.all(np.diff(used) > 0) and np.all(got[i, h][len(used):] == -1)
                    assert used.max() == rows[i][1] // 16 and (unit != unit or used.min() == 0)
    finally:
        c.close()


def test_long_selection(kvc):
    """Hundreds of thousands of blocks in one row, lists of tens of thousands."""
    c = Cache(kvc, [1, 200000 * 1], H_KV=1, D=64, bs=1)
    try:
        codes, units = random_bounds(c, 8)
        q = bf16(np.random.default_rng(9).standard_normal((1, 1, 64))).cuda()
        for top_k in (64, 30001):
            got = select(c, q, [(1, 199999)], top_k, 1, 1)
            check_select(c, q, [(1, 199999)], codes, units, got, top_k, 1, 1)
    finally:
        c.close()


# ------------------------------------------------------------------ attention
def check_attend(c, q, rows, lists, out, lse, scale=None, untouched=7.0):
    vals, q64, out, lse = c.values(), f64(q), f64(out), None if lse is None else f64(lse)
    lists = lists.cpu().numpy()
    H_Q = q64.shape[1]
    g = H_Q // c.H_KV
    weights = "f16" if c.dtype != "bf16" else ("pair" if g <= 16 else "bf16")
    scale = c.D ** -0.5 if scale is None else scale
    for i, (s, p) in enumerate(rows):
        if s == -1 or p == -1:
            assert np.all(out[i] == untouched) and (lse is None or np.all(lse[i] == untouched))
            continue
        for h in range(c.H_KV):
            t = [(c.table[s, j], x) for j in lists[i, h] if 0 <= j <= p // c.bs and 0 <= c.table[s, j] < c.N
                 for x in range(c.bs) if j * c.bs + x <= p]
            blk, place = (np.array([a[k] for a in t], int) for k in (0, 1))
            K, V = vals[blk, h, 0, place][:, None], vals[blk, h, 1, place][:, None]
            ro, rl, to, tl = attend(q64[i, h * g:(h + 1) * g], K, V, p, np.ones(len(t), bool), Mod(), scale, g, kind=c.dtype,
                                    weights=weights)
            got = out[i, h * g:(h + 1) * g]
            assert np.all(np.abs(got - ro) <= to), (i, h, np.max(np.abs(got - ro) / np.maximum(to, 1e-30)))
            if lse is not None:
                gl = lse[i, h * g:(h + 1) * g]
                assert np.array_equal(np.isinf(gl), np.isinf(rl))
                fin = np.isfinite(rl)
                assert np.all(np.abs(gl[fin] - rl[fin]) <= tl[fin])


def random_lists(c, rows, top_k, seed, shuffle=False):
    r = np.random.default_rng(seed)
    lists = np.full((len(rows), c.H_KV, top_k), -1, np.int32)
    for i, (s, p) in enumerate(rows):
        if s < 0 or p < 0:
            continue
        nb = p // c.bs + 1
        for h in range(c.H_KV):
            k = min(top_k, nb)
            pick = np.sort(r.choice(nb, k, replace=False))
            if r.random() < 0.7 and nb - 1 not in pick:
                pick[-1] = nb - 1
            at = np.arange(k) if not shuffle else np.sort(r.choice(top_k, k, replace=False))
            lists[i, h, at] = r.permutation(pick) if shuffle else pick
    return lists


def attend_rows(c, q, rows, lists, seq=True, lse=True, place=False, scale=None, **how):
    seqs, pos = c.rows(rows)
    out = q if place else torch.full_like(q, 7.0)
    l = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    c.kvc.kvc_sparse_attn(c.pool, c.layer, q, dev(c.table), pos, dev(lists) if isinstance(lists, np.ndarray) else lists, out, l,
                          seq_ids=seqs if seq else None, scale=scale, **how)
    return out, l


SHAPES = [("bf16", 64, 1, 2), ("bf16", 64, 4, 2), ("bf16", 64, 12, 1), ("bf16", 64, 32, 1), ("bf16", 128, 1, 3), ("bf16", 128, 4, 2),
          ("bf16", 128, 5, 2), ("bf16", 128, 8, 1), ("bf16", 128, 9, 1), ("bf16", 128, 32, 1), ("fp8", 128, 4, 2), ("fp8", 128, 16, 1),
          ("fp8", 128, 25, 1), ("int4", 128, 1, 2), ("int4", 128, 8, 2), ("int4", 128, 32, 1)]


@pytest.mark.parametrize("dtype,D,g,H_KV", SHAPES)
def test_attention_over_lists(kvc, dtype, D, g, H_KV):
    lens = [1, 16, 17, 40, 0, 333, 700, 1201]
    c = Cache(kvc, lens, D=D, H_KV=H_KV, dtype=dtype, layers=2, layer=1)
    try:
        r = np.random.default_rng(g)
        rows = [(b, n - 1) for b, n in enumerate(lens)]
        for top_k in (1, 2, 7, 40, 100):
            q = bf16(r.standard_normal((len(lens), g * H_KV, D)) * 2).cuda()
            lists = random_lists(c, rows, top_k, top_k, shuffle=top_k == 40)
            out, lse = attend_rows(c, q, rows, lists, seq=False)
            assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
            check_attend(c, q, rows, dev(lists), out, lse)
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("bs", [32, 48, 64, 128])
def test_wide_blocks(kvc, dtype, bs):
    """Blocks of several tiles; the query's own block ends at the query, whole tiles of it past the query."""
    lens = [1, bs, bs + 1, 3 * bs - 17, 900]
    c = Cache(kvc, lens, dtype=dtype, bs=bs)
    try:
        q = bf16(np.random.default_rng(bs).standard_normal((len(lens), 8, 128)) * 2).cuda()
        rows = [(b, n - 1) for b, n in enumerate(lens)]
        for top_k in (2, 9):
            lists = random_lists(c, rows, top_k, 3)
            out, lse = attend_rows(c, q, rows, lists)
            check_attend(c, q, rows, dev(lists), out, lse)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


@pytest.mark.parametrize("dtype,g", [("bf16", 4), ("bf16", 16), ("bf16", 32), ("fp8", 4), ("fp8", 32), ("int4", 8), ("int4", 32)])
@pytest.mark.parametrize("top_k", [70, 129, 300])
def test_long_lists_of_many_rows(kvc, dtype, g, top_k):
    """So many rows that one CTA walks a row's whole list: tens of tiles for every warp, more than it looks up at once."""
    c = Cache(kvc, [16 * 320 + 5, 16 * 200], H_KV=1, dtype=dtype)
    try:
        rows = [(0, p) for p in range(16 * 320 + 5 - 600, 16 * 320 + 5)] + [(1, 3199)] * 100
        q = bf16(np.random.default_rng(top_k).standard_normal((len(rows), g, 128)) * 2).cuda()
        lists = random_lists(c, rows, top_k, top_k, shuffle=top_k == 129)
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        keep = [0, 1, 317, 599, 600, 699]
        check_attend(c, q[keep], [rows[i] for i in keep], dev(lists[keep]), out[keep], lse[keep])
        few, few_l = attend_rows(c, q[keep].contiguous(), [rows[i] for i in keep], lists[keep])   # clusters of CTAs
        check_attend(c, q[keep], [rows[i] for i in keep], dev(lists[keep]), few, few_l)
    finally:
        c.close()


@pytest.mark.parametrize("dtype,D,g", [("bf16", 64, 5), ("bf16", 128, 4), ("bf16", 128, 13), ("bf16", 128, 32), ("fp8", 128, 1),
                                       ("fp8", 128, 16), ("int4", 128, 8), ("int4", 128, 27)])
@pytest.mark.parametrize("top_k", [1, 13, 100])
def test_thousands_of_rows(kvc, dtype, D, g, top_k):
    """Rows for several turns of the whole GPU, whose CTAs have fewer warps; short ones, empty ones and padding among them."""
    c = Cache(kvc, [2600, 33], H_KV=2, D=D, dtype=dtype)
    try:
        rows = [(0, p) for p in range(2600)] + [(1, p) for p in range(33)] + [(-1, 5), (1, -1)]
        q = bf16(np.random.default_rng(top_k).standard_normal((len(rows), 2 * g, D)) * 2).cuda()
        lists = random_lists(c, rows, top_k, 1, shuffle=top_k == 13)
        lists[2000] = -1
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        keep = [0, 1, 15, 16, 17, 511, 1999, 2000, 2001, 2598, 2599, 2600, 2616, 2632, 2633, 2634]
        check_attend(c, q[keep], [rows[i] for i in keep], dev(lists[keep]), out[keep], lse[keep])
        few, few_l = attend_rows(c, q[keep].contiguous(), [rows[i] for i in keep], lists[keep])   # more warps, clusters
        check_attend(c, q[keep], [rows[i] for i in keep], dev(lists[keep]), few, few_l)
    finally:
        c.close()


@pytest.mark.parametrize("dtype,H_KV,B,n_rows,top_k", [("bf16", 8, 64, 64, 40), ("bf16", 4, 97, 90, 7), ("fp8", 2, 512, 512, 9),
                                                       ("int4", 8, 33, 33, 64), ("fp8", 8, 130, 130, 3), ("bf16", 1, 512, 400, 1)])
def test_batches_of_different_lengths(kvc, dtype, H_KV, B, n_rows, top_k):
    """Decoding batches that fill the GPU once or a few times, whose rows are taken in an order of their own: lengths that
    are equal, rising, zero (padding) and wrong, rows that are not the sequences in order, and unused sequences."""
    r = np.random.default_rng(n_rows + top_k)
    lens = [int(n) for n in r.integers(1, 900, B)]
    lens[:6] = [1, 16, 17, 900, 900, 900]
    c = Cache(kvc, lens, H_KV=H_KV, dtype=dtype)
    try:
        order = [int(b) for b in r.permutation(B)[:n_rows]]
        rows = [(b, lens[b] - 1) for b in order]
        rows[3] = rows[n_rows - 1] = (-1, -1)
        q = bf16(r.standard_normal((n_rows, 2 * H_KV, 128)) * 2).cuda()
        lists = random_lists(c, rows, top_k, 2, shuffle=n_rows == 90)
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        check_attend(c, q, rows, dev(lists), out, lse)
        # a row out of range is recorded and sums nothing; the others keep their bits
        seqs, pos = c.rows(rows)
        pos[5], pos[6] = 2 ** 31 - 1, -7
        bad, bad_l = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
        kvc.kvc_sparse_attn(c.pool, 0, q, dev(c.table), pos, dev(lists), bad, bad_l, seq_ids=seqs)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        same = [i for i in range(n_rows) if i not in (5, 6)]
        assert torch.equal(bad[same], out[same]) and torch.equal(bad_l[same], lse[same])
        assert torch.all(bad[5:7] == 0) and torch.all(bad_l[5:7] == -float("inf"))
    finally:
        c.close()


@pytest.mark.parametrize("n_q", [2, 45, 700])
def test_chunks_and_padding(kvc, n_q):
    c = Cache(kvc, [1500, 90], H_KV=2, D=64)
    try:
        rows = [(0, p) for p in range(1500 - n_q, 1500)] + [(-1, 4), (-1, -1)] + [(1, p) for p in range(80, 90)] + [(1, -1)]
        q = bf16(np.random.default_rng(n_q).standard_normal((len(rows), 6, 64)) * 2).cuda()
        lists = random_lists(c, rows, 13, 5)
        lists[-1] = 0
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        check_attend(c, q, rows, dev(lists), out, lse)
        again, _ = attend_rows(c, q.clone(), rows, lists, place=True, lse=False)   # out may be q
        live = torch.tensor([s >= 0 and p >= 0 for s, p in rows], device="cuda")
        assert torch.equal(again[live], out[live]) and torch.equal(again[~live], q[~live])
    finally:
        c.close()


def test_every_block_listed_is_decode_attention(kvc):
    lens = [1000, 37, 16, 2500]
    c = Cache(kvc, lens, H_KV=8)
    try:
        q = bf16(np.random.default_rng(0).standard_normal((4, 32, 128)) * 2).cuda()
        rows = [(b, n - 1) for b, n in enumerate(lens)]
        width = c.table.shape[1]
        lists = np.array([[[j if j * 16 < n else -1 for j in range(width)]] * 8 for n in lens], np.int32)
        out, lse = attend_rows(c, q, rows, lists)
        ref_o, ref_l = torch.empty_like(q), torch.empty((4, 32), device="cuda")
        kvc.kvc_decode_attn_mod(c.pool, 0, q, dev(c.table), dev(lens), ref_o, ref_l,
                                workspace=kvc.kvc_mod_workspace(c.pool, 4, 32, width))
        # the same products; sums joined in another order: one bf16 step where the two straddle a border
        assert torch.all((out.float() - ref_o.float()).abs() <= 2 ** -7 * ref_o.float().abs() + 2 ** -12)
        assert torch.all((lse - ref_l).abs() <= 2 ** -20 * ref_l.abs() + 2 ** -18)
    finally:
        c.close()


def test_a_block_listed_twice_counts_twice_and_odd_entries(kvc):
    c = Cache(kvc, [500, 500], H_KV=1, D=64)
    try:
        q = bf16(np.random.default_rng(0).standard_normal((2, 4, 64)) * 2).cuda()
        rows = [(0, 499), (1, 300)]
        lists = np.array([[[3, 3, -1, 31, 0, -1, 3, 9]], [[-1] * 8]], np.int32)
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        check_attend(c, q, rows, dev(lists), out, lse)
        assert torch.all(out[1] == 0) and torch.all(lse[1] == -float("inf"))
        lists[1] = [[18, 19, 1, 2, -1, -1, -1, 4]]   # 19 begins at position 304, after the query
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        check_attend(c, q, rows, dev(lists), out, lse)
        lists[1] = [[18, -5, 1, 2 ** 30, 2 ** 31 - 1, -1, -1, 4]]
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        check_attend(c, q, rows, dev(lists), out, lse)
        lists[1] = [[18, 2, 1, 0, -1, -1, -1, 4]]
        c.table[1, 2], c.table[1, 18] = -1, c.N
        out, lse = attend_rows(c, q, rows, lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        check_attend(c, q, rows, dev(lists), out, lse)
        for bad in [(2, 5), (-2, 5), (0, -2), (0, 512)]:
            out, lse = attend_rows(c, q, [(0, 499), bad], lists)
            assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
            assert torch.all(out[1] == 0) and torch.all(lse[1] == -float("inf"))
            check_attend(c, q[:1], [(0, 499)], dev(lists[:1]), out[:1], lse[:1])
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_nothing_past_the_query_matters(kvc, dtype):
    """NaN and infinities in the places behind the query, in blocks that are not listed, and in another head."""
    c = Cache(kvc, [200], H_KV=2, dtype=dtype)
    try:
        q = bf16(np.random.default_rng(0).standard_normal((1, 8, 128)) * 2).cuda()
        rows, lists = [(0, 182)], np.array([[[2, 11, -1], [2, 11, -1]]], np.int32)
        want, want_l = attend_rows(c, q, rows, lists)
        raw = c.pool.bytes_view().view(c.N, 2, 2, 16, -1)
        nan = 0x7F   # e4m3: NaN; bf16: 0x7F7F is its largest finite range's end, so write NaN through the values
        blk = torch.from_numpy(c.table[0].astype(np.int64)).cuda()
        if dtype == "bf16":
            x = c.pool.bytes_view().view(torch.bfloat16).view(c.N, 2, 2, 16, 128)
            x[blk[11], :, :, 7:] = float("nan")
            x[blk[12]] = float("inf")
            x[blk[3]] = float("nan")
        else:
            raw[blk[11], :, :, 7:] = nan
            raw[blk[12]], raw[blk[3]] = nan, nan
        out, lse = attend_rows(c, q, rows, lists)
        assert torch.equal(out, want) and torch.equal(lse, want_l)
    finally:
        c.close()


def test_scores_of_minus_infinity_weigh_nothing(kvc):
    """A key whose product is -inf has weight zero, even alone in the tile that a warp reads first."""
    c = Cache(kvc, [65], H_KV=1, D=64)
    try:
        q = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
        c.patch(int(c.table[0, 4]), 0, 0, 0, float("-inf"))
        full = np.array([[[0, 1, 2, 3, 4]]], np.int32)
        out, lse = attend_rows(c, q, [(0, 64)], full)
        want, want_l = attend_rows(c, q, [(0, 64)], np.array([[[0, 1, 2, 3, -1]]], np.int32))
        assert torch.equal(out, want) and torch.equal(lse, want_l)
    finally:
        c.close()


def test_climbing_scores(kvc):
    """Scores that grow from block to block by more than any slack of the running maximum."""
    c = Cache(kvc, [16 * 64], H_KV=1, D=64)
    try:
        q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
        q[:, :, 0] = 1.0
        for j in range(64):
            for place in range(16):
                row = torch.randn(64, generator=torch.Generator().manual_seed(j * 16 + place)).to(torch.bfloat16)
                row[0] = float(j * 16)
                c.patch(int(c.table[0, j]), 0, 0, place, row)
        lists = np.arange(64, dtype=np.int32)[None, None]
        for order in (lists, lists[:, :, ::-1].copy()):
            out, lse = attend_rows(c, q, [(0, 1023)], order, scale=1.0)
            check_attend(c, q, [(0, 1023)], dev(order), out, lse, scale=1.0)
    finally:
        c.close()


def test_runs_do_not_change_a_bit_and_graphs_share_nothing(kvc):
    """Two captured calls replayed side by side, on inputs that change between replays."""
    c = Cache(kvc, [3000] * 6, H_KV=4)
    try:
        r = np.random.default_rng(0)
        rows = [(b, 2999) for b in range(6)]
        lists = [dev(random_lists(c, rows, 60, i)) for i in range(2)]
        seqs, pos = c.rows(rows)
        table = dev(c.table)
        q = [bf16(r.standard_normal((6, 16, 128))).cuda() for _ in range(2)]
        out, lse = [torch.empty_like(x) for x in q], [torch.empty((6, 16), device="cuda") for _ in q]
        graphs = [torch.cuda.CUDAGraph() for _ in q]
        for i in range(2):
            with torch.cuda.graph(graphs[i]):
                kvc.kvc_sparse_attn(c.pool, 0, q[i], table, pos, lists[i], out[i], lse[i], seq_ids=seqs)
        streams = [torch.cuda.Stream() for _ in q]
        for _ in range(10):
            for x in q:
                x.copy_(bf16(r.standard_normal(x.shape)))
            want = [attend_rows(c, q[i], rows, lists[i]) for i in range(2)]
            torch.cuda.synchronize()
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for i in range(2):
                assert torch.equal(out[i], want[i][0]) and torch.equal(lse[i], want[i][1])
    finally:
        c.close()


def test_expired_waits(kvc, monkeypatch):
    c = Cache(kvc, [400])
    try:
        q = bf16(np.random.default_rng(0).standard_normal((1, 8, 128))).cuda()
        lists = np.array([[[0, 5, 24]] * 2], np.int32)
        want, _ = attend_rows(c, q, [(0, 399)], lists)
        monkeypatch.setenv("KVC_TEST_STALL", "1")
        attend_rows(c, q, [(0, 399)], lists)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_TIMEOUT
        monkeypatch.delenv("KVC_TEST_STALL")
        out, _ = attend_rows(c, q, [(0, 399)], lists)
        assert torch.equal(out, want) and kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("fp8", 32), ("int4", 16)])
def test_a_server_of_planned_sparse_steps(kvc, dtype, bs):
    """Prompts, then decode steps in a captured graph: plan, rotary write by slot, bounds, selection, attention.
    The selection keeps enough blocks that leaving the others out must agree with a list made by hand."""
    B, H_Q, H_KV, D, width, top_k, rows = 3, 8, 2, 128, 24, 6, 400
    r = np.random.default_rng(1)
    N = 60
    pool = kvc.kvc_pool_create(N, bs, 1, H_KV, D, DT[dtype])
    c = Cache.__new__(Cache)
    c.kvc, c.pool, c.N, c.bs, c.D, c.H_KV, c.dtype, c.layer, c.scales = kvc, pool, N, bs, D, H_KV, dtype, 0, None
    if dtype != "bf16":
        c.scales = np.full((2, H_KV, D), 0.02 if dtype == "fp8" else 0.5, np.float32)
        sc = torch.from_numpy(c.scales).cuda()
        kvc.kvc_pool_set_scales(pool, 0, sc[0].contiguous(), sc[1].contiguous())
    zeros = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    table, lens, new, stack, count = zeros(B, width), zeros(B), zeros(B), dev(r.permutation(N)), dev([N])
    cu = zeros(B + 1)
    half = D // 2
    rope = kvc.Rope(torch.tensor([10000.0 ** (-i / half) for i in range(half)], device="cuda"),
                    axis_of=torch.tensor([i % 3 for i in range(half)], dtype=torch.uint8, device="cuda"))
    bounds = kvc.kvc_block_bounds(pool)

    class Step:
        def __init__(s, n):
            s.slots, s.pos, s.seq = zeros(n), zeros(n), zeros(n)
            s.axes = zeros(3, n)
            s.qkv = torch.zeros((n, (H_Q + 2 * H_KV) * D), dtype=torch.bfloat16, device="cuda")
            s.q_rot = torch.zeros((n, H_Q, D), dtype=torch.bfloat16, device="cuda")
            s.lists, s.out = zeros(n, H_KV, top_k), torch.full((n, H_Q, D), 7.0, dtype=torch.bfloat16, device="cuda")
            s.lse = torch.full((n, H_Q), 7.0, device="cuda")

        def run(s):
            q, k, v = (x.unflatten(1, (-1, D)) for x in s.qkv.split([H_Q * D, H_KV * D, H_KV * D], 1))
            kvc.kvc_plan_step(pool, table, lens, new, stack, count, lens, count, cu, s.slots, s.pos, s.seq)
            s.axes.copy_(s.pos.expand(3, -1))
            kvc.kvc_rope_write_slots(pool, 0, s.slots, s.axes, q, k, v, s.q_rot, rope)
            kvc.kvc_update_bounds(pool, 0, bounds, s.slots)
            kvc.kvc_select_blocks(pool, 0, bounds, s.q_rot, table, s.pos, s.lists, seq_ids=s.seq, sink=1, recent=1)
            kvc.kvc_sparse_attn(pool, 0, s.q_rot, table, s.pos, s.lists, s.out, s.lse, seq_ids=s.seq)

    def check(s):
        torch.cuda.synchronize()
        assert kvc.kvc_pool_sync_status(pool) == kvc.KVC_OK
        c.table = table.cpu().numpy()
        row_list = list(zip(s.seq.tolist(), s.pos.tolist()))
        vals = c.values()[:, :, 0]
        codes, units = np.zeros((N, H_KV, 2, D), np.int8), np.ones((N, H_KV), np.float32)
        for b, n in enumerate(lens.tolist()):
            for j in range(-(-n // bs)):
                for h in range(H_KV):
                    blk = c.table[b, j]
                    codes[blk, h], units[blk, h] = bounds_of(vals[blk, h, :min(bs, n - j * bs)])
        q64, lists = f64(s.q_rot), s.lists.cpu().numpy()
        g = H_Q // H_KV
        for i, (b, p) in enumerate(row_list):
            if b < 0:
                continue
            ids = c.table[b, :p // bs + 1]
            for h in range(H_KV):
                want = choose(block_scores(q64[i, h * g:(h + 1) * g], codes[ids, h], units[ids, h]), np.ones(len(ids), bool),
                              top_k, 1, 1)
                assert np.array_equal(lists[i, h], want)
        check_attend(c, s.q_rot, row_list, s.lists, s.out, s.lse)

    try:
        first, later = Step(rows), Step(5)
        new.copy_(dev([210, 37, 130]))
        first.qkv.copy_(bf16(r.standard_normal(first.qkv.shape)))
        first.run()
        check(first)
        assert lens.tolist() == [210, 37, 130]
        state = [x.clone() for x in (table, lens, stack, count)]
        new.copy_(lens + 1)
        later.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            later.run()
        for x, y in zip((table, lens, stack, count), state):
            x.copy_(y)
        for step in range(20):
            now = lens.tolist()
            new.copy_(dev([now[0] + 1, now[1] + (2 if step % 3 == 0 else 1), 0 if step == 12 else now[2] + 1 if step < 12 else 0]))
            later.qkv.copy_(bf16(r.standard_normal(later.qkv.shape)))
            later.out.fill_(7.0), later.lse.fill_(7.0)
            graph.replay()
            check(later)
        assert lens.tolist()[2] == 0
    finally:
        pool.close()


# ------------------------------------------------------------------ refusals
def test_refusals(kvc):
    c = Cache(kvc, [100, 50], H_KV=2, D=64)
    odd = Cache(kvc, [30], H_KV=2, D=64, bs=8)
    try:
        q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
        table, pos, lists = dev(c.table), dev([99, 49]), torch.zeros((2, 2, 5), dtype=torch.int32, device="cuda")
        pick = dict(pool=c.pool, layer=0, bounds=c.bounds, q=q, block_tables=table, positions=pos, selected=lists)
        look = dict(pool=c.pool, layer=0, q=q, block_tables=table, positions=pos, selected=lists, out=torch.empty_like(q))
        kvc.kvc_select_blocks(**pick)
        kvc.kvc_sparse_attn(**look)
        status = lambda f, **how: pytest.raises(kvc.KvcError, f, **how).value.status
        for f, good in ((kvc.kvc_select_blocks, pick), (kvc.kvc_sparse_attn, look)):
            for name, bad in [("q", q.float()), ("q", q[:, :, :32]), ("q", q[0]), ("block_tables", table[0]), ("positions", pos[:1]),
                              ("positions", pos.long()), ("selected", lists[:, :1]), ("selected", lists[:1]),
                              ("selected", lists.transpose(1, 2)), ("q", q.transpose(0, 1)), ("q", None)]:
                with pytest.raises(ValueError):
                    f(**{**good, name: bad})
            with pytest.raises(ValueError):   # more rows than sequences, and no sequences named
                f(**{**good, "block_tables": table[:1].contiguous()})
            assert status(f, **{**good, "layer": 1}) == kvc.KVC_ERR_ARG
            wide = torch.zeros((2, 66, 64), dtype=torch.bfloat16, device="cuda")
            assert status(f, **{**good, "q": wide, **({"out": torch.empty_like(wide)} if "out" in good else {})}) == kvc.KVC_ERR_UNSUPPORTED
            uneven = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda")
            assert status(f, **{**good, "q": uneven, **({"out": torch.empty_like(uneven)} if "out" in good else {})}) == kvc.KVC_ERR_ARG
            assert status(f, **{**good, "selected": lists[:, :, :0].contiguous()}) == kvc.KVC_ERR_ARG
            none = {"q": q[:0], "positions": pos[:0], "selected": lists[:0], **({"out": q[:0]} if "out" in good else {})}
            f(**{**good, **none})
        for how in [dict(sink=-1), dict(recent=0), dict(sink=4, recent=2)]:
            assert status(kvc.kvc_select_blocks, **{**pick, **how}) == kvc.KVC_ERR_ARG
        assert status(kvc.kvc_select_blocks, **{**pick, "bounds": c.bounds[:-1]}) == kvc.KVC_ERR_ARG
        assert status(kvc.kvc_update_bounds, pool=c.pool, layer=0, bounds=c.bounds[256:], slots=pos) == kvc.KVC_ERR_ARG
        assert status(kvc.kvc_update_bounds, pool=c.pool, layer=-1, bounds=c.bounds, slots=pos) == kvc.KVC_ERR_ARG
        kvc.kvc_update_bounds(c.pool, 0, c.bounds, pos[:0])
        for scale in (0.0, -1.0, float("nan"), float("inf")):
            assert status(kvc.kvc_sparse_attn, **{**look, "scale": scale}) == kvc.KVC_ERR_ARG
        both = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
        assert status(kvc.kvc_sparse_attn, **{**look, "q": both[:2], "out": both[1:]}) == kvc.KVC_ERR_ARG
        one = dict(pool=odd.pool, layer=0, q=q[:1], block_tables=dev(odd.table), positions=pos[:1] * 0 + 29,
                   selected=lists[:1].clone())
        kvc.kvc_select_blocks(bounds=odd.bounds, **one)
        assert status(kvc.kvc_sparse_attn, out=torch.empty_like(q[:1]), **one) == kvc.KVC_ERR_UNSUPPORTED
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()
        odd.close()
