"""Attention with modified scores (kvc_decode_attn_mod, kvc_prefill_attn_mod) against its 64-bit form."""
import numpy as np
import pytest
import torch

from mod_reference import Mod, attend, bf16, f64, pool_values, visible

pytestmark = pytest.mark.gpu

DT = {"bf16": 0, "fp8": 1, "int4": 2}
NAN_BYTE = 0xFF   # bf16 and e4m3 NaN


class Rows:
    """A pool of NaN bytes with `lens` positions of random keys and values per sequence, blocks permuted."""

    def __init__(self, kvc, lens, H_Q=8, H_KV=2, D=128, dtype="bf16", seed=0, layers=2, layer=1, spare=0, sharp=2.0):
        self.kvc, self.lens, self.dtype, self.layer, self.D, self.H_KV, self.H_Q = kvc, lens, dtype, layer, D, H_KV, H_Q
        r = np.random.default_rng(seed)
        self.r = r
        mb = max(1, max(-(-n // 16) for n in lens)) + spare
        need = sum(-(-n // 16) for n in lens)
        self.N = need + 2
        ids = r.permutation(self.N)[:need]
        self.table = np.full((len(lens), mb), -1, np.int32)
        at = 0
        for b, n in enumerate(lens):
            k = -(-n // 16)
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.pool = kvc.kvc_pool_create(self.N, 16, layers, H_KV, D, DT[dtype])
        self.pool.bytes_view().fill_(NAN_BYTE)
        self.scales = np.ones((2, H_KV, D), np.float32)
        if dtype != "bf16":
            self.scales = (0.5 + r.random((2, H_KV, D))).astype(np.float32) * np.float32(0.01 if dtype == "fp8" else 0.4)
            sc = torch.from_numpy(self.scales).cuda()
            kvc.kvc_pool_set_scales(self.pool, layer, sc[0].contiguous(), sc[1].contiguous())
        self.bt = torch.from_numpy(self.table).cuda()
        self.len_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            if n:
                x = bf16(r.standard_normal((2, n, H_KV, D))).cuda()
                kvc.kvc_write_tokens(self.pool, layer, self.bt[b:b + 1].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                                     torch.tensor([0, n], dtype=torch.int32, device="cuda"), x[0].contiguous(), x[1].contiguous(), max_tokens=n)
        torch.cuda.synchronize()
        raw = self.pool.bytes_view().cpu().numpy().reshape(layers, -1)[layer]
        self.stored = pool_values(raw, dtype, self.N, H_KV, 16, D)   # [N, H_KV, 2, 16, D]
        self.q = bf16(r.standard_normal((max(len(lens), 1), H_Q, D)) * sharp).cuda()
        self.scale = D ** -0.5

    def kv(self, b, n):
        """fp64 keys and values [n, H_KV, D] of a row (blocks that are not mapped: NaN)."""
        out = np.full((2, -(-max(n, 1) // 16) * 16, self.H_KV, self.D), np.nan)
        for j in range(-(-n // 16)):
            if self.table[b, j] >= 0:
                x = self.stored[self.table[b, j]]
                for kv in (0, 1):
                    out[kv, 16 * j:16 * j + 16] = np.swapaxes(x[:, kv], 0, 1) * self.scales[kv]
        return out[0, :n], out[1, :n]

    def poke_nan(self, b, t):
        """NaN keys and values at position t of row b (bf16 and e4m3)."""
        view = self.pool.bytes_view().view(self.pool.num_layers, self.N, self.H_KV, 2, 16, -1)
        view[self.layer, int(self.table[b, t // 16]), :, :, t % 16] = NAN_BYTE
        self.stored[self.table[b, t // 16], :, :, t % 16] = np.nan

    def dev_mod(self, m: Mod):
        cu = lambda a, d: None if a is None else torch.from_numpy(np.asarray(a, dtype=d)).cuda()
        return self.kvc.ScoreMod(m.softcap, m.window, m.sink, m.prefix, cu(m.alibi, np.float32), cu(m.doc_start, np.int32))

    def outputs(self, n):
        return (torch.full((n, self.H_Q, self.D), float("nan"), dtype=torch.bfloat16, device="cuda"),
                torch.full((n, self.H_Q), float("nan"), device="cuda"))

    def decode(self, m: Mod, workspace="own", out=None, lse=None):
        n = len(self.lens)
        if out is None:
            out, lse = self.outputs(n)
        ws = self.kvc.kvc_mod_workspace(self.pool, n, self.H_Q, self.table.shape[1]) if isinstance(workspace, str) else workspace
        self.kvc.kvc_decode_attn_mod(self.pool, self.layer, self.q, self.bt, self.len_t, out, lse, mod=self.dev_mod(m),
                                     scale=self.scale, workspace=ws)
        return out, lse

    def prefill(self, m: Mod, q, q_start, row=0, workspace="own"):
        out, lse = self.outputs(q.shape[0])
        ws = (self.kvc.kvc_mod_workspace(self.pool, q.shape[0], self.H_Q, self.table.shape[1])
              if isinstance(workspace, str) else workspace)
        self.kvc.kvc_prefill_attn_mod(self.pool, self.layer, q, self.bt[row].contiguous(), q_start, out, lse,
                                      mod=self.dev_mod(m), scale=self.scale, workspace=ws)
        return out, lse

    def hold(self, out, lse, row, q, K, V, p, see, m, weights):
        ro, rl, to, tl = attend(f64(q), K, V, p, see, m, self.scale, self.H_Q // self.H_KV, self.dtype, weights)
        o, l = f64(out), f64(lse)
        assert np.array_equal(np.isneginf(l), np.isneginf(rl)), (row, l, rl)
        assert np.all(np.abs(o - ro) <= to), (row, float(np.max(np.abs(o - ro) - to)), float(np.max(np.abs(o - ro))))
        f = np.isfinite(rl)
        assert np.all(np.abs(l[f] - rl[f]) <= tl[f]), (row, l[f], rl[f], tl[f])

    def decode_weights(self):
        """The weights' operand type: f16 on e4m3 and int4 pools; on bf16 pools a pair for groups of up to 16 heads,
        one bf16 for larger ones."""
        return "f16" if self.dtype != "bf16" else ("bf16" if self.H_Q // self.H_KV > 16 else "pair")

    def check_decode(self, out, lse, m):
        torch.cuda.synchronize()
        assert self.kvc.kvc_pool_sync_status(self.pool) == self.kvc.KVC_OK
        for b, n in enumerate(self.lens):
            K, V = self.kv(b, n)
            self.hold(out[b], lse[b], b, self.q[b], K, V, n - 1, visible(m, b, n - 1, n), m, self.decode_weights())

    def check_prefill(self, out, lse, m, q, q_start, row=0, some=None):
        torch.cuda.synchronize()
        assert self.kvc.kvc_pool_sync_status(self.pool) == self.kvc.KVC_OK
        n_q = q.shape[0]
        K, V = self.kv(row, q_start + n_q)
        for i in range(n_q) if some is None else some:
            p = q_start + i
            self.hold(out[i], lse[i], i, q[i], K, V, p, visible(m, i, p, q_start + n_q), m,
                      "bf16" if self.dtype == "bf16" else "f16")

    def queries(self, n):
        return bf16(self.r.standard_normal((n, self.H_Q, self.D)) * 2).cuda()

    def close(self):
        self.pool.close()


def slopes(H):
    return np.array([2.0 ** (-8.0 * (i + 1) / H) for i in range(H)])


HEADS = [dict(H_Q=8, H_KV=2, D=64), dict(H_Q=8, H_KV=2), dict(H_Q=4, H_KV=4), dict(H_Q=5, H_KV=1), dict(H_Q=12, H_KV=1),
         dict(H_Q=16, H_KV=1, D=64), dict(H_Q=32, H_KV=1), dict(H_Q=27, H_KV=1, D=64), dict(H_Q=8, H_KV=2, dtype="fp8"),
         dict(H_Q=12, H_KV=1, dtype="fp8"), dict(H_Q=32, H_KV=1, dtype="fp8"), dict(H_Q=8, H_KV=2, dtype="int4"),
         dict(H_Q=16, H_KV=1, dtype="int4"), dict(H_Q=32, H_KV=1, dtype="int4")]
head_ids = ["-".join(f"{k}{v}" for k, v in h.items()) for h in HEADS]
MODS = {"plain": lambda H: Mod(), "cap": lambda H: Mod(softcap=5.0), "alibi": lambda H: Mod(alibi=slopes(H)),
        "window1": lambda H: Mod(window=1), "window17_sink3": lambda H: Mod(window=17, sink=3),
        "window40_sink70_cap_alibi": lambda H: Mod(softcap=20.0, window=40, sink=70, alibi=slopes(H)),
        "prefix30": lambda H: Mod(prefix=30), "window5_prefix18": lambda H: Mod(window=5, prefix=18)}
LENS = [0, 1, 2, 15, 16, 17, 64, 65, 200, 1000]


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("heads", HEADS, ids=head_ids)
def test_decode(kvc, heads, mod):
    c = Rows(kvc, LENS, **heads)
    try:
        m = MODS[mod](c.H_Q)
        c.check_decode(*c.decode(m), m)
    finally:
        c.close()


@pytest.mark.parametrize("heads", [HEADS[1], HEADS[4], HEADS[6], HEADS[8], HEADS[13]], ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
@pytest.mark.parametrize("mod", ["cap", "window40_sink70_cap_alibi"])
def test_decode_long_and_few(kvc, heads, mod):
    """Few long sequences: many splits, merged in the kernel or after it; and the unsplit plan."""
    c = Rows(kvc, [9001, 40, 3000], **heads)
    try:
        m = MODS[mod](c.H_Q)
        ws = kvc.kvc_mod_workspace(c.pool, 3, c.H_Q, c.table.shape[1])
        out, lse = c.decode(m, ws)
        c.check_decode(out, lse, m)
        for _ in range(3):   # the workspace is ready for the next call, and repeats are bit-identical
            o2, l2 = c.decode(m, ws)
            assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert not torch.any(ws[:65536])
        c.check_decode(*c.decode(m, None), m)
    finally:
        c.close()


def test_one_workspace_serves_calls_of_other_shapes(kvc):
    c, d = Rows(kvc, [5000, 4000], H_Q=8, H_KV=2), Rows(kvc, [700] * 40, H_Q=16, H_KV=8, D=64)
    try:
        n = max(kvc.kvc_mod_workspace(x.pool, 40, x.H_Q, x.table.shape[1]).numel() for x in (c, d))
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        m = Mod(softcap=30.0)
        q = c.queries(3)
        first = c.decode(m, ws), d.decode(m, ws), c.prefill(m, q, 4000, workspace=ws)
        for _ in range(2):
            again = c.decode(m, ws), d.decode(m, ws), c.prefill(m, q, 4000, workspace=ws)
            for a, b in zip(first, again):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        c.check_decode(*first[0], m)
        d.check_decode(*first[1], m)
    finally:
        c.close()
        d.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int4"])
def test_decode_blocks_outside_the_window_are_not_looked_at(kvc, dtype):
    """Freed blocks (-1 in the table) between the sinks and the window, NaN in the hidden positions of the blocks
    at the window's edge."""
    n, m = 500, Mod(window=100, sink=3)
    c = Rows(kvc, [n, n], dtype=dtype)
    try:
        lo = n - m.window   # 400: block 25 holds it at its first row; 37 hidden rows are in sink and edge blocks
        c.table[:, 1:lo // 16] = -1
        c.bt.copy_(torch.from_numpy(c.table))
        if dtype != "int4":
            for t in list(range(3, 16)) + list(range(lo // 16 * 16, lo)):
                c.poke_nan(0, t)
        c.check_decode(*c.decode(m), m)
        m = Mod(window=93, sink=3)   # the window starts inside a block
        if dtype != "int4":
            for t in range(400, 407):
                c.poke_nan(0, t)
        c.check_decode(*c.decode(m), m)
    finally:
        c.close()


def test_decode_bad_entries_and_lengths(kvc):
    c = Rows(kvc, [100, 200, 30])
    try:
        m = Mod(softcap=10.0)
        saved = c.bt.clone()
        c.bt[1, 3] = c.N
        out, lse = c.decode(m)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        c.bt.copy_(saved)
        c.len_t[1] = 16 * c.table.shape[1] + 1
        out, lse = c.decode(m)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        assert torch.all(out[1] == 0) and torch.all(lse[1] == -float("inf"))
        c.len_t[1] = -1
        out, lse = c.decode(m)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        c.len_t[1] = 200
        c.check_decode(*c.decode(m), m)
    finally:
        c.close()


PREFILL_MODS = {"plain": lambda H, q0, n: Mod(), "cap": lambda H, q0, n: Mod(softcap=5.0),
                "alibi": lambda H, q0, n: Mod(alibi=slopes(H)), "window1": lambda H, q0, n: Mod(window=1),
                "window33_sink20_cap": lambda H, q0, n: Mod(window=33, sink=20, softcap=8.0),
                "prefix": lambda H, q0, n: Mod(prefix=q0 + max(1, n // 2), alibi=slopes(H)),
                "prefix_past_the_end": lambda H, q0, n: Mod(prefix=10 ** 6),
                "window7_prefix5": lambda H, q0, n: Mod(window=7, prefix=5),
                "documents": lambda H, q0, n: Mod(doc_start=(np.arange(q0, q0 + n) // 29) * 29),
                "documents_window_sink": lambda H, q0, n: Mod(doc_start=(np.arange(q0, q0 + n) // 61) * 61, window=9, sink=5),
                "documents_with_empty_rows": lambda H, q0, n: Mod(
                    doc_start=np.where(np.arange(n) % 5 == 2, q0 + n + 3, np.arange(q0, q0 + n) - 40), softcap=9.0)}
CHUNKS = [(0, 1), (37, 1), (0, 5), (100, 33), (13, 150), (1, 64)]


@pytest.mark.parametrize("mod", PREFILL_MODS)
@pytest.mark.parametrize("heads", HEADS, ids=head_ids)
def test_prefill(kvc, heads, mod):
    total = max(a + b for a, b in CHUNKS)
    c = Rows(kvc, [total], **heads)
    try:
        for q_start, n_q in CHUNKS:
            m = PREFILL_MODS[mod](c.H_Q, q_start, n_q)
            q = c.queries(n_q)
            c.check_prefill(*c.prefill(m, q, q_start), m, q, q_start)
    finally:
        c.close()


@pytest.mark.parametrize("heads", [HEADS[0], HEADS[1], HEADS[2], HEADS[6], HEADS[8], HEADS[11]],
                         ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
@pytest.mark.parametrize("mod", ["cap", "window33_sink20_cap", "prefix", "documents"])
def test_prefill_long(kvc, heads, mod):
    c = Rows(kvc, [3100], **heads)
    try:
        for q_start, n_q in ((3000, 4), (2000, 300), (0, 700)):
            m = PREFILL_MODS[mod](c.H_Q, q_start, n_q)
            q = c.queries(n_q)
            out, lse = c.prefill(m, q, q_start)
            some = sorted({0, 1, n_q // 3, n_q // 2, n_q - 2, n_q - 1} & set(range(n_q)))
            c.check_prefill(out, lse, m, q, q_start, some=some)
            o2, l2 = c.prefill(m, q, q_start)
            assert torch.equal(out, o2) and torch.equal(lse, l2)
    finally:
        c.close()


LONG_MODS = {"plain": lambda H, q0, n: Mod(), "cap": lambda H, q0, n: Mod(softcap=5.0), "alibi": lambda H, q0, n: Mod(alibi=slopes(H)),
             "cap_alibi": lambda H, q0, n: Mod(softcap=20.0, alibi=slopes(H)), "cap_past_the_fixed_reference": lambda H, q0, n: Mod(softcap=90.0),
             "cap_window_sink": lambda H, q0, n: Mod(softcap=20.0, window=1500, sink=70),
             "cap_documents": lambda H, q0, n: Mod(softcap=20.0, doc_start=(np.arange(q0, q0 + n) // 1501) * 1501)}


@pytest.mark.parametrize("heads", [dict(H_Q=32, H_KV=8), dict(H_Q=32, H_KV=8, D=64), dict(H_Q=32, H_KV=8, dtype="fp8"),
                                   dict(H_Q=32, H_KV=8, dtype="int4")], ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
@pytest.mark.parametrize("mod", LONG_MODS)
def test_prefill_many_tiles(kvc, heads, mod):
    """Chunks with tens of tiles for every SM: units cut across SMs and the code for long calls."""
    c = Rows(kvc, [3300], **heads)
    try:
        for q_start, n_q in ((2100, 1200), (0, 2500)):
            m = LONG_MODS[mod](c.H_Q, q_start, n_q)
            q = c.queries(n_q)
            out, lse = c.prefill(m, q, q_start)
            c.check_prefill(out, lse, m, q, q_start, some=[0, 1, 63, 64, n_q // 2, n_q - 100, n_q - 1])
            o2, l2 = c.prefill(m, q, q_start)
            assert torch.equal(out, o2) and torch.equal(lse, l2)
    finally:
        c.close()


@pytest.mark.parametrize("D", [64, 128])
def test_one_key_read_in_a_long_call(kvc, D):
    """As test_one_key_read_gives_its_value, with documents of one position, on the code for long calls."""
    n_q, q_start = 2048, 1000
    c = Rows(kvc, [q_start + n_q], H_Q=32, H_KV=8, D=D)
    try:
        m = Mod(softcap=50.0, doc_start=np.arange(q_start, q_start + n_q))
        out, lse = c.prefill(m, c.queries(n_q), q_start)
        torch.cuda.synchronize()
        assert np.array_equal(f64(out), np.repeat(c.kv(0, q_start + n_q)[1][q_start:], 4, axis=1))
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_prefill_hidden_positions_may_hold_nan(kvc, dtype):
    """Positions that no query reads (behind the window, past the row's end, freed blocks) may hold anything."""
    c = Rows(kvc, [400], dtype=dtype, spare=3)
    try:
        m = Mod(window=50, sink=2)
        q_start, n_q = 300, 37
        for t in list(range(2, 16)) + list(range(240, 251)) + list(range(q_start + n_q, 340)):
            c.poke_nan(0, t)
        c.table[0, 1:15] = -1
        c.bt.copy_(torch.from_numpy(c.table))
        q = c.queries(n_q)
        c.check_prefill(*c.prefill(m, q, q_start), m, q, q_start)
    finally:
        c.close()


@pytest.mark.parametrize("heads", [HEADS[1], HEADS[6], HEADS[8], HEADS[11]], ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
@pytest.mark.parametrize("mod", ["cap", "window33_sink20_cap", "prefix", "documents_with_empty_rows"])
def test_warp_level_kernels(kvc, monkeypatch, heads, mod):
    """KVC_TC=0: chunks and large decode groups on the split kernel, with and without a workspace."""
    monkeypatch.setenv("KVC_TC", "0")
    c = Rows(kvc, [1500, 40], **heads)
    try:
        for q_start, n_q in ((1400, 70), (0, 1), (13, 150)):
            m = PREFILL_MODS[mod](c.H_Q, q_start, n_q)
            q = c.queries(n_q)
            some = sorted({0, n_q // 2, n_q - 1})
            c.check_prefill(*c.prefill(m, q, q_start), m, q, q_start, some=some)
            c.check_prefill(*c.prefill(m, q, q_start, workspace=None), m, q, q_start, some=some)
        m = Mod(softcap=9.0, window=300, sink=4)
        c.check_decode(*c.decode(m), m)
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int4"])
def test_more_units_than_one_launch_takes(kvc, dtype):
    """A chunk of 17 000 queries of 32 heads on one KV head (2 125 units of 8 positions), and 2 100 sequences."""
    n = 17000
    c = Rows(kvc, [n], H_Q=32, H_KV=1, dtype=dtype)
    try:
        doc = (np.arange(n) // 700) * 700
        q = c.queries(n)
        for m in (Mod(window=40, sink=3, softcap=9.0), Mod(doc_start=doc, window=50)):
            out, lse = c.prefill(m, q, 0)
            c.check_prefill(out, lse, m, q, 0, some=[0, 39, 40, 8000, 16383, 16384, 16391, n - 1])
    finally:
        c.close()
    d = Rows(kvc, [1 + (7 * i) % 90 for i in range(2100)], H_Q=32, H_KV=1, dtype=dtype)
    try:
        m = Mod(softcap=9.0, window=60)
        out, lse = d.decode(m)
        torch.cuda.synchronize()
        for b in (0, 1, 89, 2047, 2048, 2049, 2099):
            K, V = d.kv(b, d.lens[b])
            d.hold(out[b], lse[b], b, d.q[b], K, V, d.lens[b] - 1, visible(m, b, d.lens[b] - 1, d.lens[b]), m, d.decode_weights())
    finally:
        d.close()


@pytest.mark.parametrize("heads", [HEADS[1], HEADS[6], HEADS[8], HEADS[11]], ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
def test_whole_and_cut_units(kvc, heads):
    """Chunks on both sides of the choice between whole units and cut ones, with and without a workspace."""
    c = Rows(kvc, [5000], **heads)
    try:
        for q_start, n_q in ((0, 64), (400, 100), (1900, 100), (4000, 1000), (4990, 10)):
            m = Mod(softcap=7.0)
            q = c.queries(n_q)
            some = sorted({0, n_q // 2, n_q - 1})
            c.check_prefill(*c.prefill(m, q, q_start), m, q, q_start, some=some)
            c.check_prefill(*c.prefill(m, q, q_start, workspace=None), m, q, q_start, some=some)
    finally:
        c.close()


def test_nan_and_infinite_scores(kvc):
    """A NaN key of a read position makes its row NaN and no other; hidden ones do nothing; huge scores under a cap
    weigh like the cap."""
    c = Rows(kvc, [300, 300], H_Q=8, H_KV=2)
    try:
        view = c.pool.bytes_view().view(torch.bfloat16).view(2, c.N, 2, 2, 16, 128)
        view[1, int(c.table[0, 6]), :, 0, 4] = float("nan")   # key 100 of row 0
        m = Mod(softcap=8.0, window=150)
        out, lse = c.decode(m)   # reads 150..299
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        out, lse = c.decode(Mod(softcap=8.0))
        assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
        q = c.queries(200)
        for cap in (8.0, 0.0):
            out, lse = c.prefill(Mod(softcap=cap), q, 0)
            assert torch.isfinite(out[:100]).all() and torch.isnan(out[100:]).all()
        # a huge finite key: with |q| < 20 the 128 products of up to 2e36 sum to under 2.6e38, inside fp32 (a larger one
        # overflows to infinities of both signs, whose sum is NaN whatever the cap)
        assert q.abs().max() < 20 and c.q.abs().max() < 20
        view[1, int(c.table[1, 6]), :, 0, 4] = 1e35
        out, lse = c.decode(Mod(softcap=8.0))
        assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()
        out, lse = c.prefill(Mod(softcap=8.0), q, 0, row=1)
        assert torch.isfinite(out).all()
    finally:
        c.close()


@pytest.mark.parametrize("softcap", [0.0, 50.0, 100.0, 4096.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int4"])
def test_scores_that_climb(kvc, dtype, softcap):
    """Scores that grow along the row past every slack of the running references, up to about 150."""
    n, D = 1500, 128
    c = Rows(kvc, [n, 40], dtype=dtype)
    try:
        u = np.where(c.r.random(D) < 0.5, -1.0, 1.0)
        ramp = np.linspace(0.0, 1.2, n)[:, None, None] * u + 0.05 * c.r.standard_normal((n, c.H_KV, D))
        k, v = bf16(ramp).cuda(), bf16(c.r.standard_normal((n, c.H_KV, D))).cuda()
        kvc.kvc_write_tokens(c.pool, c.layer, c.bt[:1].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                             torch.tensor([0, n], dtype=torch.int32, device="cuda"), k, v, max_tokens=n)
        torch.cuda.synchronize()
        raw = c.pool.bytes_view().cpu().numpy().reshape(c.pool.num_layers, -1)[c.layer]
        c.stored = pool_values(raw, dtype, c.N, c.H_KV, 16, D)
        m = Mod(softcap=softcap)
        q = bf16(11.0 * u + 0.5 * c.r.standard_normal((70, c.H_Q, D))).cuda()
        c.check_prefill(*c.prefill(m, q, n - 70), m, q, n - 70)
        c.q = q[:2].contiguous()
        c.check_decode(*c.decode(m), m)
    finally:
        c.close()


@pytest.mark.parametrize("softcap", [0.0, 5.0, 50.0])
@pytest.mark.parametrize("heads", HEADS[:8], ids=head_ids[:8])
def test_one_key_read_gives_its_value(kvc, heads, softcap):
    """A row that reads one key has that key's value as its output, bit for bit: the weight w (one bf16, or a pair)
    is divided by the same w in fp32, and the few fp32 roundings of (w v) / w stay far inside bf16's half step."""
    n_q, q_start = 150, 700
    c = Rows(kvc, [q_start + n_q, 77], **heads)
    try:
        m = Mod(softcap=softcap, window=1)
        q = c.queries(n_q)
        out, lse = c.prefill(m, q, q_start)
        c.check_prefill(out, lse, m, q, q_start)
        V = np.repeat(c.kv(0, q_start + n_q)[1][q_start:], c.H_Q // c.H_KV, axis=1)
        assert np.array_equal(f64(out), V)
        out, lse = c.decode(m)
        c.check_decode(out, lse, m)
        for b, n in enumerate(c.lens):
            assert np.array_equal(f64(out[b]), np.repeat(c.kv(b, n)[1][n - 1], c.H_Q // c.H_KV, axis=0))
    finally:
        c.close()


def test_decode_equals_a_chunk_of_one(kvc):
    """The decode form and the chunk form of one token agree within both forms' bounds."""
    c = Rows(kvc, [777])
    try:
        for m in (Mod(softcap=9.0, window=300, sink=4), Mod(alibi=slopes(8), prefix=40)):
            c.check_decode(*c.decode(m), m)
            c.check_prefill(*c.prefill(m, c.q, 776), m, c.q, 776)
    finally:
        c.close()


def test_no_mod_matches_the_plain_calls(kvc):
    c = Rows(kvc, [500, 1300], H_Q=8, H_KV=2)
    try:
        out, lse = c.outputs(2)
        kvc.kvc_decode_attn_mod(c.pool, 1, c.q, c.bt, c.len_t, out, lse)
        ref, rl = torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 8, device="cuda")
        kvc.kvc_decode_attn(c.pool, 1, c.q, c.bt, c.len_t, ref, rl)
        c.check_decode(out, lse, Mod())
        c.check_decode(ref.to(torch.bfloat16), rl, Mod())
    finally:
        c.close()


def test_two_graphs_side_by_side(kvc):
    """Two captured graphs with a workspace each, replayed on two streams, give the eager results."""
    c, d = Rows(kvc, [4000, 100], H_Q=32, H_KV=1), Rows(kvc, [3000], H_Q=8, H_KV=2)
    try:
        m = Mod(softcap=30.0, window=2500, sink=4)
        wc = kvc.kvc_mod_workspace(c.pool, 2, 32, c.table.shape[1])
        wd = kvc.kvc_mod_workspace(d.pool, 64, 8, d.table.shape[1])
        q, mc, md = d.queries(40), c.dev_mod(m), d.dev_mod(m)
        row = d.bt[0].contiguous()
        oc, lc = c.decode(m, wc)
        od, ld = d.prefill(m, q, 2900, workspace=wd)
        torch.cuda.synchronize()
        o1, l1 = c.outputs(2)
        o2, l2 = d.outputs(40)
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1):
            kvc.kvc_decode_attn_mod(c.pool, 1, c.q, c.bt, c.len_t, o1, l1, mod=mc, scale=c.scale, workspace=wc)
        with torch.cuda.graph(g2):
            kvc.kvc_prefill_attn_mod(d.pool, 1, q, row, 2900, o2, l2, mod=md, scale=d.scale, workspace=wd)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(5):
            with torch.cuda.stream(s1):
                g1.replay()
            with torch.cuda.stream(s2):
                g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, oc) and torch.equal(l1, lc) and torch.equal(o2, od) and torch.equal(l2, ld)
    finally:
        c.close()
        d.close()


def test_first_calls_inside_a_capture():
    """The first calls of a process, captured into a graph at once, then replayed (a child process)."""
    import os
    import subprocess
    import sys
    code = """
import torch
import paged_kv_cache_kvc_gb300 as kvc
p = kvc.kvc_pool_create(64, 16, 1, 2, 128)
p.bytes_view().view(torch.bfloat16).normal_()
bt = torch.arange(60, device="cuda").int().view(2, 30)
lens = torch.tensor([300, 470], device="cuda").int()
q = torch.randn(2, 8, 128, device="cuda").bfloat16()
kv = torch.randn(2, 2, 128, device="cuda").bfloat16()
ws = kvc.kvc_mod_workspace(p, 64, 8, 30)
rope = kvc.Rope(torch.ones(64, device="cuda") * 0.01)
mod = kvc.ScoreMod(softcap=20.0)
qr, out, out2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
row = bt[0].contiguous()
after = lens + 1
torch.cuda.synchronize()
def step():
    kvc.kvc_rope_append(p, 0, bt, lens, q, kv, kv, qr, rope)
    kvc.kvc_decode_attn_mod(p, 0, qr, bt, after, out, mod=mod, workspace=ws)
    kvc.kvc_prefill_attn_mod(p, 0, qr, row, 299, out2, mod=mod, workspace=ws)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
a, b = out.clone(), out2.clone()
step()
torch.cuda.synchronize()
assert kvc.kvc_pool_sync_status(p) == kvc.KVC_OK
assert torch.equal(a, out) and torch.equal(b, out2) and torch.isfinite(a).all() and torch.isfinite(b).all()
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_write_then_attend(kvc):
    """As a model's layer uses them: a prompt's chunk rotated and written, attended, then decode steps."""
    from mod_reference import rotate
    H_Q, H_KV, D, n0, steps = 8, 2, 128, 75, 3
    r = np.random.default_rng(3)
    total = n0 + steps
    pool = kvc.kvc_pool_create(8, 16, 1, H_KV, D)
    try:
        pool.bytes_view().fill_(NAN_BYTE)
        bt = torch.tensor([[5, 2, 7, 0, 3]], dtype=torch.int32, device="cuda")
        qkv = bf16(r.standard_normal((total, (H_Q + 2 * H_KV) * D))).cuda()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([H_Q * D, H_KV * D, H_KV * D], 1))
        f = np.array([10000.0 ** (-2.0 * i / D) for i in range(D // 2)], np.float32)
        w = bf16(1 + 0.1 * r.standard_normal(D))
        rope = kvc.Rope(torch.from_numpy(f).cuda(), q_norm=w.cuda(), k_norm=w.cuda())
        m = Mod(softcap=20.0, window=40, sink=4)
        mod = kvc.ScoreMod(softcap=20.0, window=40, sink=4)
        ws = kvc.kvc_mod_workspace(pool, n0, H_Q, 5)
        q_rot = torch.empty((total, H_Q, D), dtype=torch.bfloat16, device="cuda")
        out = torch.empty((total, H_Q, D), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((total, H_Q), device="cuda")
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n0], dtype=torch.int32, device="cuda")
        kvc.kvc_rope_write_tokens(pool, 0, bt, zero, cu, q[:n0], k[:n0], v[:n0], q_rot[:n0], rope)
        kvc.kvc_prefill_attn_mod(pool, 0, q_rot[:n0], bt[0], 0, out[:n0], lse[:n0], mod=mod, workspace=ws)
        lens = torch.tensor([n0], dtype=torch.int32, device="cuda")
        for i in range(n0, total):
            kvc.kvc_rope_append(pool, 0, bt, lens, q[i:i + 1], k[i:i + 1], v[i:i + 1], q_rot[i:i + 1], rope)
            lens += 1
            kvc.kvc_decode_attn_mod(pool, 0, q_rot[i:i + 1], bt, lens, out[i:i + 1], lse[i:i + 1], mod=mod, workspace=ws)
        torch.cuda.synchronize()
        assert kvc.kvc_pool_sync_status(pool) == kvc.KVC_OK
        pos = np.arange(total)
        qr, qt = rotate(f64(q), pos, f, False, f64(w))
        kr, kt = rotate(f64(k), pos, f, False, f64(w))
        # the operators hand each other bf16: take their rounded values where they are within a half step of the
        # definition's, so that the attention is held to its own bound
        got_q = f64(q_rot)
        assert np.all(np.abs(got_q - qr) <= 2.0 ** -8 * (np.abs(qr) + qt) + qt)
        image = pool_values(pool.bytes_view().cpu().numpy(), "bf16", 8, H_KV, 16, D)
        flat = np.stack([image[int(bt[0, t // 16]), :, :, t % 16] for t in range(total)])   # [T, H_KV, 2, D]
        K, V = flat[:, :, 0], flat[:, :, 1]
        assert np.all(np.abs(K - kr) <= 2.0 ** -8 * (np.abs(kr) + kt) + kt) and np.array_equal(V, f64(v))
        for i in range(total):
            n = n0 if i < n0 else i + 1
            ro, rl, to, tl = attend(got_q[i], K[:n], V[:n], i, visible(m, i, i, n), m, D ** -0.5, H_Q // H_KV, "bf16", "pair" if i >= n0 else "bf16")
            assert np.all(np.abs(f64(out[i]) - ro) <= to) and np.all(np.abs(f64(lse[i]) - rl) <= tl), i
    finally:
        pool.close()


@pytest.mark.parametrize("heads", [HEADS[1], HEADS[6]], ids=[head_ids[1], head_ids[6]])
@pytest.mark.parametrize("first", ["decode", "decode_unsplit", "prefill", "prefill_short"])
def test_a_step_after_the_call_sees_its_outputs(kvc, first, heads):
    """kvc_mixed_step's chunk starts without waiting for the kernel before the step: these calls' kernels let nothing
    but their own merge start early, so a chunk whose queries are the outputs of such a call reads them finished."""
    n = 64 if first == "prefill_short" else 200
    rows = n if first.startswith("decode") else 2
    c = Rows(kvc, [9000] + [33] * (rows - 1), **heads)
    try:
        q, m = c.queries(n), Mod(softcap=5.0)
        ws = kvc.kvc_mod_workspace(c.pool, n, c.H_Q, c.table.shape[1])
        one, lens = c.bt[1:2].contiguous(), torch.tensor([33], dtype=torch.int32, device="cuda")
        k_new, v_new = (bf16(c.r.standard_normal((1, c.H_KV, c.D))).cuda() for _ in range(2))

        def run(wait):
            out, lse = c.outputs(n)
            if first == "prefill":
                c.kvc.kvc_prefill_attn_mod(c.pool, c.layer, q, c.bt[0].contiguous(), 8800, out, lse, mod=c.dev_mod(m), workspace=ws)
            elif first == "prefill_short":
                c.kvc.kvc_prefill_attn_mod(c.pool, c.layer, q, c.bt[0].contiguous(), 0, out, lse, mod=c.dev_mod(m), workspace=ws)
            else:
                c.decode(m, ws if first == "decode" else None, out, lse)
            if wait:
                torch.cuda.synchronize()
            o1, chunk = torch.empty((1, c.H_Q, c.D), device="cuda"), torch.empty((n, c.H_Q, c.D), device="cuda")
            kvc.kvc_mixed_step(c.pool, c.layer, q[:1].contiguous(), one, lens, k_new, v_new, o1, None, out, c.bt[0].contiguous(), 300, chunk)
            return chunk

        want = run(True)
        assert bool(torch.isfinite(want).all())
        for _ in range(4):
            assert torch.equal(run(False), want)
    finally:
        c.close()


def test_expired_waits_are_reported(kvc, monkeypatch):
    """With every load withheld (a test hook) the calls report KVC_ERR_TIMEOUT and return; the pool then works."""
    c = Rows(kvc, [300, 20])
    try:
        m = Mod(softcap=10.0)
        q = c.queries(20)
        monkeypatch.setenv("KVC_TEST_STALL", "1")
        c.decode(m)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_TIMEOUT
        c.prefill(m, q, 200)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_TIMEOUT
        monkeypatch.delenv("KVC_TEST_STALL")
        c.check_decode(*c.decode(m), m)
        c.check_prefill(*c.prefill(m, q, 200), m, q, 200)
    finally:
        c.close()


def test_refusals(kvc):
    c = Rows(kvc, [100, 50], H_Q=8, H_KV=2)
    try:
        out, lse = c.outputs(2)
        q1, row = c.q[:1].contiguous(), c.bt[0].contiguous()

        def dec(**k):
            a = dict(layer=1, q=c.q, bt=c.bt, lens=c.len_t, out=out, lse=lse, mod=None, scale=None, ws=None) | k
            kvc.kvc_decode_attn_mod(c.pool, a["layer"], a["q"], a["bt"], a["lens"], a["out"], a["lse"], mod=a["mod"],
                                    scale=a["scale"], workspace=a["ws"])

        def pre(**k):
            a = dict(q_start=99, mod=None, ws=None) | k
            kvc.kvc_prefill_attn_mod(c.pool, 1, q1, row, a["q_start"], out[:1], lse[:1], mod=a["mod"], workspace=a["ws"])

        doc = torch.zeros(2, dtype=torch.int32, device="cuda")
        for k in (dict(q=c.q.float()), dict(out=out.float()), dict(out=out[:1]), dict(lse=lse[:1]), dict(lens=c.len_t[:1]),
                  dict(lens=c.len_t.long()), dict(q=c.q[:, :, :64].contiguous()),
                  dict(mod=kvc.ScoreMod(alibi=torch.ones(3, device="cuda")))):
            with pytest.raises(ValueError):
                dec(**k)
        for status, k in ((kvc.KVC_ERR_ARG, dict(layer=2)), (kvc.KVC_ERR_ARG, dict(mod=kvc.ScoreMod(softcap=-1.0))),
                          (kvc.KVC_ERR_ARG, dict(mod=kvc.ScoreMod(softcap=float("nan")))),
                          (kvc.KVC_ERR_ARG, dict(mod=kvc.ScoreMod(softcap=1e-42))),
                          (kvc.KVC_ERR_UNSUPPORTED, dict(mod=kvc.ScoreMod(softcap=4097.0))),
                          (kvc.KVC_ERR_ARG, dict(mod=kvc.ScoreMod(window=-1))), (kvc.KVC_ERR_ARG, dict(mod=kvc.ScoreMod(sink=-1))),
                          (kvc.KVC_ERR_ARG, dict(mod=kvc.ScoreMod(doc_start=doc))), (kvc.KVC_ERR_ARG, dict(scale=0.0)),
                          (kvc.KVC_ERR_ARG, dict(scale=-1.0)), (kvc.KVC_ERR_ARG, dict(scale=float("inf")))):
            with pytest.raises(kvc.KvcError) as e:
                dec(**k)
            assert e.value.status == status, k
        for status, k in ((kvc.KVC_ERR_RANGE, dict(q_start=16 * c.table.shape[1])), (kvc.KVC_ERR_ARG, dict(q_start=-1)),
                          (kvc.KVC_ERR_UNSUPPORTED, dict(mod=kvc.ScoreMod(prefix=3, doc_start=doc[:1])))):
            with pytest.raises(kvc.KvcError) as e:
                pre(**k)
            assert e.value.status == status, k
        d = Rows(kvc, [4000], H_Q=8, H_KV=2)
        small = torch.zeros(70000, dtype=torch.uint8, device="cuda")
        with pytest.raises(kvc.KvcError) as e:   # a workspace that does not hold the call's splits
            d.decode(Mod(), small[:65536 + 256])
        assert e.value.status == kvc.KVC_ERR_ARG
        d.close()
        other = kvc.kvc_pool_create(4, 4, 1, 2, 64)   # blocks of 4 positions: written, not attended
        with pytest.raises(kvc.KvcError) as e:
            kvc.kvc_decode_attn_mod(other, 0, torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda"),
                                    torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"),
                                    torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda"))
        assert e.value.status == kvc.KVC_ERR_UNSUPPORTED
        other.close()
        assert torch.all(torch.isnan(out.float()))   # nothing ran
    finally:
        c.close()
