"""The rotary write (kvc_rope_append, kvc_rope_write_tokens) against its 64-bit form."""
import numpy as np
import pytest
import torch

from mod_reference import HALF, bf16, f64, pool_values, rotate

pytestmark = pytest.mark.gpu

DT = {"bf16": 0, "fp8": 1, "int4": 2}


def inv_freq(R, base=10000.0):
    return np.array([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=np.float32)


class Case:
    """Random tokens of ragged sequences, a pool full of a marker byte, and a table of distinct blocks."""

    def __init__(self, kvc, runs, H_Q=4, H_KV=2, D=64, dtype="bf16", bs=16, R=None, interleaved=False, norm=False,
                 layers=2, layer=1, extra=0, fused=True, seed=0, far_table=None):
        self.kvc, self.runs, self.dtype, self.layer, self.bs, self.D, self.H_KV, self.H_Q = (
            kvc, runs, dtype, layer, bs, D, H_KV, H_Q)
        r = np.random.default_rng(seed)
        self.T = sum(n for _, n in runs)
        rows = self.T + extra
        w = (H_Q + 2 * H_KV) * D
        x = bf16(r.standard_normal((rows, w)) * 2).cuda()
        if not fused:
            x = torch.cat([x, torch.zeros_like(x[:, :8])], 1)[:, :w]   # rows 16 bytes further apart
        self.q, self.k, self.v = (a.unflatten(1, (-1, D)) for a in x.split([H_Q * D, H_KV * D, H_KV * D], 1))
        R = D if R is None else R
        self.f = inv_freq(R) if R else np.zeros(0, np.float32)
        self.wq, self.wk = ((bf16(1 + 0.2 * r.standard_normal(D)), bf16(1 + 0.2 * r.standard_normal(D)))
                            if norm else (None, None))
        self.inter = interleaved
        self.rope = kvc.Rope(torch.from_numpy(self.f).cuda() if R else None, interleaved=interleaved,
                             q_norm=self.wq.cuda() if norm else None, k_norm=self.wk.cuda() if norm else None, eps=1e-5)
        mb = far_table or max(1, max(-(-(s + n) // bs) for s, n in runs))
        need = [(b, j) for b, (s, n) in enumerate(runs) if n for j in range(s // bs, (s + n - 1) // bs + 1)]
        self.N = len(need) + 3
        ids = r.permutation(self.N)[:len(need)]
        self.table = np.full((len(runs), mb), -1, np.int32)
        for (b, j), p in zip(need, ids):
            self.table[b, j] = p
        self.pool = kvc.kvc_pool_create(self.N, bs, layers, H_KV, D, DT[dtype])
        self.pool.bytes_view().fill_(0x5A)
        self.scales = None
        if dtype != "bf16":
            self.scales = (0.02 + 0.03 * r.random((2, H_KV, D))).astype(np.float32) * (1 if dtype == "fp8" else 20)
            sc = torch.from_numpy(self.scales).cuda()
            kvc.kvc_pool_set_scales(self.pool, layer, sc[0].contiguous(), sc[1].contiguous())
        self.bt = torch.from_numpy(self.table).cuda()
        self.start = torch.tensor([s for s, _ in runs], dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum([n for _, n in runs])]), dtype=torch.int32, device="cuda")
        self.q_out = torch.full((rows, H_Q, D), 7.0, dtype=torch.bfloat16, device="cuda")

    def write(self, q="own", out="own", append=False, stream=None):
        q, out = (self.q if isinstance(q, str) else q), (self.q_out if isinstance(out, str) else out)
        if append:
            self.kvc.kvc_rope_append(self.pool, self.layer, self.bt, self.start, q, self.k, self.v, out, self.rope,
                                     stream=stream)
        else:
            self.kvc.kvc_rope_write_tokens(self.pool, self.layer, self.bt, self.start, self.cu, q, self.k, self.v, out,
                                           self.rope, stream=stream)

    def positions(self):
        return np.concatenate([np.arange(s, s + n) for s, n in self.runs]).astype(np.int64)

    def image(self):
        """The layer's bytes, and every other layer must still hold the marker."""
        raw = self.pool.bytes_view().cpu().numpy().reshape(self.pool.num_layers, -1)
        others = np.delete(raw, self.layer, axis=0)
        assert np.all(others == 0x5A)
        return raw[self.layer]

    def check(self, q_out=None, stored=None):
        """stored: bool per token (default: all)."""
        torch.cuda.synchronize()
        T, D = self.T, self.D
        pos = self.positions()
        q_out = self.q_out if q_out is None else q_out
        w64 = (None, None) if self.wq is None else (f64(self.wq), f64(self.wk))
        if T and self.H_Q:
            ref, tol = rotate(f64(self.q)[:T], pos, self.f, self.inter, w64[0], 1e-5)
            got = f64(q_out)[:T]
            bad = np.abs(got - ref) > HALF["bf16"] * (np.abs(ref) + tol) + tol
            assert not bad.any(), f"{bad.sum()} queries off, worst {np.max(np.abs(got - ref))}"
        raw = self.image()
        vals = pool_values(raw, self.dtype, self.N, self.H_KV, self.bs, D)
        marker = pool_values(np.full_like(raw, 0x5A), self.dtype, self.N, self.H_KV, self.bs, D)
        touched = np.zeros(vals.shape[:1] + vals.shape[3:4], bool)
        ref, tol = rotate(f64(self.k)[:T], pos, self.f, self.inter, w64[1], 1e-5)
        at = 0
        for b, (s, n) in enumerate(self.runs):
            for i in range(n):
                if stored is None or stored[at]:
                    blk, slot = self.table[b, (s + i) // self.bs], (s + i) % self.bs
                    touched[blk, slot] = True
                    got = vals[blk, :, :, slot]
                    v = f64(self.v)[at]
                    if self.dtype == "bf16":
                        assert np.all(np.abs(got[:, 0] - ref[at]) <= HALF["bf16"] * (np.abs(ref[at]) + tol[at]) + tol[at])
                        assert np.array_equal(got[:, 1], v)
                    else:
                        y = ref[at] / self.scales[0]
                        e = tol[at] / self.scales[0] + np.abs(y) * 2.0 ** -23
                        if self.dtype == "fp8":   # half a step: 2^-4 relative, 2^-10 below the normal range
                            y = np.clip(y, -448, 448)
                            assert np.all(np.abs(got[:, 0] - y) <= np.maximum(2.0 ** -4 * (np.abs(y) + e), 2.0 ** -10) + e)
                        else:
                            assert np.all(np.abs(got[:, 0] - np.clip(y, -7, 7)) <= 0.5 + e)
                at += 1
        untouched = ~touched
        assert np.array_equal(np.moveaxis(vals, 3, 1)[untouched], np.moveaxis(marker, 3, 1)[untouched], equal_nan=True)

    def close(self):
        self.pool.close()


SHAPES = [
    dict(H_Q=4, H_KV=2, D=64), dict(H_Q=32, H_KV=8, D=128), dict(H_Q=5, H_KV=5, D=64), dict(H_Q=32, H_KV=1, D=128),
    dict(H_Q=12, H_KV=3, D=128, interleaved=True), dict(H_Q=8, H_KV=2, D=64, interleaved=True, norm=True),
    dict(H_Q=4, H_KV=2, D=128, norm=True), dict(H_Q=4, H_KV=2, D=128, norm=True, R=64),
    dict(H_Q=4, H_KV=2, D=128, R=48), dict(H_Q=4, H_KV=2, D=64, R=16, interleaved=True), dict(H_Q=4, H_KV=2, D=64, R=0),
    dict(H_Q=4, H_KV=2, D=128, R=0, norm=True), dict(H_Q=3, H_KV=1, D=64, bs=4), dict(H_Q=3, H_KV=1, D=128, bs=37),
    dict(H_Q=8, H_KV=8, D=128, dtype="fp8"), dict(H_Q=8, H_KV=2, D=128, dtype="fp8", norm=True, interleaved=True),
    dict(H_Q=8, H_KV=2, D=128, dtype="int4"), dict(H_Q=8, H_KV=2, D=128, dtype="int4", norm=True, R=96),
    dict(H_Q=4, H_KV=2, D=64, fused=False),
]
ids = ["-".join(f"{k}{v}" for k, v in s.items()) for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_append(kvc, shape):
    c = Case(kvc, [(s, 1) for s in (0, 1, 15, 16, 17, 300, 4095, 4096, 100001)], **shape)
    try:
        c.write(append=True)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        c.check()
    finally:
        c.close()


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_ragged_write(kvc, shape):
    c = Case(kvc, [(7, 20), (0, 0), (0, 1), (33, 67), (5000, 3), (9, 0)], extra=5, **shape)
    try:
        c.write()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        c.check()
        assert torch.all(c.q_out[c.T:] == 7.0)   # rows behind the last sequence
    finally:
        c.close()


def test_values_are_stored_as_the_plain_write_stores_them(kvc):
    for dtype in ("fp8", "int4"):
        c = Case(kvc, [(3, 40), (100, 9)], H_Q=2, H_KV=2, D=128, dtype=dtype)
        try:
            c.write()
            torch.cuda.synchronize()
            mine = c.pool.bytes_view().clone()
            kvc.kvc_write_tokens(c.pool, c.layer, c.bt, c.start, c.cu, c.k.contiguous(), c.v.contiguous(), max_tokens=40)
            view = lambda x: x.view(2, c.N, 2, 2, 16, -1)[:, :, :, 1]
            assert torch.equal(view(mine), view(c.pool.bytes_view()))
        finally:
            c.close()


@pytest.mark.parametrize("n", [600, 5000])
def test_many_tokens(kvc, n):
    c = Case(kvc, [(11, n), (0, 13), (40, 1)], H_Q=4, H_KV=2, D=128, norm=True)
    try:
        c.write()
        c.check()
    finally:
        c.close()


def test_many_sequences(kvc):
    """More sequences than one search step probes, empty ones among them."""
    r = np.random.default_rng(5)
    c = Case(kvc, [(int(r.integers(0, 50)), int(r.integers(0, 4))) for _ in range(1500)], H_Q=2, H_KV=1, D=64)
    try:
        c.write()
        c.check()
    finally:
        c.close()


@pytest.mark.parametrize("pos", [2 ** 20 + 5, 2 ** 24 - 1, 2 ** 27 + 3])
def test_far_positions(kvc, pos):
    c = Case(kvc, [(pos, 2)], H_Q=2, H_KV=1, D=64, bs=128)
    try:
        c.write()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
        c.check()
    finally:
        c.close()


def test_in_place_and_keys_only(kvc):
    c = Case(kvc, [(5, 30), (2, 1)], H_Q=6, H_KV=2, D=64, norm=True)
    try:
        q = c.q.contiguous()
        c.write(q=q, out=q)
        c.check(q_out=q)
        c.pool.bytes_view().fill_(0x5A)
        c.write(q=None, out=None)
        c.H_Q = 0
        c.check()
    finally:
        c.close()


def test_bad_entries_and_positions_are_skipped_and_recorded(kvc):
    c = Case(kvc, [(0, 3), (16, 2), (40, 2)], H_Q=2, H_KV=1, D=64)
    try:
        c.table[0, 0], saved = c.N, c.table[0, 0]
        c.bt.copy_(torch.from_numpy(c.table))
        c.write()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        c.check(stored=[False] * 3 + [True] * 4)
        c.table[0, 0] = saved
        c.bt.copy_(torch.from_numpy(c.table))
        c.pool.bytes_view().fill_(0x5A)
        c.start[1] = 16 * c.table.shape[1]   # past the row
        c.write()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        c.start[1] = -2
        c.write()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        c.runs = [(0, 3), (-2, 2), (40, 2)]   # the query rows are rotated by the positions as given
        c.check(stored=[True] * 3 + [False] * 2 + [True] * 2)
    finally:
        c.close()


def test_captured_and_on_another_stream(kvc):
    c = Case(kvc, [(5, 30), (2, 1)], H_Q=4, H_KV=2, D=64)
    try:
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        c.write(stream=side)
        side.synchronize()
        c.check()
        c.pool.bytes_view().fill_(0x5A)
        c.q_out.fill_(7.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.write()
        c.q_out.fill_(7.0)
        for _ in range(3):
            graph.replay()
        c.check()
    finally:
        c.close()


def test_refusals(kvc):
    c = Case(kvc, [(5, 4)], H_Q=4, H_KV=2, D=64)
    try:
        before = c.pool.bytes_view().clone()
        bad = [dict(q=c.q.float()), dict(k=c.k[:, :1]), dict(v=c.v[:2]), dict(q_out=c.q_out[:2]), dict(q=None),
               dict(q=c.q.transpose(0, 1).contiguous().transpose(0, 1)),
               dict(rope=kvc.Rope(c.rope.inv_freq, q_norm=torch.ones(32, dtype=torch.bfloat16, device="cuda"))),
               dict(bt=c.bt.long()), dict(cu=c.cu[:1]), dict(start=c.start.repeat(2))]
        for b in bad:
            a = dict(bt=c.bt, start=c.start, cu=c.cu, q=c.q, k=c.k, v=c.v, q_out=c.q_out, rope=c.rope) | b
            with pytest.raises(ValueError):
                kvc.kvc_rope_write_tokens(c.pool, 1, a["bt"], a["start"], a["cu"], a["q"], a["k"], a["v"], a["q_out"], a["rope"])
        buf = torch.zeros(4 * 4 * 64 + 64, dtype=torch.bfloat16, device="cuda")
        for status, b in [
                (kvc.KVC_ERR_ARG, dict(layer=2)), (kvc.KVC_ERR_ARG, dict(layer=-1)),
                (kvc.KVC_ERR_ARG, dict(q=buf[1:1 + 1024].view(4, 4, 64))),                       # misaligned
                (kvc.KVC_ERR_ARG, dict(q=buf[:1024].view(4, 4, 64), q_out=buf[64:64 + 1024].view(4, 4, 64))),
                (kvc.KVC_ERR_UNSUPPORTED, dict(rope=kvc.Rope(c.rope.inv_freq[:4].contiguous()))),
                (kvc.KVC_ERR_ARG, dict(rope=kvc.Rope(torch.ones(64, device="cuda")))),            # wider than the head
                (kvc.KVC_ERR_ARG, dict(rope=kvc.Rope(c.rope.inv_freq, q_norm=torch.ones(64, dtype=torch.bfloat16, device="cuda"),
                                                     eps=float("nan"))))]:
            a = dict(layer=1, q=c.q, q_out=c.q_out, rope=c.rope) | b
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_rope_write_tokens(c.pool, a["layer"], c.bt, c.start, c.cu, a["q"], c.k, c.v, a["q_out"], a["rope"])
            assert e.value.status == status
        torch.cuda.synchronize()
        assert torch.equal(before, c.pool.bytes_view())
    finally:
        c.close()
