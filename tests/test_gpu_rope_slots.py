"""kvc_rope_write_slots: rows by slot, positions with several axes."""
import numpy as np
import pytest
import torch

from mod_reference import HALF, bf16, f64, pool_values
from sparse_reference import rotate_axes

pytestmark = pytest.mark.gpu

DT = {"bf16": 0, "fp8": 1, "int4": 2}


def freqs(R):
    return np.array([10000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=np.float32)


class Case:
    def __init__(self, kvc, T, axes=3, H_Q=4, H_KV=2, D=64, dtype="bf16", bs=16, R=None, interleaved=False, norm=False,
                 far=5000, pad=(), seed=0, axis_of="turns", layer=1):
        r = np.random.default_rng(seed)
        self.kvc, self.T, self.D, self.bs, self.H_Q, self.H_KV, self.dtype, self.layer = kvc, T, D, bs, H_Q, H_KV, dtype, layer
        self.N = -(-2 * T // bs) + 2
        self.slots = r.permutation(self.N * bs)[:T].astype(np.int32)
        self.slots[list(pad)] = -1
        self.positions = r.integers(-far, far, (axes, T)).astype(np.int32)
        R = D if R is None else R
        self.f, self.inter = freqs(R), interleaved
        self.axis_of = {"turns": np.arange(R // 2) % axes, "sections": np.arange(R // 2) * axes // max(1, R // 2),
                        "none": np.zeros(R // 2)}[axis_of].astype(np.uint8)
        x = bf16(r.standard_normal((T, (H_Q + 2 * H_KV) * D)) * 2).cuda()
        self.q, self.k, self.v = (a.unflatten(1, (-1, D)) for a in x.split([H_Q * D, H_KV * D, H_KV * D], 1))
        self.wq, self.wk = ((bf16(1 + 0.2 * r.standard_normal(D)), bf16(1 + 0.2 * r.standard_normal(D))) if norm else (None, None))
        self.rope = kvc.Rope(torch.from_numpy(self.f).cuda() if R else None, interleaved=interleaved,
                             q_norm=self.wq.cuda() if norm else None, k_norm=self.wk.cuda() if norm else None, eps=1e-5,
                             axis_of=torch.from_numpy(self.axis_of).cuda() if R and axis_of != "none" else None)
        self.pool = kvc.kvc_pool_create(self.N, bs, 2, H_KV, D, DT[dtype])
        self.pool.bytes_view().fill_(0x5A)
        self.scales = None
        if dtype != "bf16":
            self.scales = (0.02 + 0.03 * r.random((2, H_KV, D))).astype(np.float32) * (1 if dtype == "fp8" else 20)
            sc = torch.from_numpy(self.scales).cuda()
            kvc.kvc_pool_set_scales(self.pool, layer, sc[0].contiguous(), sc[1].contiguous())
        self.q_out = torch.full((T, H_Q, D), 7.0, dtype=torch.bfloat16, device="cuda")

    def write(self, positions=None, slots=None, **how):
        s = torch.from_numpy(self.slots).cuda() if slots is None else slots
        p = torch.from_numpy(self.positions).cuda() if positions is None else positions
        self.kvc.kvc_rope_write_slots(self.pool, self.layer, s, p, self.q, self.k, self.v, self.q_out, self.rope, **how)

    def check(self):
        torch.cuda.synchronize()
        live = self.slots != -1
        ref, tol = rotate_axes(f64(self.q), self.positions, self.axis_of, self.f, self.inter,
                               None if self.wq is None else f64(self.wq), 1e-5)
        got = f64(self.q_out)
        assert np.all((np.abs(got - ref) <= HALF["bf16"] * (np.abs(ref) + tol) + tol)[live])
        assert np.all(got[~live] == 7.0)
        raw = self.pool.bytes_view().cpu().numpy().reshape(2, -1)
        assert np.all(raw[1 - self.layer] == 0x5A)
        vals = pool_values(raw[self.layer], self.dtype, self.N, self.H_KV, self.bs, self.D)
        marker = pool_values(np.full_like(raw[0], 0x5A), self.dtype, self.N, self.H_KV, self.bs, self.D)
        ref, tol = rotate_axes(f64(self.k), self.positions, self.axis_of, self.f, self.inter,
                               None if self.wk is None else f64(self.wk), 1e-5)
        v = f64(self.v)
        touched = np.zeros((self.N, self.bs), bool)
        for r in np.flatnonzero(live):
            blk, at = divmod(int(self.slots[r]), self.bs)
            touched[blk, at] = True
            got = vals[blk, :, :, at]
            if self.dtype == "bf16":
                assert np.all(np.abs(got[:, 0] - ref[r]) <= HALF["bf16"] * (np.abs(ref[r]) + tol[r]) + tol[r])
                assert np.array_equal(got[:, 1], v[r])
            else:   # half a step of the stored type, see the rotary write's tests
                y = ref[r] / self.scales[0]
                e = tol[r] / self.scales[0] + np.abs(y) * 2.0 ** -23
                if self.dtype == "fp8":
                    y = np.clip(y, -448, 448)
                    assert np.all(np.abs(got[:, 0] - y) <= np.maximum(2.0 ** -4 * (np.abs(y) + e), 2.0 ** -10) + e)
                else:
                    assert np.all(np.abs(got[:, 0] - np.clip(y, -7, 7)) <= 0.5 + e)
        both = np.moveaxis(vals, 3, 1)[~touched], np.moveaxis(marker, 3, 1)[~touched]
        assert np.array_equal(*both, equal_nan=True)

    def close(self):
        self.pool.close()


@pytest.mark.parametrize("T", [1, 3, 17, 130, 1500])
@pytest.mark.parametrize("how", [dict(), dict(axes=1, axis_of="none"), dict(axes=4, axis_of="sections", D=128, norm=True),
                                 dict(axes=2, interleaved=True, R=32), dict(dtype="fp8", D=128, H_KV=3, H_Q=6),
                                 dict(dtype="int4", D=128, bs=48, norm=True), dict(R=0, axes=1), dict(bs=7, H_Q=5, axes=8)])
def test_rows_by_slot(kvc, T, how):
    c = Case(kvc, T, pad=() if T < 3 else (1, T - 1), seed=T, **how)
    try:
        c.write()
        c.check()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("T", [40, 700, 3000])
def test_one_axis_is_the_write_by_table_bit_for_bit(kvc, dtype, T):
    c = Case(kvc, T, axes=3, D=128, dtype=dtype, norm=True, seed=3)
    try:
        blocks = -(-(T + 5) // 16)
        table = torch.randperm(c.N, generator=torch.Generator().manual_seed(1))[:blocks].int()
        t = torch.arange(5, 5 + T)
        slots = (table[t // 16] * 16 + t % 16).int().cuda()
        same = t.int().cuda()
        c.write(positions=same.expand(3, T).contiguous(), slots=slots)
        torch.cuda.synchronize()
        image, q_out = c.pool.bytes_view().clone(), c.q_out.clone()
        c.pool.bytes_view().fill_(0x5A)
        plain = kvc.Rope(c.rope.inv_freq, q_norm=c.rope.q_norm, k_norm=c.rope.k_norm, eps=1e-5)
        kvc.kvc_rope_write_tokens(c.pool, c.layer, table.cuda()[None], torch.tensor([5], dtype=torch.int32, device="cuda"),
                                  torch.tensor([0, T], dtype=torch.int32, device="cuda"), c.q, c.k, c.v, c.q_out, plain)
        assert torch.equal(image, c.pool.bytes_view()) and torch.equal(q_out, c.q_out)
        c.pool.bytes_view().fill_(0x5A)   # one row of positions for every axis, by its stride
        c.write(positions=same[None].expand(3, T), slots=slots)
        assert torch.equal(image, c.pool.bytes_view()) and torch.equal(q_out, c.q_out)
    finally:
        c.close()


def test_far_positions_of_either_sign(kvc):
    c = Case(kvc, 60, far=2 ** 24)
    try:
        c.write()
        c.check()
    finally:
        c.close()


def test_bad_slots_and_axes_are_recorded(kvc):
    c = Case(kvc, 6)
    try:
        keep = c.slots.copy()
        c.slots[2], c.slots[4] = c.N * c.bs, -2
        c.write()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_BAD_BLOCK
        ref, tol = rotate_axes(f64(c.q), c.positions, c.axis_of, c.f, False)
        assert np.all(np.abs(f64(c.q_out) - ref) <= HALF["bf16"] * (np.abs(ref) + tol) + tol)   # their queries too
        c.slots = keep
        c.pool.bytes_view().fill_(0x5A)
        c.rope.axis_of[5] = 3   # there are axes 0, 1, 2
        c.axis_of[5] = 0
        c.write()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_RANGE
        c.check()
    finally:
        c.close()


def test_keys_only_in_place_graph_and_stream(kvc):
    c = Case(kvc, 33, pad=(0, 5))
    try:
        s, p = torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.positions).cuda()
        c.write()
        torch.cuda.synchronize()
        image, q_out = c.pool.bytes_view().clone(), c.q_out.clone()
        c.pool.bytes_view().fill_(0x5A)
        kvc.kvc_rope_write_slots(c.pool, c.layer, s, p, None, c.k, c.v, None, c.rope)
        assert torch.equal(image, c.pool.bytes_view())
        c.pool.bytes_view().fill_(0x5A)
        q = c.q.contiguous()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kvc.kvc_rope_write_slots(c.pool, c.layer, s, p, q, c.k, c.v, q, c.rope)
        want = q.clone()
        graph.replay()
        live = torch.from_numpy(c.slots != -1).cuda()
        assert torch.equal(image, c.pool.bytes_view()) and torch.equal(q[live], q_out[live])
        assert torch.equal(q[~live], want[~live])
        c.pool.bytes_view().fill_(0x5A)
        c.q_out.fill_(7.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        c.write(positions=p, slots=s, stream=side)
        side.synchronize()
        assert torch.equal(image, c.pool.bytes_view()) and torch.equal(q_out, c.q_out)
    finally:
        c.close()


def test_no_rows_and_refusals(kvc):
    c = Case(kvc, 4)
    try:
        p = torch.from_numpy(c.positions).cuda()
        s = torch.from_numpy(c.slots).cuda()
        none = torch.zeros(0, dtype=torch.int32, device="cuda")
        kvc.kvc_rope_write_slots(c.pool, 1, none, none, c.q[:0], c.k[:0], c.v[:0], c.q_out[:0], c.rope)
        assert torch.all(c.pool.bytes_view() == 0x5A)
        for bad in [p[:, :3], p.t().contiguous().t(), p[None], p.long()]:
            with pytest.raises(ValueError):
                c.write(positions=bad)
        with pytest.raises(ValueError):
            c.write(slots=s[:3])
        with pytest.raises(kvc.KvcError) as e:
            c.write(positions=torch.zeros((9, 4), dtype=torch.int32, device="cuda"))
        assert e.value.status == kvc.KVC_ERR_ARG
        with pytest.raises(ValueError, match="axes"):
            kvc.kvc_rope_append(c.pool, 1, s[None], s[:1], c.q[:1], c.k[:1], c.v[:1], c.q_out[:1], c.rope)
        with pytest.raises(ValueError, match="axes"):
            kvc.kvc_rope_write_tokens(c.pool, 1, s[None], s[:1], s[:2], c.q[:1], c.k[:1], c.v[:1], c.q_out[:1], c.rope)
    finally:
        c.close()
