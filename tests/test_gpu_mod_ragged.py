"""Decode with modified scores for head groups above 16, ragged batches: every row against the 64-bit form.

Such a call is dealt in whole sequences (one launch) or cut evenly over the SMs (attention and merge: two); which of the
two it was shows in the launch count.  In a cut call a CTA's share of the keys may hold the end of one sequence, any
number of whole ones and the start of another."""
import math

import numpy as np
import pytest
import torch

from mod_reference import HALF, WEIGHTS, Mod, e4m3_table

pytestmark = pytest.mark.gpu

DT = {"bf16": 0, "fp8": 1, "int4": 2}


class Batch:
    """A pool of random keys and values (made on the device as stored bytes), `lens` positions per sequence."""

    def __init__(self, kvc, lens, H_Q=32, H_KV=1, D=128, dtype="bf16", seed=0, spare=0):
        self.kvc, self.lens, self.H_Q, self.H_KV, self.D, self.dtype = kvc, lens, H_Q, H_KV, D, dtype
        need = [-(-n // 16) for n in lens]
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.N = sum(need) + 2
        ids = np.random.default_rng(seed).permutation(self.N).astype(np.int32)
        self.table = np.full((len(lens), max(1, max(need)) + spare), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.pool = kvc.kvc_pool_create(self.N, 16, 1, H_KV, D, DT[dtype])
        raw = self.pool.bytes_view()
        self.shape = (self.N, H_KV, 2, 16)
        if dtype == "bf16":
            raw.view(torch.bfloat16).normal_(generator=g)
        elif dtype == "fp8":
            raw.copy_((torch.randn(raw.numel(), generator=g, device="cuda") * 96).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            code = torch.randint(1, 16, (raw.numel(), 2), generator=g, device="cuda", dtype=torch.uint8)
            raw.copy_(code[:, 0] | (code[:, 1] << 4))
        self.scales = None
        if dtype != "bf16":
            self.scales = (0.5 + torch.rand((2, H_KV, D), generator=g, device="cuda")) / (96 if dtype == "fp8" else 4)
            kvc.kvc_pool_set_scales(self.pool, 0, self.scales[0].contiguous(), self.scales[1].contiguous())
        self.bt = torch.from_numpy(self.table).cuda()
        self.len_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = (torch.randn((len(lens), H_Q, D), generator=g, device="cuda") * 2).to(torch.bfloat16)
        self.scale = D ** -0.5
        self.ws = kvc.kvc_mod_workspace(self.pool, len(lens), H_Q, self.table.shape[1])
        self.e4m3 = torch.from_numpy(e4m3_table()).cuda()

    def kv(self, b, n):
        """fp64 [2, H_KV, n, D]"""
        ids = self.bt[b, :-(-n // 16)].long()
        x = self.pool.bytes_view().view(*self.shape, -1)[ids]
        if self.dtype == "bf16":
            x = x.view(torch.bfloat16).double()
        elif self.dtype == "fp8":
            x = self.e4m3[x.long()]
        else:
            x = torch.stack([(x & 15).double() - 8, (x >> 4).double() - 8], -1).flatten(-2)
        x = x.permute(2, 1, 0, 3, 4).reshape(2, self.H_KV, -1, self.D)[:, :, :n]
        return x if self.scales is None else x * self.scales.double()[:, :, None]

    def decode(self, m, workspace="own"):
        n = len(self.lens)
        out = torch.full((n, self.H_Q, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, self.H_Q), float("nan"), device="cuda")
        slopes = None if m.alibi is None else torch.tensor(m.alibi, dtype=torch.float32, device="cuda")
        mod = self.kvc.ScoreMod(m.softcap, m.window, m.sink, m.prefix, slopes)
        before = self.kvc.kvc_launch_count()
        self.kvc.kvc_decode_attn_mod(self.pool, 0, self.q, self.bt, self.len_t, out, lse, mod=mod, scale=self.scale,
                                     workspace=self.ws if isinstance(workspace, str) else workspace)
        self.launches = self.kvc.kvc_launch_count() - before
        return out, lse

    def check(self, out, lse, m):
        """Every row within the bounds of mod_reference.attend (the same terms, on the device), and two more.

        bf16 pools, capped scores: in tiles that a row does not read whole its outputs are divided by the sum of the
        rounded weights.  With weights w (1 + e), |e| <= h, and p = w / sum w, the mixture is sum p (1 + e) v over
        1 + E, E = sum p e: off by sum p (e - E) v to first order in h, and |e - E| <= 2 h.
        e4m3 and int4 pools: a weight under 2^-14 of the largest is a subnormal f16, off by half of its step, 2^-25 of
        the largest; the largest is at most sum w = L of those scaled to 1, so the mixture is off by 2^-25 sum |v| / L
        more, which shows where the values of the heavy keys are zero."""
        assert self.kvc.kvc_pool_sync_status(self.pool) == self.kvc.KVC_OK
        w_half = WEIGHTS["bf16"] * (2 if m.softcap else 1) if self.dtype == "bf16" else WEIGHTS["f16"]
        g = self.H_Q // self.H_KV
        slope = torch.zeros(self.H_Q, device="cuda", dtype=torch.float64)
        if m.alibi is not None:
            slope = torch.tensor(m.alibi, dtype=torch.float32, device="cuda").double()
        bad = []
        for b, n in enumerate(self.lens):
            o, l = out[b].double(), lse[b].double()
            if n == 0:
                if not (bool((o == 0).all()) and bool((l == -math.inf).all())):
                    bad.append(b)
                continue
            K, V = self.kv(b, n)   # [H_KV, n, D]
            t = torch.arange(n, device="cuda")
            p = n - 1
            see = t > p - m.window if m.window else t >= 0
            if m.window:
                see = see | (t < m.sink)
            see = see | (t < m.prefix)
            K, V, t = K[:, see], V[:, see], t[see]
            q = self.q[b].double().view(self.H_KV, g, self.D)
            x = self.scale * (q @ K.transpose(1, 2)).reshape(self.H_Q, -1)
            size = self.scale * (q.abs() @ K.abs().transpose(1, 2)).reshape(self.H_Q, -1).amax(-1)
            if m.softcap:
                x = m.softcap * torch.tanh(x / m.softcap)
            away = (p - t).double()
            x = x - slope[:, None] * away
            top = x.amax(-1, keepdim=True)
            w = torch.exp(x - top)
            L = w.sum(-1, keepdim=True)
            w = w / L
            wg = w.view(self.H_KV, g, -1)
            ro, mix = (wg @ V).reshape(self.H_Q, -1), (wg @ V.abs()).reshape(self.H_Q, -1)
            rl = (top + torch.log(L)).squeeze(-1)
            ds = (self.D + 8) * 2.0 ** -23 * size
            if self.dtype != "bf16":
                ds = ds + HALF["f16"] * size
            if m.softcap:
                ds = ds + 8 * m.softcap * 2.0 ** -23
            ds = ds + 4 * 2.0 ** -23 * (x.abs().amax(-1) + away.max() * slope.abs())
            terms = min(int(t.numel()), 4096)
            rel = (2 * torch.expm1(ds) + w_half + (16 + terms) * 2.0 ** -23)[:, None]
            off = rel * mix
            if self.dtype != "bf16":
                off = off + 2.0 ** -25 * V.abs().sum(1).repeat_interleave(g, 0) / L
            to = HALF["bf16"] * (ro.abs() + off) + off + 2.0 ** -130
            tl = torch.expm1(ds) + (16 + terms) * 2.0 ** -23 + 4 * 2.0 ** -24 * rl.abs()
            if not (bool(((o - ro).abs() <= to).all()) and bool(((l - rl).abs() <= tl).all())):
                bad.append(b)
        assert not bad, f"rows {bad} of {len(self.lens)}"

    def close(self):
        self.pool.close()


def spread(B, longest, seed=7):
    """Lengths spread over their logarithm, 1 .. longest."""
    r = np.random.default_rng(seed)
    return [longest] + [max(1, int(round(math.exp(r.uniform(0.0, math.log(longest)))))) for _ in range(B - 1)]


def mods(H):
    alibi = [2.0 ** (-8.0 * (i + 1) / H) for i in range(H)]
    return {"cap": Mod(softcap=5.0), "plain": Mod(), "cap_window_sink_alibi": Mod(softcap=20.0, window=700, sink=5, alibi=alibi),
            "window": Mod(softcap=50.0, window=4000)}


LENS = {"long_then_short": [8192] * 32 + [50] * 32, "in_turn": [8192, 50] * 32, "eight_long": [32768] * 8 + [50] * 24,
        "ones": [16384] * 16 + [1] * 16, "five_long": [32768] * 5 + [16] * 59, "spread": spread(64, 30000),
        "spread_with_empty": [0] + spread(40, 20000, 3) + [0, 0, 17, 0]}


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("g", [17, 20, 32])
@pytest.mark.parametrize("lens", LENS)
def test_long_sequences_beside_short_ones(kvc, lens, g, dtype):
    c = Batch(kvc, LENS[lens], H_Q=g, dtype=dtype)
    try:
        for name, m in mods(g).items():
            out, lse = c.decode(m)
            if m.window == 0:
                assert c.launches == 2, "a cut call"
            c.check(out, lse, m)
            again = c.decode(m)
            assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    finally:
        c.close()


@pytest.mark.parametrize("heads", [dict(H_Q=64, H_KV=2), dict(H_Q=64, H_KV=2, D=64), dict(H_Q=40, H_KV=2, dtype="fp8"),
                                   dict(H_Q=96, H_KV=3, dtype="int4"), dict(H_Q=24, H_KV=1, D=64)],
                         ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
def test_more_heads_and_widths(kvc, heads):
    """A head's units lie side by side on the line: a CTA's share may pass from one head to the next."""
    c = Batch(kvc, spread(24, 16000, 5) + [40] * 20, **heads)
    try:
        for m in mods(c.H_Q).values():
            c.check(*c.decode(m), m)
    finally:
        c.close()


@pytest.mark.parametrize("dtype", DT)
def test_both_sides_of_the_cut(kvc, dtype):
    """Batches of growing size: cut while few, dealt whole once they fill the SMs; the split kernel (no workspace)
    holds the same bounds."""
    seen = set()
    for B in (3, 20, 60, 76, 77, 120, 152, 153, 304, 500):
        c = Batch(kvc, spread(B, 3000, B), dtype=dtype)
        try:
            m = Mod(softcap=30.0)
            out, lse = c.decode(m)
            seen.add(c.launches)
            c.check(out, lse, m)
            if B in (20, 500):
                c.check(*c.decode(m, None), m)
        finally:
            c.close()
    assert seen == {1, 2}


MANY = {"cut": ([64] * 1376, 2), "cut_two_launches": ([1 + (7 * i) % 64 for i in range(2060)], 4),
        "whole_two_launches": ([1 + (11 * i) % 130 for i in range(2100)] + [6000] * 3, 2)}


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("many", MANY)
def test_many_short_sequences(kvc, many, dtype):
    """Sequences of a tile or two by the thousand, and more of them than one launch takes (2 048)."""
    lens, launches = MANY[many]
    c = Batch(kvc, lens, dtype=dtype)
    try:
        for m in (Mod(softcap=9.0), Mod(softcap=9.0, window=60), Mod(window=33, sink=2)):
            out, lse = c.decode(m)
            if not m.window:
                assert c.launches == launches
            c.check(out, lse, m)
    finally:
        c.close()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lens", [[8192, 50] * 16, [40] * 30], ids=["cut", "whole"])
def test_expired_waits_are_reported(kvc, monkeypatch, lens, dtype):
    """With every load withheld (a test hook) a cut call and a whole one report KVC_ERR_TIMEOUT and return, both chains
    of every CTA together; with a fresh workspace the pool then works."""
    c = Batch(kvc, lens, dtype=dtype)
    try:
        m = Mod(softcap=10.0)
        monkeypatch.setenv("KVC_TEST_STALL", "1")
        c.decode(m)
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_ERR_TIMEOUT
        monkeypatch.delenv("KVC_TEST_STALL")
        c.ws.zero_()
        c.check(*c.decode(m), m)
    finally:
        c.close()
