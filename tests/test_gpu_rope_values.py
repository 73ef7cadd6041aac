"""The rotary write on values and weights that are not finite: they stay in the channels that they belong to."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [0, 48])
@pytest.mark.parametrize("rows", [3, 700, 2000])
def test_channels_past_the_rotation_keep_to_themselves(kvc, R, rows, interleaved):
    """A norm weight or an element that is not finite, in a channel at or past R, shows in that channel alone (an
    element also through its row's norm, where there is one)."""
    D, H_Q, H_KV = 128, 4, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    pool = kvc.kvc_pool_create(-(-rows // 16), 16, 1, H_KV, D)
    try:
        bt = torch.arange(-(-rows // 16), device="cuda", dtype=torch.int32)[None]
        zero, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        rnd = lambda h: torch.randn((rows, h, D), generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = rnd(H_Q), rnd(H_KV), rnd(H_KV)
        f = torch.full((R // 2,), 0.01, device="cuda") if R else None
        w = torch.rand(D, generator=g, device="cuda").add(0.5).to(torch.bfloat16)

        def run(qq, kk, weight):
            out = torch.empty_like(q)
            kvc.kvc_rope_write_tokens(pool, 0, bt, zero, cu, qq, kk, v, out, kvc.Rope(f, interleaved, weight, weight))
            torch.cuda.synchronize()
            assert kvc.kvc_pool_sync_status(pool) == kvc.KVC_OK
            keys = pool.bytes_view().view(torch.bfloat16).view(-1, H_KV, 2, 16, D)[:, :, 0].transpose(1, 2).reshape(-1, H_KV, D)[:rows]
            return out, keys.clone()

        for bad, at in ((float("nan"), 50), (float("inf"), 127), (float("-inf"), 72)):
            others = [c for c in range(D) if c != at]
            want = run(q, k, w)
            wb = w.clone()
            wb[at] = bad
            for a, b in zip(run(q, k, wb), want):
                assert torch.equal(a[..., others], b[..., others]) and not torch.isfinite(a[..., at]).any()
            want = run(q, k, None)
            qb, kb = q.clone(), k.clone()
            qb[..., at], kb[..., at] = bad, bad
            for a, b in zip(run(qb, kb, None), want):
                assert torch.equal(a[..., others], b[..., others]) and not torch.isfinite(a[..., at]).any()
    finally:
        pool.close()
