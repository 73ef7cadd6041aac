"""Attention with modified scores that writes its outputs over its queries, and the overlaps that are refused."""
import numpy as np
import pytest
import torch

from mod_reference import Mod
from test_gpu_mod import Rows

pytestmark = pytest.mark.gpu

HEADS = [dict(H_Q=8, H_KV=2), dict(H_Q=16, H_KV=1, D=64), dict(H_Q=32, H_KV=1), dict(H_Q=8, H_KV=2, dtype="fp8"),
         dict(H_Q=32, H_KV=1, dtype="int4")]
ids = ["-".join(f"{k}{v}" for k, v in h.items()) for h in HEADS]


@pytest.mark.parametrize("heads", HEADS, ids=ids)
@pytest.mark.parametrize("workspace", [True, False])
def test_decode_over_its_queries(kvc, heads, workspace):
    """Batches whose sequences are split and merged (in the kernel, after it), cut, and dealt whole."""
    for lens in ([9000, 40, 0, 3000], [700] * 40 + [2100], [60] * 200, [8000] * 5 + [30] * 30):
        c = Rows(kvc, lens, layers=1, layer=0, **heads)
        try:
            ws = kvc.kvc_mod_workspace(c.pool, len(lens), c.H_Q, c.table.shape[1]) if workspace else None
            for m in (Mod(softcap=7.0), Mod(window=90, sink=3)):
                want = c.decode(m, ws)
                out, lse = c.q.clone(), torch.empty_like(want[1])
                kvc.kvc_decode_attn_mod(c.pool, 0, out, c.bt, c.len_t, out, lse, mod=c.dev_mod(m), scale=c.scale, workspace=ws)
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        finally:
            c.close()


@pytest.mark.parametrize("heads", HEADS, ids=ids)
@pytest.mark.parametrize("tensor_memory", [True, False])
def test_prefill_over_its_queries(kvc, monkeypatch, heads, tensor_memory):
    if not tensor_memory:
        monkeypatch.setenv("KVC_TC", "0")
    c = Rows(kvc, [3000], layers=1, layer=0, **heads)
    try:
        for q_start, n_q in ((2990, 5), (1000, 300), (0, 1500), (37, 1)):
            for m in (Mod(softcap=7.0), Mod(doc_start=(np.arange(q_start, q_start + n_q) // 61) * 61)):
                q = c.queries(n_q)
                ws = kvc.kvc_mod_workspace(c.pool, n_q, c.H_Q, c.table.shape[1])
                want = c.prefill(m, q, q_start, workspace=ws)
                out, lse = q.clone(), torch.empty_like(want[1])
                kvc.kvc_prefill_attn_mod(c.pool, 0, out, c.bt[0].contiguous(), q_start, out, lse, mod=c.dev_mod(m), scale=c.scale, workspace=ws)
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    finally:
        c.close()


def test_shifted_outputs_are_refused(kvc):
    c = Rows(kvc, [100] * 4, layers=1, layer=0)
    try:
        buf = torch.zeros(9, c.H_Q, c.D, dtype=torch.bfloat16, device="cuda")
        row = c.bt[0].contiguous()
        for q, out in ((buf[:4], buf[1:5]), (buf[1:5], buf[:4]), (buf[3:7], buf[:4]), (buf[:4], buf[3:7])):
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_decode_attn_mod(c.pool, 0, q, c.bt, c.len_t, out)
            assert e.value.status == kvc.KVC_ERR_ARG
            with pytest.raises(kvc.KvcError) as e:
                kvc.kvc_prefill_attn_mod(c.pool, 0, q, row, 96, out)
            assert e.value.status == kvc.KVC_ERR_ARG
        torch.cuda.synchronize()
        assert not bool(buf.any())   # nothing ran
        kvc.kvc_decode_attn_mod(c.pool, 0, buf[:4], c.bt, c.len_t, buf[4:8])   # side by side
        torch.cuda.synchronize()
        assert kvc.kvc_pool_sync_status(c.pool) == kvc.KVC_OK and bool(buf[4:8].any()) and not bool(buf[8].any())
    finally:
        c.close()
