"""Calls that follow kvc_mixed_step directly on its stream start after both of its parts have ended.

The chunk of a mixed step runs beside the decode step without waiting for it, and may have done its work long before; a
call behind it that writes what the decode step still reads (the pool, its queries) has to wait for both."""
import pytest
import torch

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, B, CTX = 32, 8, 128, 48, 8000


@pytest.mark.parametrize("then", ["rope_append", "rope_write", "decode_step"])
def test_a_call_after_the_mixed_step_waits_for_its_decode(kvc, then):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    mb = CTX // 16 + 1
    pool = kvc.kvc_pool_create(B * mb + 8, 16, 1, H_KV, D)
    try:
        pool.bytes_view().view(torch.bfloat16).normal_(generator=g)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        bt = torch.arange(B * mb, device="cuda", dtype=torch.int32).view(B, mb)
        chunk_row = torch.arange(B * mb, B * mb + 4, device="cuda", dtype=torch.int32)
        lens = torch.full((B,), CTX, device="cuda", dtype=torch.int32)
        q, k, v, chunk_q = rnd(B, H_Q, D), rnd(B, H_KV, D), rnd(B, H_KV, D), rnd(16, H_Q, D)
        k2, v2 = rnd(B, H_KV, D), 100 * rnd(B, H_KV, D)
        rope = kvc.Rope(torch.full((64,), 0.3, device="cuda"))
        last = lens - 1        # positions that the decode step reads, in its last blocks
        cu = torch.arange(B + 1, device="cuda", dtype=torch.int32)
        kvc.kvc_pool_reserve(pool, B, H_Q, mb)
        saved = pool.bytes_view().clone()

        def run(wait):
            pool.bytes_view().copy_(saved)
            qq, out, o2 = q.clone(), torch.empty((B, H_Q, D), device="cuda"), torch.empty((B, H_Q, D), device="cuda")
            chunk = torch.empty((16, H_Q, D), device="cuda")
            torch.cuda.synchronize()
            kvc.kvc_mixed_step(pool, 0, qq, bt, lens, k, v, out, None, chunk_q, chunk_row, 0, chunk)
            if wait:
                torch.cuda.synchronize()
            if then == "rope_append":      # in place: the decode step's queries and the values that it reads
                kvc.kvc_rope_append(pool, 0, bt, last, qq, k2, v2, qq, rope)
            elif then == "rope_write":
                kvc.kvc_rope_write_tokens(pool, 0, bt, last, cu, qq, k2, v2, qq, rope)
            else:                          # the same workspace, the same rows
                kvc.kvc_decode_step(pool, 0, qq, bt, last, k2, v2, o2)
            torch.cuda.synchronize()
            assert kvc.kvc_pool_sync_status(pool) == kvc.KVC_OK
            return out, chunk, qq, pool.bytes_view().clone(), o2 if then == "decode_step" else out

        want = run(True)
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(run(False), want))
    finally:
        pool.close()
