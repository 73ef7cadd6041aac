"""Cases and plain forms of the rotary write and modified-score attention operators.

Three operators of a paged key/value cache, each with a plain form in
elementary torch operations (fp32, fp64 for angles) and, where ``own`` is true,
the library's calls:

  rope     q, k of new tokens optionally RMS-normalised per head, rotated by
           position, k and v stored into the paged pool (``kvc_rope_append`` for
           one token per sequence, ``kvc_rope_write_tokens`` for ragged runs)
  decode   attention of one new token per sequence over its cached positions,
           with tanh-capped scores, a distance bias, a sliding window with
           leading sink positions (``kvc_decode_attn_mod``)
  prefill  causal attention of a chunk of one sequence with the same
           modifiers, a bidirectional prefix or packed documents
           (``kvc_prefill_attn_mod``)
"""
import math
import random

import numpy as np
import torch

own = False

BS = 16   # positions per cache block
DEV = "cuda"
BITS = {"bf16": 16, "fp8": 8, "int4": 4}

ROPE = dict(op="rope", mode="append", B=1, tokens=1, H_Q=32, H_KV=8, D=128, dtype="bf16", rotary=128,
            interleaved=False, norm=False, far=8192)
DECODE = dict(op="decode", B=4, len_max=256, ragged=False, H_Q=32, H_KV=8, D=128, dtype="bf16", softcap=0.0,
              window=0, sink=0, alibi=False)
PREFILL = dict(op="prefill", n_q=600, q_start=1200, H_Q=32, H_KV=8, D=128, dtype="bf16", softcap=0.0, window=0,
               sink=0, prefix=0, alibi=False, doc_len=0)


def listed():
    return [
        # a single user's decode step: what counts is latency
        dict(ROPE, name="rope append, 1 sequence"),
        # a serving batch with normalised queries and keys, an e4m3 cache and long contexts
        dict(ROPE, name="rope append, 64 sequences", B=64, tokens=64, dtype="fp8", norm=True, far=131072),
        # prompts of several requests written in one call; half of each head rotates
        dict(ROPE, name="rope write, ragged prompts", mode="write", B=24, tokens=16384, rotary=64, norm=True,
             far=16384),
        # the tiny layer: launch latency
        dict(DECODE, name="decode tiny, capped", B=4, len_max=256, ragged=True, H_Q=8, H_KV=2, D=64, softcap=50.0),
        # a full batch at 8k context with capped scores
        dict(DECODE, name="decode gqa, capped", B=32, len_max=8193, softcap=50.0),
        # ragged lengths, a sliding window and sink positions: most of the cache is not read
        dict(DECODE, name="decode ragged, window", B=64, len_max=32768, ragged=True, window=4096, sink=4),
        # distance bias, a key head for each query head, e4m3
        dict(DECODE, name="decode mha e4m3, alibi", B=8, len_max=8000, H_KV=32, dtype="fp8", alibi=True),
        # one key head for 32 query heads, 4-bit cache
        dict(DECODE, name="decode mqa int4, capped", B=8, len_max=32768, H_KV=1, dtype="int4", softcap=30.0),
        # a chunk of a prompt behind a shared prefix
        dict(PREFILL, name="prefill chunk, capped", softcap=50.0),
        # a few drafted tokens verified against a long cache: few rows, a long axis
        dict(PREFILL, name="prefill 5 of 20005, capped", n_q=5, q_start=20000, softcap=50.0),
        # short documents packed into one prompt, distance bias, e4m3
        dict(PREFILL, name="prefill documents e4m3, alibi", n_q=2000, q_start=48, dtype="fp8", alibi=True,
             doc_len=333),
        # a long prompt's late chunk: compute-bound
        dict(PREFILL, name="prefill 2048 of 18432, capped", n_q=2048, q_start=16384, softcap=50.0),
    ]


HEADS = [(32, 8, 128), (32, 32, 128), (32, 1, 128), (8, 2, 64), (24, 8, 64), (40, 8, 128), (12, 4, 128)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _kv_bytes(c, positions):
    return 2 * positions * c["H_KV"] * c["D"] * BITS[c["dtype"]] // 8


def draw(rng):
    """One more case of the ranges above: tokens 1 to 16384, contexts 1 to 32768, chunks 1 to 2048."""
    op = rng.choice(["rope", "decode", "prefill"])
    H_Q, H_KV, D = rng.choice(HEADS)
    if op == "rope":
        c = dict(ROPE, mode=rng.choice(["append", "write"]), H_Q=H_Q, H_KV=H_KV, D=D, norm=rng.random() < 0.5,
                 interleaved=rng.random() < 0.4, far=_log(rng, 64, 131072),
                 dtype=rng.choice(["bf16", "bf16", "fp8"]) if D == 128 else "bf16")
        c["rotary"] = rng.choice([D, D, D // 2, 16 * rng.randint(1, D // 16)])
        c["B"] = _log(rng, 1, 256) if c["mode"] == "append" else _log(rng, 1, 32)
        per_token = 2 * D * (2 * H_Q + 3 * H_KV)
        most = min(16384, 350_000_000 // per_token)
        c["tokens"] = c["B"] if c["mode"] == "append" else _log(rng, 1, most)
        return c
    dtype = rng.choice(["bf16", "bf16", "fp8", "int4"]) if D == 128 else "bf16"
    mods = dict(softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.3)
    if op == "decode":
        c = dict(DECODE, H_Q=H_Q, H_KV=H_KV, D=D, dtype=dtype, B=_log(rng, 1, 64), len_max=_log(rng, 1, 32768),
                 ragged=rng.random() < 0.5, **mods)
        if rng.random() < 0.4:
            c.update(window=_log(rng, 1, 8192), sink=rng.choice([0, 4, 37]))
        while _kv_bytes(c, c["B"] * c["len_max"]) > 1_000_000_000 or c["B"] * c["len_max"] * max(H_KV, 8) > 16_000_000:
            c["len_max"] = (c["len_max"] * 2) // 3
        return c
    c = dict(PREFILL, H_Q=H_Q, H_KV=H_KV, D=D, dtype=dtype, n_q=_log(rng, 1, 2048),
             q_start=rng.choice([0, _log(rng, 1, 16000)]), **mods)
    shape = rng.choice(["causal", "window", "prefix", "documents"])
    if shape == "window":
        c.update(window=_log(rng, 1, 4096), sink=rng.choice([0, 4, 37]))
    elif shape == "prefix":
        c.update(prefix=_log(rng, 1, c["q_start"] + c["n_q"]))
    elif shape == "documents":
        c.update(doc_len=_log(rng, 1, 2048))
    while 4 * c["n_q"] * (c["q_start"] + c["n_q"]) * H_Q * D > 550_000_000_000:
        c["q_start"] = c["q_start"] // 2
    return c


# ------------------------------------------------------------------ layout of a case (the same for every seed)
def _lens(c):
    """Cached positions of each decode sequence; a ragged batch of 8 or more holds one empty sequence."""
    if not c["ragged"]:
        return [c["len_max"]] * c["B"]
    r = random.Random(c["B"] * 1000003 + c["len_max"])
    lens = [c["len_max"]] + [_log(r, max(1, c["len_max"] // 256), c["len_max"]) for _ in range(c["B"] - 1)]
    if c["B"] >= 8:
        lens[3] = 0
    return lens


def _runs(c):
    """(first position, tokens) of each sequence of a rope case."""
    r = random.Random(c["B"] * 7919 + c["tokens"])
    starts = [_log(r, 1, c["far"]) - 1 for _ in range(c["B"])]
    if c["mode"] == "append":
        return [(s, 1) for s in starts]
    cuts = sorted(r.randint(0, c["tokens"]) for _ in range(c["B"] - 1))
    edges = [0] + cuts + [c["tokens"]]
    return [(s, b - a) for s, a, b in zip(starts, edges, edges[1:])]


def _visible(c, i):
    """Positions that query i of a prefill case reads."""
    p = c["q_start"] + i
    total = c["q_start"] + c["n_q"]
    d = (p // c["doc_len"]) * c["doc_len"] if c["doc_len"] else 0
    lo = max(d, p - c["window"] + 1) if c["window"] else d
    n = p + 1 - lo
    lead = max(min(d + c["sink"], lo) - d, 0) if c["window"] else 0
    if c["prefix"]:
        e = min(c["prefix"], total)
        return max(e, p + 1) - lo + lead if lo < e else n + max(e, lead)
    return n + lead


def work(case):
    c = case
    if c["op"] == "rope":
        T, D = c["tokens"], c["D"]
        nb = T * D * (2 * (2 * c["H_Q"] + 2 * c["H_KV"]) + 2 * c["H_KV"] * BITS[c["dtype"]] // 8) + 4 * c["rotary"] // 2
        return {"bytes": nb, "flops": T * D * (c["H_Q"] + c["H_KV"]) * (8 if c["norm"] else 3)}
    row = c["H_Q"] * c["D"]
    if c["op"] == "decode":
        w = c["window"] or (1 << 30)
        seen = [min(n, w) + max(0, min(c["sink"], n - w)) for n in _lens(c)]
        return {"bytes": _kv_bytes(c, sum(seen)) + sum(-(-n // BS) for n in seen) * 4 + c["B"] * row * 4,
                "flops": 4 * sum(seen) * row}
    total = c["q_start"] + c["n_q"]
    first = 0
    if c["doc_len"]:
        first = (c["q_start"] // c["doc_len"]) * c["doc_len"]
    if c["window"] and not c["sink"]:
        first = max(first, c["q_start"] - c["window"] + 1)
    return {"bytes": _kv_bytes(c, total - first) + c["n_q"] * row * 4,
            "flops": 4 * sum(_visible(c, i) for i in range(c["n_q"])) * row}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _filled_pool(c, g, blocks):
    """A pool's bytes [blocks, H_KV, 2, 16, row bytes] holding normal keys and values, and its scales."""
    shape = (blocks, c["H_KV"], 2, BS, c["D"])
    n = math.prod(shape)
    if c["dtype"] == "bf16":
        data = torch.empty(n, device=DEV, dtype=torch.bfloat16)
        for a in range(0, n, 1 << 28):
            m = min(1 << 28, n - a)
            data[a:a + m] = torch.randn(m, generator=g, device=DEV, dtype=torch.bfloat16)
        return data.view(shape), None
    scales = torch.rand((2, c["H_KV"], c["D"]), generator=g, device=DEV) + 0.5
    if c["dtype"] == "fp8":
        data = torch.empty(n, device=DEV, dtype=torch.float8_e4m3fn)
        for a in range(0, n, 1 << 28):
            m = min(1 << 28, n - a)
            data[a:a + m] = (torch.randn(m, generator=g, device=DEV) * 96).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return data.view(shape), scales / 96
    data = torch.empty(n // 2, device=DEV, dtype=torch.uint8)
    for a in range(0, n // 2, 1 << 27):
        m = min(1 << 27, n // 2 - a)
        code = (torch.randn((m, 2), generator=g, device=DEV) * 2).round_().clamp_(-7, 7).to(torch.uint8) + 8
        code &= 15
        data[a:a + m] = code[:, 0] | (code[:, 1] << 4)
    return data.view(shape[:-1] + (c["D"] // 2,)), scales / 2


def _slopes(c):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / c["H_Q"]) for i in range(c["H_Q"])], device=DEV)


def _inv_freq(c):
    r = c["rotary"]
    return torch.tensor([500000.0 ** (-2.0 * i / r) for i in range(r // 2)], device=DEV, dtype=torch.float32)


def _inputs(c, seed):
    g = _gen(seed)
    s = {"case": c}
    H_Q, H_KV, D = c["H_Q"], c["H_KV"], c["D"]
    if c["op"] == "rope":
        runs, T = _runs(c), c["tokens"]
        # the fused projection's output, of which q, k and v are strided views
        s["qkv"] = (_normal(g, T, (H_Q + 2 * H_KV) * D) * (2.0 if c["norm"] else 1.0)).to(torch.bfloat16)
        mb = max(-(-(a + n) // BS) for a, n in runs)
        used = [(b, j) for b, (a, n) in enumerate(runs) for j in range(a // BS, -(-(a + n) // BS)) if n]
        blocks = len(used) + 3
        perm = torch.randperm(blocks, generator=torch.Generator().manual_seed(int(seed)))[:len(used)].numpy()
        table = np.full((len(runs), mb), -1, dtype=np.int32)   # blocks of earlier positions do not matter here
        for (b, j), p in zip(used, perm):
            table[b, j] = p
        s["table"] = torch.from_numpy(table).to(DEV)
        s["start"] = torch.tensor([a for a, _ in runs], device=DEV, dtype=torch.int32)
        s["cu"] = torch.tensor([0] + list(np.cumsum([n for _, n in runs])), device=DEV, dtype=torch.int32)
        s["inv_freq"] = _inv_freq(c)
        s["q_norm"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16) if c["norm"] else None
        s["k_norm"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16) if c["norm"] else None
        s["pool"], s["scales"] = _filled_pool(c, g, blocks)
        return s
    if c["op"] == "decode":
        lens = _lens(c)
        rows = c["B"]
    else:
        lens = [c["q_start"] + c["n_q"]]
        rows = c["n_q"]
    mb = max(1, max(-(-n // BS) for n in lens))
    need = sum(-(-n // BS) for n in lens)
    perm = torch.randperm(need + 2, generator=torch.Generator().manual_seed(int(seed)))[:need].numpy().astype(np.int32)
    table = np.full((len(lens), mb), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // BS)
        table[b, :k] = perm[at:at + k]
        at += k
    s["table"] = torch.from_numpy(table).to(DEV)
    s["row"] = s["table"][0]
    s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    # queries of the size that a trained head has: scores with a spread of a few units
    s["q"] = (_normal(g, rows, H_Q, D) * 2.0).to(torch.bfloat16)
    s["alibi"] = _slopes(c) if c["alibi"] else None
    s["doc_start"] = None
    if c.get("doc_len"):
        p = torch.arange(c["q_start"], c["q_start"] + rows, device=DEV, dtype=torch.int32)
        s["doc_start"] = (p // c["doc_len"]) * c["doc_len"]
    s["pool"], s["scales"] = _filled_pool(c, g, need + 2)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case
    if c["op"] == "rope":
        q, k, v = s["qkv"].split([c["H_Q"] * c["D"], c["H_KV"] * c["D"], c["H_KV"] * c["D"]], dim=1)
        s["q"], s["k"], s["v"] = (x.view(c["tokens"], -1, c["D"]) for x in (q, k, v))
        s["q_out"] = torch.empty((c["tokens"], c["H_Q"], c["D"]), device=DEV, dtype=torch.bfloat16)
    else:
        s["out"] = torch.empty(s["q"].shape, device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.empty(s["q"].shape[:2], device=DEV) if c["dtype"] == "bf16" else None
    if own:
        import paged_kv_cache_kvc_gb300 as kvc
        dt = {"bf16": kvc.KVC_BF16, "fp8": kvc.KVC_FP8_E4M3, "int4": kvc.KVC_INT4}[c["dtype"]]
        s["kvc"] = kvc
        data = s["pool"]
        pool = kvc.kvc_pool_create(data.shape[0], BS, 1, c["H_KV"], c["D"], dt)
        pool.bytes_view().copy_(data.view(-1).view(torch.uint8))
        if s["scales"] is not None:
            kvc.kvc_pool_set_scales(pool, 0, s["scales"][0].contiguous(), s["scales"][1].contiguous())
        s["handle"] = pool
        s["pool"] = pool.bytes_view().view(data.dtype).view(data.shape)
        s["pool"].handle = pool   # the view does not own the pool's memory: keep the pool while it is in use
        if c["op"] == "rope":
            s["rope"] = kvc.Rope(s["inv_freq"], interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                                 eps=1e-6)
        else:
            s["mod"] = kvc.ScoreMod(softcap=c["softcap"], window=c["window"], sink=c["sink"],
                                    prefix=c.get("prefix", 0), alibi=s["alibi"], doc_start=s["doc_start"])
            s["workspace"] = kvc.kvc_mod_workspace(pool, s["q"].shape[0], c["H_Q"], s["table"].shape[1])
    return s


# ------------------------------------------------------------------ plain forms
def _rotated(s, x, weight, pos):
    """x [T, H, D] RMS-normalised (with a weight) and rotated by its positions, fp32."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = c["rotary"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rope(s):
    c = s["case"]
    T = c["tokens"]
    row = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), row.int(), right=True)
    pos = s["start"][seq].long() + row - s["cu"][seq].long()
    block = s["table"][seq, pos // BS].long()
    q = _rotated(s, s["q"], s["q_norm"], pos).to(torch.bfloat16)
    k = _rotated(s, s["k"], s["k_norm"], pos)
    v = s["v"]
    if c["dtype"] == "fp8":
        k = (k / s["scales"][0]).clamp(-448, 448)
        v = (v.float() / s["scales"][1]).clamp(-448, 448)
    kv = torch.stack([k.to(s["pool"].dtype), v.to(s["pool"].dtype)], 2)   # [T, H_KV, 2, D]
    raw = {2: torch.int16, 1: torch.uint8}[kv.element_size()]
    s["pool"].view(raw)[block, :, :, pos % BS] = kv.view(raw)
    return [q, s["pool"]]


def _cached(s):
    """Keys and values of every table row, fp32 [rows, H_KV, positions, D] each."""
    c = s["case"]
    x = s["pool"][s["table"].clamp(min=0).long()]   # [rows, blocks, H_KV, 2, 16, row]
    if c["dtype"] == "int4":
        x = torch.stack([(x & 15).to(torch.int8) - 8, (x >> 4).to(torch.int8) - 8], -1).flatten(-2)
    rows, blocks = x.shape[:2]
    k, v = (x[:, :, :, i].float().transpose(1, 2).reshape(rows, c["H_KV"], blocks * BS, c["D"]) for i in (0, 1))
    if s["scales"] is not None:
        k, v = k * s["scales"][0][:, None], v * s["scales"][1][:, None]
    return k, v


def _mix(c, scores, seen, bias, v):
    """softmax over the seen positions of the modified scores, times v: (out bf16, lse)."""
    if c["softcap"]:
        scores = c["softcap"] * torch.tanh(scores / c["softcap"])
    if bias is not None:
        scores = scores - bias
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return out, (m + torch.log(total)).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    B, g = c["B"], c["H_Q"] // c["H_KV"]
    k, v = _cached(s)
    t = torch.arange(k.shape[2], device=DEV)
    n = s["lens"].long()[:, None]
    seen = t < n
    if c["window"]:
        seen &= (t >= n - c["window"]) | (t < c["sink"])
    seen = seen[:, None, None]
    bias = None
    if c["alibi"]:
        bias = s["alibi"].view(c["H_KV"], g, 1) * (n - 1 - t)[:, None, None].float()
    q = s["q"].float().view(B, c["H_KV"], g, c["D"])
    scores = (q @ k.transpose(2, 3)) * c["D"] ** -0.5
    out, lse = _mix(c, scores, seen, bias, v)
    out = out.reshape(B, c["H_Q"], c["D"]).to(torch.bfloat16)
    return [out, lse.reshape(B, c["H_Q"])] if s["lse"] is not None else [out]


def _plain_prefill(s):
    c = s["case"]
    n_q, g = c["n_q"], c["H_Q"] // c["H_KV"]
    k, v = _cached(s)
    k, v = k[0, :, :c["q_start"] + n_q], v[0, :, :c["q_start"] + n_q]
    t = torch.arange(k.shape[1], device=DEV)
    p = torch.arange(c["q_start"], c["q_start"] + n_q, device=DEV)[:, None]
    seen = t <= p
    if c["window"]:
        near = t > p - c["window"]
        if c["sink"]:
            first = s["doc_start"].long()[:, None] if c["doc_len"] else 0
            near = near | (t < first + c["sink"])
        seen = seen & near
    if c["prefix"]:
        seen = seen | (t < c["prefix"])
    if c["doc_len"]:
        seen = seen & (t >= s["doc_start"].long()[:, None])
    bias = None
    if c["alibi"]:
        bias = s["alibi"].view(c["H_KV"], g, 1, 1) * (p - t).abs().float()
    q = s["q"].float().view(n_q, c["H_KV"], g, c["D"]).permute(1, 2, 0, 3)
    scores = (q @ k.transpose(1, 2)[:, None]) * c["D"] ** -0.5
    out, lse = _mix(c, scores, seen, bias, v[:, None])
    out = out.permute(2, 0, 1, 3).reshape(n_q, c["H_Q"], c["D"]).to(torch.bfloat16)
    return [out, lse.permute(2, 0, 1).reshape(n_q, c["H_Q"])] if s["lse"] is not None else [out]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rope": _plain_rope, "decode": _plain_decode, "prefill": _plain_prefill}[c["op"]](s)
    kvc = s["kvc"]
    if c["op"] == "rope":
        if c["mode"] == "append":
            kvc.kvc_rope_append(s["handle"], 0, s["table"], s["start"], s["q"], s["k"], s["v"], s["q_out"], s["rope"])
        else:
            kvc.kvc_rope_write_tokens(s["handle"], 0, s["table"], s["start"], s["cu"], s["q"], s["k"], s["v"],
                                      s["q_out"], s["rope"])
        return [s["q_out"], s["pool"]]
    if c["op"] == "decode":
        kvc.kvc_decode_attn_mod(s["handle"], 0, s["q"], s["table"], s["lens"], s["out"], s["lse"], mod=s["mod"],
                                workspace=s["workspace"])
    else:
        kvc.kvc_prefill_attn_mod(s["handle"], 0, s["q"], s["row"], c["q_start"], s["out"], s["lse"],
                                 mod=s["mod"], workspace=s["workspace"])
    return [s["out"], s["lse"]] if s["lse"] is not None else [s["out"]]


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_values():
    """The 256 values of the 8-bit format with 4 exponent and 3 fraction bits, bias 7, no infinities."""
    table = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        x = math.nan if (code & 127) == 127 else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        table.append(-x if code & 128 else x)
    return torch.tensor(table, device=DEV, dtype=torch.float64)


def _stored(c, s, ids, head, kind):
    """Stored keys (kind 0) or values (1) of one head in the given blocks, fp64 [positions, D], scales applied."""
    x = s["pool"][ids, head, kind]
    if c["dtype"] == "bf16":
        y = x.double()
    elif c["dtype"] == "fp8":
        y = _e4m3_values()[x.view(torch.uint8).long()]
    else:
        b = x.long()
        y = torch.empty(b.shape[:-1] + (c["D"],), device=DEV, dtype=torch.float64)
        y[..., 0::2], y[..., 1::2] = (b % 16 - 8).double(), (b // 16 - 8).double()
    y = y.reshape(-1, c["D"])
    return y if s["scales"] is None else y * s["scales"][kind, head].double()


def _attend(c, s, q, ids, total, head, where, distance):
    """out [g, n, D] and lse [g, n] of queries q [g, n, D] (fp64) of one key head."""
    k, v = _stored(c, s, ids, head, 0)[:total], _stored(c, s, ids, head, 1)[:total]
    g = q.shape[0]
    x = torch.einsum("gnd,td->gnt", q, k) / math.sqrt(c["D"])
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    if c["alibi"]:
        x -= s["alibi"].double()[head * g:(head + 1) * g, None, None] * distance
    x = torch.where(where, x, torch.full((), -math.inf, device=DEV, dtype=torch.float64))
    lse = torch.logsumexp(x, -1)
    weight = torch.exp(x - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    return torch.einsum("gnt,td->gnd", weight, v), lse


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    H_Q, H_KV, D = c["H_Q"], c["H_KV"], c["D"]
    g = H_Q // H_KV
    if c["op"] == "rope":
        x = s["qkv"].double().view(c["tokens"], H_Q + 2 * H_KV, D)
        runs = _runs(c)
        pos = torch.cat([torch.arange(a, a + n) for a, n in runs]).to(DEV)
        seq = torch.cat([torch.full((n,), b) for b, (a, n) in enumerate(runs)]).to(DEV)
        y = x.clone()
        for lo, hi, w in ((0, H_Q, s["q_norm"]), (H_Q, H_Q + H_KV, s["k_norm"])):
            if w is not None:
                y[:, lo:hi] = x[:, lo:hi] / torch.sqrt((x[:, lo:hi] ** 2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        half = c["rotary"] // 2
        i = torch.arange(half, device=DEV)
        i0, i1 = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.polar(torch.ones((), device=DEV, dtype=torch.float64),
                        pos.double()[:, None, None] * s["inv_freq"].double())
        u = torch.complex(y[:, :H_Q + H_KV][..., i0], y[:, :H_Q + H_KV][..., i1]) * z
        y[:, :H_Q + H_KV, i0], y[:, :H_Q + H_KV, i1] = u.real, u.imag
        pool = _e4m3_values()[s["pool"].view(torch.uint8).long()] if c["dtype"] == "fp8" else s["pool"].double()
        ids = s["table"][seq, pos // BS].long()
        for kind in (0, 1):
            kv = y[:, H_Q + kind * H_KV:H_Q + (kind + 1) * H_KV]
            if s["scales"] is not None:
                kv = torch.clamp(kv / s["scales"][kind].double(), -448, 448)
            pool[ids, :, kind, pos % BS] = kv
        return [y[:, :H_Q].contiguous(), pool]
    q = s["q"].double()
    out = torch.zeros(q.shape, device=DEV, dtype=torch.float64)
    lse = torch.zeros(q.shape[:2], device=DEV, dtype=torch.float64)
    if c["op"] == "decode":
        for b, n in enumerate(_lens(c)):
            t = torch.arange(n, device=DEV)
            where = (t < c["sink"]) | (t > n - 1 - c["window"]) if c["window"] else t >= 0
            for h in range(H_KV):
                if n == 0:
                    lse[b] = -math.inf
                    continue
                o, l = _attend(c, s, q[b, h * g:(h + 1) * g, None], s["table"][b, :-(-n // BS)].long(), n, h, where,
                               (n - 1 - t).double())
                out[b, h * g:(h + 1) * g], lse[b, h * g:(h + 1) * g] = o[:, 0], l[:, 0]
    else:
        total = c["q_start"] + c["n_q"]
        t = torch.arange(total, device=DEV)[None]
        p = c["q_start"] + torch.arange(c["n_q"], device=DEV)[:, None]
        first = p - p % c["doc_len"] if c["doc_len"] else torch.zeros_like(p)
        behind = p - t
        where = (behind >= 0) & (t >= first)
        if c["window"]:
            where &= (behind < c["window"]) | (t - first < c["sink"])
        if c["prefix"]:
            where |= t < c["prefix"]
        for h in range(H_KV):
            o, l = _attend(c, s, q[:, h * g:(h + 1) * g].transpose(0, 1), s["table"][0].long(), total, h, where,
                           behind.abs().double())
            out[:, h * g:(h + 1) * g], lse[:, h * g:(h + 1) * g] = o.transpose(0, 1), l.transpose(0, 1)
    return [out, lse if c["dtype"] == "bf16" else None]
