"""Cases and plain forms of the planned step, the rotary write by slots, and sparse attention over scored blocks.

Five operators of a paged key/value cache, each with a plain form in elementary
torch operations (fp32, fp64 for angles) and, where ``own`` is true, the
library's calls:

  plan     block tables, slot map, positions and sequence of every new token
           from the lengths that the sequences have and shall have, blocks
           taken from and returned to a free list (``kvc_plan_step``)
  axes     q, k of new tokens optionally RMS-normalised per head, rotated by
           positions with several axes, k and v stored at the slots of a slot
           map (``kvc_rope_write_slots``)
  bounds   8-bit bounds of every channel of the keys of the blocks that new
           tokens went to (``kvc_update_bounds``)
  select   for each query the blocks whose bounds allow the largest scores
           (``kvc_select_blocks``)
  attend   attention of each query over its list of blocks
           (``kvc_sparse_attn``)
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BITS = {"bf16": 16, "fp8": 8, "int4": 4}

PLAN = dict(op="plan", B=8, bs=16, far=8192, prompts=0, tokens=0, finish=0, cut=0, idle=0, short=False, pad=0)
AXES = dict(op="axes", runs=1, tokens=1, pad=0, H_Q=32, H_KV=8, D=128, bs=16, dtype="bf16", rotary=128, axes=3,
            cyclic=False, interleaved=False, norm=False, far=8192)
BOUNDS = dict(op="bounds", runs=1, tokens=1, pad=0, H_KV=8, D=128, bs=16, dtype="bf16")
SELECT = dict(op="select", B=1, len_max=8192, ragged=False, n_q=1, pad=0, H_Q=32, H_KV=8, D=128, bs=16, top_k=64,
              sink=1, recent=2)
ATTEND = dict(op="attend", B=1, len_max=32768, ragged=False, n_q=1, pad=0, H_Q=32, H_KV=8, D=128, bs=16,
              dtype="bf16", top_k=64)


def listed():
    return [
        # a small decoding batch: every sequence grows by a token; what counts is latency
        dict(PLAN, name="plan decode, 8 sequences"),
        # a busy server's step: most sequences decode, some finish, some drop rejected drafts, some wait, long
        # prompts begin; there are fewer free blocks than the step asks for, and the row buffers are padded
        dict(PLAN, name="plan mixed, 512 sequences", B=512, far=32768, prompts=12, tokens=65536, finish=24, cut=40,
             idle=16, short=True, pad=77),
        # one new text token of one sequence
        dict(AXES, name="axes append, 1 sequence"),
        # prompts of text and images written in one call, queries and keys normalised, three axes by turns
        dict(AXES, name="axes write, image prompts", runs=24, tokens=16384, pad=19, cyclic=True, norm=True, far=16384),
        # the blocks of a decoding batch's new tokens
        dict(BOUNDS, name="bounds decode, 64 sequences", runs=64, tokens=64),
        # the blocks of long prompts, e4m3 cache
        dict(BOUNDS, name="bounds prompts e4m3", runs=5, tokens=65500, pad=36, dtype="fp8"),
        # a single user's step: what counts is latency
        dict(SELECT, name="select decode, 1 of 8k"),
        # a batch of long contexts
        dict(SELECT, name="select decode, 16 of 128k", B=16, len_max=131072, top_k=128),
        # a chunk of a long prompt: every query scores every block
        dict(SELECT, name="select chunk, 512 of 32k", len_max=32768, n_q=512, top_k=64),
        # a single user's step at a long context
        dict(ATTEND, name="attend decode, 1 sequence"),
        # a serving batch, ragged contexts, e4m3 cache
        dict(ATTEND, name="attend decode e4m3, 64 sequences", B=64, len_max=16384, ragged=True, dtype="fp8",
             top_k=128),
        # the queries of a chunk, each with its own blocks
        dict(ATTEND, name="attend chunk, 512 of 32k", n_q=512),
    ]


HEADS = [(32, 8, 128), (32, 32, 128), (32, 1, 128), (8, 2, 64), (24, 8, 64), (40, 8, 128), (12, 4, 128)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above: sequences 1 to 512, tokens 1 to 65536, contexts 1 to 131072, lists of 2 to
    128 blocks of 16 to 64 positions."""
    op = rng.choice(["plan", "axes", "bounds", "select", "attend"])
    pad = rng.choice([0, 0, rng.randint(1, 100)])
    if op == "plan":
        B = _log(rng, 1, 512)
        c = dict(PLAN, B=B, bs=rng.choice([16, 16, 32, 64]), far=_log(rng, 16, 32768), short=rng.random() < 0.4, pad=pad)
        left = B
        for kind, share in (("prompts", 0.3), ("finish", 0.3), ("cut", 0.3), ("idle", 0.2)):
            c[kind] = min(left, rng.randint(0, max(1, int(B * share))))
            left -= c[kind]
        c["tokens"] = _log(rng, c["prompts"], 65536) if c["prompts"] else 0
        return c
    H_Q, H_KV, D = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "fp8", "int4"]) if D == 128 else "bf16"
    if op == "axes":
        c = dict(AXES, H_Q=H_Q, H_KV=H_KV, D=D, dtype="fp8" if dtype == "int4" else dtype, pad=pad,
                 bs=rng.choice([16, 16, 32, 64]), runs=_log(rng, 1, 256), axes=rng.randint(1, 4),
                 cyclic=rng.random() < 0.5, interleaved=rng.random() < 0.4, norm=rng.random() < 0.5,
                 far=_log(rng, 64, 131072))
        c["rotary"] = rng.choice([D, D, D // 2, 16 * rng.randint(1, D // 16)])
        per_token = 2 * D * (2 * H_Q + 3 * H_KV)
        c["tokens"] = max(c["runs"], _log(rng, 1, min(16384, 350_000_000 // per_token)))
        return c
    if op == "bounds":
        c = dict(BOUNDS, H_KV=H_KV, D=D, dtype=dtype, pad=pad, bs=rng.choice([16, 16, 32, 64]), runs=_log(rng, 1, 256))
        c["tokens"] = max(c["runs"], _log(rng, 1, min(65536, 250_000_000 // (2 * D * H_KV))))
        return c
    c = dict(SELECT if op == "select" else ATTEND, H_Q=H_Q, H_KV=H_KV, D=D, pad=pad, bs=rng.choice([16, 16, 32, 64]),
             top_k=_log(rng, 2, 128))
    if rng.random() < 0.6:   # decode: one query a sequence
        c.update(B=_log(rng, 1, 64), len_max=_log(rng, 1, 131072), ragged=rng.random() < 0.6)
    else:                    # a chunk, or drafted tokens of some sequences
        c.update(B=rng.choice([1, 1, 2, 5]), len_max=_log(rng, 1, 32768), ragged=rng.random() < 0.5)
        c["n_q"] = _log(rng, 1, max(1, min(c["len_max"], 512 // c["B"])))
    if op == "select":   # at least one query has more blocks than its list takes
        c["len_max"] = max(c["len_max"], 8 * c["bs"])
        while (c["B"] * c["len_max"] // c["bs"] * H_KV * 2 * D > 500_000_000
               or c["B"] * c["n_q"] * (c["len_max"] // c["bs"]) * H_Q * D > 4_000_000_000):
            c["len_max"] = max(c["n_q"], 8 * c["bs"], c["len_max"] // 2)
        c["top_k"] = min(c["top_k"], c["len_max"] // c["bs"] // 2)
        c["sink"] = rng.choice([0, 1, 1, 2]) if c["top_k"] > 4 else 0
        c["recent"] = rng.choice([1, 2]) if c["top_k"] > 4 else 1
        return c
    c["dtype"] = dtype
    while c["B"] * c["len_max"] * H_KV * D > 1_000_000_000:
        c["len_max"] = max(c["n_q"], c["len_max"] // 2)
    while c["B"] * c["n_q"] * c["top_k"] * c["bs"] * H_KV * D * BITS[dtype] > 512 * 64 * 16 * 8 * 128 * 16:
        c["top_k"] = max(2, c["top_k"] // 2)
    return c


# ------------------------------------------------------------------ layout of a case (the same for every seed)
def _layout(c):
    return random.Random(",".join(f"{k}={c[k]}" for k in sorted(c) if k != "name"))


def _parts(r, total, n):
    """total split at random into n positive parts."""
    cuts = sorted(r.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _requests(c):
    """(lengths held, lengths wanted) of a plan case's sequences."""
    r = _layout(c)
    kinds = sum(([k] * c[n] for k, n in (("p", "prompts"), ("f", "finish"), ("c", "cut"), ("i", "idle"))), [])
    kinds += ["d"] * (c["B"] - len(kinds))
    r.shuffle(kinds)
    parts = _parts(r, c["tokens"], c["prompts"]) if c["prompts"] else []
    lens, new = [], []
    for k in kinds:
        n = 0 if k == "p" else _log(r, 1, c["far"])
        lens.append(n)
        new.append({"p": parts.pop() if k == "p" else 0, "f": 0, "c": max(0, n - r.randint(1, 5)), "i": n,
                    "d": n + 1}[k])
    return lens, new


def _blocks(c, n):
    return -(-n // c["bs"])


def _plan_sizes(c):
    """(lens, new, table width, blocks in all, free blocks, rows) of a plan case."""
    lens, new = _requests(c)
    mb = max(1, max(_blocks(c, n) for n in lens + new))
    grow = sum(max(0, _blocks(c, b) - _blocks(c, a)) for a, b in zip(lens, new))
    held = sum(_blocks(c, n) for n in lens)
    free = grow * 3 // 4 if c["short"] else grow + 5
    return lens, new, mb, held + grow + 5, free, sum(max(0, b - a) for a, b in zip(lens, new)) + c["pad"]


def _runs(c):
    """(first slot of its first block, tokens) of each run of new tokens of an axes or a bounds case."""
    r = _layout(c)
    return [(r.randrange(c["bs"]), n) for n in _parts(r, c["tokens"], c["runs"])]


def _rows(c):
    """(length, queries) of each sequence of a select or an attend case; a ragged batch of 8 or more holds an empty
    sequence.  The queries are a sequence's last positions."""
    r = _layout(c)
    lens = [c["len_max"]] + [_log(r, max(1, c["len_max"] // 256), c["len_max"]) if c["ragged"] else c["len_max"]
                             for _ in range(c["B"] - 1)]
    if c["ragged"] and c["B"] >= 8:
        lens[3] = 0
    return [(n, min(n, c["n_q"])) for n in lens]


def _decode(c):
    return c["n_q"] == 1 and not c["pad"]   # row b is sequence b: no sequence ids


def work(case):
    c = case
    if c["op"] == "plan":
        lens, new, _, _, free, rows = _plan_sizes(c)
        moved = sum(abs(_blocks(c, b) - _blocks(c, a)) for a, b in zip(lens, new))
        return {"bytes": 16 * c["B"] + 8 * moved + 12 * rows, "flops": 4 * c["B"] + 4 * rows}
    D = c["D"]
    if c["op"] == "axes":
        T = c["tokens"]
        nb = T * D * (2 * (2 * c["H_Q"] + 2 * c["H_KV"]) + 2 * c["H_KV"] * BITS[c["dtype"]] // 8) + T * 4 * (1 + c["axes"])
        return {"bytes": nb, "flops": T * D * (c["H_Q"] + c["H_KV"]) * (8 if c["norm"] else 3)}
    if c["op"] == "bounds":
        read = sum(a + n for a, n in _runs(c))
        blocks = sum(_blocks(c, a + n) for a, n in _runs(c))
        return {"bytes": read * c["H_KV"] * D * BITS[c["dtype"]] // 8 + blocks * c["H_KV"] * (2 * D + 4) + 4 * c["tokens"],
                "flops": 2 * read * c["H_KV"] * D}
    rows = _rows(c)
    T = sum(q for _, q in rows)
    io = T * c["H_Q"] * D * 2
    if c["op"] == "select":
        blocks = sum(_blocks(c, n) for n, _ in rows)
        pairs = sum(_blocks(c, n) * q for n, q in rows)
        return {"bytes": io + blocks * (c["H_KV"] * (2 * D + 4) + 4) + 4 * T * c["H_KV"] * c["top_k"],
                "flops": 4 * pairs * c["H_Q"] * D}
    listed_ = [(min(c["top_k"], _blocks(c, n)), n, q) for n, q in rows]
    read = sum(min(k * q * c["bs"], n) for k, n, q in listed_)
    seen = sum(min(k * c["bs"], n) * q for k, n, q in listed_)
    return {"bytes": 2 * io + 2 * read * c["H_KV"] * D * BITS[c["dtype"]] // 8 + 4 * T * c["H_KV"] * c["top_k"],
            "flops": 4 * seen * c["H_Q"] * D}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _perm(n, seed):
    return torch.randperm(n, generator=torch.Generator().manual_seed(int(seed))).numpy().astype(np.int32)


def _ints(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _filled_pool(c, g, blocks):
    """A pool's bytes [blocks, H_KV, 2, bs, row bytes] holding normal keys and values, and its scales."""
    shape = (blocks, c["H_KV"], 2, c["bs"], c["D"])
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
        code = (torch.randn((m, 2), generator=g, device=DEV) * 2).round_().clamp_(-7, 7).to(torch.int8) + 8
        data[a:a + m] = code[:, 0].to(torch.uint8) | (code[:, 1].to(torch.uint8) << 4)
    return data.view(shape[:-1] + (c["D"] // 2,)), scales / 2


def _slots(c, seed):
    """Slots of the new tokens (padding rows: -1), the last row in each block, and the number of blocks."""
    runs = _runs(c)
    need = sum(_blocks(c, a + n) for a, n in runs)
    ids = _perm(need + 3, seed)
    at, slots = 0, []
    for a, n in runs:
        t = np.arange(a, a + n)
        slots.append(ids[at + t // c["bs"]].astype(np.int64) * c["bs"] + t % c["bs"])
        at += _blocks(c, a + n)
    slots = np.concatenate(slots + [np.full(c["pad"], -1)])
    nxt = np.append(slots[1:], -1)
    last = np.flatnonzero((slots >= 0) & (((slots + 1) % c["bs"] == 0) | (nxt != slots + 1)))
    return slots, last, need + 3


def _axes_positions(c):
    """[axes, rows] positions: text has the same on every axis; an image's tokens share the first and walk a grid on
    the others."""
    r = _layout(c)
    cols = []
    for _, n in _runs(c):
        at = _log(r, 1, c["far"]) - 1
        while n > 0:
            m = min(n, _log(r, 1, 1024))
            i = np.arange(m)
            if r.random() < 0.5:
                cols.append(np.tile(at + i, (c["axes"], 1)))
                at += m
            else:
                w = max(1, int(math.sqrt(m)))
                grid = [np.full(m, at), at + i // w, at + i % w, at + (i // 2) % w][:c["axes"]]
                cols.append(np.stack(grid))
                at += w + 1
            n -= m
    cols.append(np.full((c["axes"], c["pad"]), -1))
    return np.concatenate(cols, 1)


def _axis_of(c):
    """The axis of every frequency: by turns, or in equal sections."""
    half = c["rotary"] // 2
    return [(i % c["axes"]) if c["cyclic"] else i * c["axes"] // half for i in range(half)]


def _inv_freq(c):
    r = c["rotary"]
    return torch.tensor([500000.0 ** (-2.0 * i / r) for i in range(r // 2)], device=DEV, dtype=torch.float32)


def _inputs(c, seed):
    g = _gen(seed)
    s = {"case": c}
    if c["op"] == "plan":
        lens, new, mb, N, free, rows = _plan_sizes(c)
        ids = _perm(N, seed)
        table = np.full((c["B"], mb), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(lens):
            k = _blocks(c, n)
            table[b, :k] = ids[at:at + k]
            at += k
        stack = np.full(N, -1, dtype=np.int32)
        stack[:free] = ids[at:at + free]
        s.update(table=_ints(table), lens=_ints(lens), new=_ints(new), stack=_ints(stack), count=_ints([free]),
                 rows=rows, N=N)
        return s
    D, H_KV = c["D"], c["H_KV"]
    if c["op"] in ("axes", "bounds"):
        slots, last, blocks = _slots(c, seed)
        s["slots"] = _ints(slots)
        if c["op"] == "axes":
            rows = len(slots)
            # the fused projection's output, of which q, k and v are strided views
            s["qkv"] = (_normal(g, rows, (c["H_Q"] + 2 * H_KV) * D) * (2.0 if c["norm"] else 1.0)).to(torch.bfloat16)
            s["positions"] = _ints(_axes_positions(c))
            s["axis_of"] = torch.tensor(_axis_of(c), dtype=torch.uint8, device=DEV)
            s["inv_freq"] = _inv_freq(c)
            s["q_norm"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16) if c["norm"] else None
            s["k_norm"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16) if c["norm"] else None
        else:
            s["last"] = torch.from_numpy(last).to(DEV)
        s["pool"], s["scales"] = _filled_pool(c, g, blocks)
        return s
    rows = _rows(c)
    lens = [n for n, _ in rows]
    N = sum(_blocks(c, n) for n in lens) + 2
    ids = _perm(N, seed)
    table = np.full((c["B"], max(1, max(_blocks(c, n) for n in lens))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = _blocks(c, n)
        table[b, :k] = ids[at:at + k]
        at += k
    s["table"], s["N"] = _ints(table), N
    if _decode(c):
        s["seq"], positions = None, [n - 1 for n in lens]
    else:
        s["seq"] = _ints([b for b, (_, q) in enumerate(rows) for _ in range(q)] + [-1] * c["pad"])
        positions = [p for n, q in rows for p in range(n - q, n)] + [-1] * c["pad"]
    s["positions"] = _ints(positions)
    T = len(positions)
    # queries of the size that a trained head has: scores with a spread of a few units
    s["q"] = (_normal(g, T, c["H_Q"], D) * 2.0).to(torch.bfloat16)
    if c["op"] == "select":
        # bounds of 16 or more normal keys: largest and smallest about 1.8 from the middle, some blocks far out
        codes = torch.empty((N, H_KV, 2, D), device=DEV, dtype=torch.int8)
        for a in range(0, N, 1 << 15):
            b = min(N, a + (1 << 15))
            x = _normal(g, b - a, H_KV, 2, D) * 17.0
            x[:, :, 0] += 57.0
            x[:, :, 1] -= 57.0
            x = x.round_().clamp_(-127, 127).sort(2, descending=True).values
            codes[a:b] = x.to(torch.int8)
        s["codes"] = codes
        s["exps"] = torch.exp2(torch.randint(-6, -3, (N, H_KV), generator=g, device=DEV).float())
        return s
    # each query's list: its first block, its own, and others at random, ascending; unused entries are -1
    lists = torch.full((T, H_KV, c["top_k"]), -1, device=DEV, dtype=torch.int32)
    at = 0
    for n, q in rows:
        if q == 0:
            at += 1 if _decode(c) else 0   # an empty sequence has a row only in a decode batch
            continue
        own_block = torch.arange(n - q, n, device=DEV) // c["bs"]
        x = torch.rand((q, H_KV, _blocks(c, n)), generator=g, device=DEV)
        j = torch.arange(x.shape[2], device=DEV)
        x[:, :, 0] = 2.0
        x = torch.where(j == own_block[:, None, None], torch.full_like(x, 3.0), x)
        x = torch.where(j > own_block[:, None, None], torch.full_like(x, -1.0), x)
        v, i = x.topk(min(c["top_k"], x.shape[2]), -1)
        i = torch.where(v < 0, 1 << 30, i).sort(-1).values
        lists[at:at + q, :, :i.shape[2]] = torch.where(i == 1 << 30, -1, i).int()
        at += q
    s["lists"] = lists
    s["pool"], s["scales"] = _filled_pool(c, g, N)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case

    def empty(*shape, dtype=torch.int32):
        return torch.zeros(shape, device=DEV, dtype=dtype)

    if c["op"] == "plan":
        s.update(lens_out=empty(c["B"]), count_out=empty(1), cu=empty(c["B"] + 1), slots=empty(s["rows"]),
                 positions=empty(s["rows"]), seq=empty(s["rows"]))
    elif c["op"] == "axes":
        q, k, v = s["qkv"].split([c["H_Q"] * c["D"], c["H_KV"] * c["D"], c["H_KV"] * c["D"]], dim=1)
        s["q"], s["k"], s["v"] = (x.view(x.shape[0], -1, c["D"]) for x in (q, k, v))
        s["q_out"] = empty(*s["q"].shape, dtype=torch.bfloat16)
    elif c["op"] == "bounds":
        s["codes"] = empty(s["pool"].shape[0], c["H_KV"], 2, c["D"], dtype=torch.int8)
        s["exps"] = empty(s["pool"].shape[0], c["H_KV"], dtype=torch.float32)
    elif c["op"] == "select":
        s["lists"] = empty(s["q"].shape[0], c["H_KV"], c["top_k"])
    else:
        s["out"] = empty(*s["q"].shape, dtype=torch.bfloat16)
        s["lse"] = empty(*s["q"].shape[:2], dtype=torch.float32) if c["dtype"] == "bf16" else None
    if own:
        import paged_kv_cache_kvc_gb300 as kvc
        s["kvc"] = kvc
        dt = {"bf16": kvc.KVC_BF16, "fp8": kvc.KVC_FP8_E4M3, "int4": kvc.KVC_INT4}[c.get("dtype", "bf16")]
        if "pool" in s:
            data = s["pool"]
            pool = kvc.kvc_pool_create(data.shape[0], c["bs"], 1, c["H_KV"], c["D"], dt)
            pool.bytes_view().copy_(data.view(-1).view(torch.uint8))
            if s["scales"] is not None:
                kvc.kvc_pool_set_scales(pool, 0, s["scales"][0].contiguous(), s["scales"][1].contiguous())
            s["pool"] = pool.bytes_view().view(data.dtype).view(data.shape)
            s["pool"].handle = pool   # the view does not own the pool's memory: keep the pool while it is in use
        elif c["op"] == "plan":       # the plan reads no keys: any pool of these blocks
            pool = kvc.kvc_pool_create(s["N"], c["bs"], 1, 1, 64, kvc.KVC_BF16)
        else:
            dt = kvc.KVC_INT4 if c["D"] == 128 else kvc.KVC_BF16
            pool = kvc.kvc_pool_create(s["N"], c["bs"], 1, c["H_KV"], c["D"], dt)
        s["handle"] = pool
        if c["op"] == "axes":
            s["rope"] = kvc.Rope(s["inv_freq"], interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                                 eps=1e-6, axis_of=s["axis_of"])
        elif c["op"] in ("bounds", "select"):
            s["bounds"] = kvc.kvc_block_bounds(pool)
            codes, exps = kvc.kvc_block_bounds_views(pool, 0, s["bounds"])
            codes.copy_(s["codes"])
            exps.copy_(s["exps"])
            s["codes"], s["exps"] = codes, exps
    return s


# ------------------------------------------------------------------ plain forms
def _plain_plan(s):
    c = s["case"]
    bs, B, rows = c["bs"], c["B"], s["rows"]
    lens, new = s["lens"].long(), s["new"].long()
    have, want = (lens + bs - 1) // bs, (new + bs - 1) // bs
    freed, grow, tokens = (want - have).clamp(max=0).neg(), (want - have).clamp(min=0), (new - lens).clamp(min=0)
    avail = s["count"].long() + freed.sum()
    ok = (tokens == 0) | ((grow.cumsum(0) <= avail) & (tokens.cumsum(0) <= rows))
    grow, tokens = grow * ok, tokens * ok
    table, stack = s["table"], s["stack"]
    width = table.shape[1]
    j = torch.arange(width, device=DEV)
    # freed entries to the stack's top, in the order of the table (others to a place past its end)
    dead = (j >= want[:, None]) & (j < have[:, None])
    place = torch.where(dead, s["count"].long() + (freed.cumsum(0) - freed)[:, None] + j - want[:, None], stack.numel())
    spare = torch.cat([stack, stack.new_zeros(1)])
    spare[place.view(-1)] = table.view(-1)
    stack.copy_(spare[:-1])
    # taken entries from its top
    fresh = (j >= have[:, None]) & (j < (have + grow)[:, None])
    source = avail - 1 - ((grow.cumsum(0) - grow)[:, None] + j - have[:, None])
    table.copy_(torch.where(fresh, stack[source.clamp(0, stack.numel() - 1)], table))
    s["lens_out"].copy_(torch.where(ok, new, lens))
    s["count_out"].copy_(avail - grow.sum())
    s["cu"][1:] = tokens.cumsum(0)
    r = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), r.int(), right=True)
    live = seq < B
    b = seq.clamp(max=B - 1)
    p = lens[b] + r - s["cu"][b]
    slot = table[b, (p // bs).clamp(0, width - 1)].long() * bs + p % bs
    s["slots"].copy_(torch.where(live, slot, -1))
    s["positions"].copy_(torch.where(live, p, -1))
    s["seq"].copy_(torch.where(live, seq, -1))
    return [s["lens_out"], s["count_out"], s["cu"], s["slots"], s["positions"], s["seq"], table, stack]


def _rotated(s, x, weight):
    """x [T, H, D] RMS-normalised (with a weight) and rotated by its positions, fp32."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = s["positions"].t()[:x.shape[0], s["axis_of"].long()].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = c["rotary"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_axes(s):
    c = s["case"]
    T = c["tokens"]
    slots = s["slots"][:T].long()
    s["q_out"][:T] = _rotated(s, s["q"][:T], s["q_norm"]).to(torch.bfloat16)
    k = _rotated(s, s["k"][:T], s["k_norm"])
    v = s["v"][:T]
    if c["dtype"] == "fp8":
        k = (k / s["scales"][0]).clamp(-448, 448)
        v = (v.float() / s["scales"][1]).clamp(-448, 448)
    kv = torch.stack([k.to(s["pool"].dtype), v.to(s["pool"].dtype)], 2)   # [T, H_KV, 2, D]
    raw = {2: torch.int16, 1: torch.uint8}[kv.element_size()]
    s["pool"].view(raw)[slots // c["bs"], :, :, slots % c["bs"]] = kv.view(raw)
    return [s["q_out"], s["pool"]]


def _values(c, s, x, kind):
    """Stored elements [..., H_KV at dim 1, ..., row] of kind 0 (keys) or 1 as fp32."""
    if c["dtype"] == "int4":
        x = torch.stack([(x & 15).to(torch.int8) - 8, (x >> 4).to(torch.int8) - 8], -1).flatten(-2)
    x = x.float()
    if s["scales"] is None:
        return x
    scale = s["scales"][kind]
    return x * scale.view((1, scale.shape[0]) + (1,) * (x.dim() - 3) + (scale.shape[1],))


def _power(x):
    """The smallest e with x <= 127 * 2^e, kept in [-100, 100]."""
    m, e = torch.frexp(x)
    return torch.where(x == 0, -100, (e - 7 + (m * 128 > 127).int()).clamp(-100, 100))


def _plain_bounds(s):
    c = s["case"]
    bs = c["bs"]
    slots = s["slots"][s["last"]].long()
    block = slots // bs
    k = _values(c, s, s["pool"][block, :, 0], 0)   # [blocks, H_KV, bs, D]
    seen = (torch.arange(bs, device=DEV) <= (slots % bs)[:, None])[:, None, :, None]
    hi = k.masked_fill(~seen, -math.inf).amax(2)
    lo = k.masked_fill(~seen, math.inf).amin(2)
    e = _power(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    small = torch.exp2(-e.float())[..., None]
    s["codes"][block] = torch.stack([torch.ceil(hi * small), torch.floor(lo * small)], 2).clamp(-127, 127).to(torch.int8)
    s["exps"][block] = torch.exp2(e.float())
    return [s["codes"], s["exps"]]


def _groups(c, s, device_rows):
    """(first row, rows, sequence) of each sequence's queries."""
    at = 0
    for b, (_, q) in enumerate(_rows(c)):
        n = 1 if _decode(c) else q
        if q:
            yield at, q, b
        at += n


def _plain_select(s):
    c = s["case"]
    H, g, D, k = c["H_KV"], c["H_Q"] // c["H_KV"], c["D"], c["top_k"]
    rows = _rows(c)
    for at, n, b in _groups(c, s, s["q"]):
        nb = _blocks(c, rows[b][0])
        ids = s["table"][b, :nb].long()
        x = s["q"][at:at + n].float().view(n, H, g, D)
        e = _power(x.abs().amax((2, 3), keepdim=True))
        x = torch.round(x * torch.exp2(-e.float()))
        x = torch.cat([x.clamp(min=0), x.clamp(max=0)], -1).permute(1, 0, 2, 3).reshape(H, n * g, 2 * D)
        code = s["codes"][ids].float().reshape(nb, H, 2 * D).permute(1, 2, 0)
        score = (x @ code).view(H, n, g, nb).amax(2) * s["exps"][ids].t()[:, None]   # whole numbers: exact
        own_block = (s["positions"][at:at + n].long() // c["bs"])[:, None]
        j = torch.arange(nb, device=DEV)
        score = torch.where((j < c["sink"]) | (j > own_block - c["recent"]), math.inf, score)
        score = torch.where(j > own_block, -math.inf, score)
        v, i = score.sort(dim=-1, descending=True, stable=True)
        m = min(k, nb)
        i = torch.where(v[..., :m] == -math.inf, nb, i[..., :m]).sort(-1).values
        s["lists"][at:at + n] = -1
        s["lists"][at:at + n, :, :m] = torch.where(i == nb, -1, i).permute(1, 0, 2).int()
    return [s["lists"]]


def _plain_attend(s):
    c = s["case"]
    H, g, D, bs = c["H_KV"], c["H_Q"] // c["H_KV"], c["D"], c["bs"]
    T = s["q"].shape[0] - c["pad"]
    step = max(1, (1 << 28) // (H * c["top_k"] * bs * D))
    head = torch.arange(H, device=DEV)[:, None]
    for a in range(0, T, step):
        z = min(T, a + step)
        n = z - a
        lists, pos = s["lists"][a:z].long(), s["positions"][a:z].long()
        seq = (torch.arange(a, z, device=DEV) if s["seq"] is None else s["seq"][a:z].long())[:, None, None]
        ids = s["table"][seq, lists.clamp(min=0)].clamp(min=0).long()
        kv = s["pool"][ids, head]   # [n, H, top_k, 2, bs, row]
        k, v = (_values(c, s, kv[:, :, :, i], i).reshape(n, H, -1, D) for i in (0, 1))
        t = lists[..., None] * bs + torch.arange(bs, device=DEV)
        seen = ((lists[..., None] >= 0) & (t <= pos[:, None, None, None])).view(n, H, 1, -1)
        q = s["q"][a:z].float().view(n, H, g, D)
        x = ((q @ k.transpose(2, 3)) * D ** -0.5).masked_fill(~seen, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
        total = p.sum(-1, keepdim=True)
        out = (p @ v) / torch.where(total == 0, 1.0, total)
        live = (pos >= 0)[:, None, None]   # a row without a query stays as it is
        s["out"][a:z] = torch.where(live, out.reshape(n, -1, D).to(torch.bfloat16), s["out"][a:z])
        if s["lse"] is not None:
            lse = (m + torch.log(total)).reshape(n, -1)
            s["lse"][a:z] = torch.where(live[..., 0], lse, s["lse"][a:z])
    return [s["out"], s["lse"]] if s["lse"] is not None else [s["out"]]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"plan": _plain_plan, "axes": _plain_axes, "bounds": _plain_bounds, "select": _plain_select,
                "attend": _plain_attend}[c["op"]](s)
    kvc, pool = s["kvc"], s["handle"]
    if c["op"] == "plan":
        kvc.kvc_plan_step(pool, s["table"], s["lens"], s["new"], s["stack"], s["count"], s["lens_out"], s["count_out"],
                          s["cu"], s["slots"], s["positions"], s["seq"])
        return [s["lens_out"], s["count_out"], s["cu"], s["slots"], s["positions"], s["seq"], s["table"], s["stack"]]
    if c["op"] == "axes":
        kvc.kvc_rope_write_slots(pool, 0, s["slots"], s["positions"], s["q"], s["k"], s["v"], s["q_out"], s["rope"])
        return [s["q_out"], s["pool"]]
    if c["op"] == "bounds":
        kvc.kvc_update_bounds(pool, 0, s["bounds"], s["slots"])
        return [s["codes"], s["exps"]]
    if c["op"] == "select":
        kvc.kvc_select_blocks(pool, 0, s["bounds"], s["q"], s["table"], s["positions"], s["lists"], seq_ids=s["seq"],
                              sink=c["sink"], recent=c["recent"])
        return [s["lists"]]
    kvc.kvc_sparse_attn(pool, 0, s["q"], s["table"], s["positions"], s["lists"], s["out"], s["lse"], seq_ids=s["seq"])
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


def _exact_plan(c, s):
    """Sequence by sequence and token by token, on the host."""
    lens, new, _, _, free, rows = _plan_sizes(c)
    table, stack = s["table"].cpu().numpy().copy(), s["stack"].cpu().numpy().copy()
    top, bs = free, c["bs"]
    for b, (a, z) in enumerate(zip(lens, new)):
        for j in range(_blocks(c, z), _blocks(c, a)):
            stack[top] = table[b, j]
            top += 1
    out, cu, slots, positions, seqs, full = [], [0], [], [], [], False
    for b, (a, z) in enumerate(zip(lens, new)):
        need = max(0, _blocks(c, z) - _blocks(c, a))
        if z > a:
            full = full or need > top or len(slots) + z - a > rows
        if z > a and not full:
            for j in range(_blocks(c, a), _blocks(c, z)):
                top -= 1
                table[b, j] = stack[top]
            for p in range(a, z):
                slots.append(table[b, p // bs] * bs + p % bs)
                positions.append(p)
                seqs.append(b)
        out.append(a if z > a and full else z)
        cu.append(len(slots))
    pad = [-1] * (rows - len(slots))
    return [_ints(x) for x in (out, [top], cu, slots + pad, positions + pad, seqs + pad, table, stack)]


def _exact_axes(c, s):
    H_Q, H_KV, D, T, bs = c["H_Q"], c["H_KV"], c["D"], c["tokens"], c["bs"]
    x = s["qkv"][:T].double().view(T, H_Q + 2 * H_KV, D)
    y = x.clone()
    for lo, hi, w in ((0, H_Q, s["q_norm"]), (H_Q, H_Q + H_KV, s["k_norm"])):
        if w is not None:
            y[:, lo:hi] = x[:, lo:hi] / torch.sqrt((x[:, lo:hi] ** 2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
    half = c["rotary"] // 2
    for i, axis in enumerate(_axis_of(c)):
        i0, i1 = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), s["positions"][axis, :T].double() * s["inv_freq"][i].double())
        u = torch.complex(y[:, :H_Q + H_KV, i0], y[:, :H_Q + H_KV, i1]) * z[:, None]
        y[:, :H_Q + H_KV, i0], y[:, :H_Q + H_KV, i1] = u.real, u.imag
    pool = _e4m3_values()[s["pool"].view(torch.uint8).long()] if c["dtype"] == "fp8" else s["pool"].double()
    slots = s["slots"][:T].long()
    for kind in (0, 1):
        kv = y[:, H_Q + kind * H_KV:H_Q + (kind + 1) * H_KV]
        if s["scales"] is not None:
            kv = torch.clamp(kv / s["scales"][kind].double(), -448, 448)
        pool[torch.div(slots, bs, rounding_mode="floor"), :, kind, slots % bs] = kv
    q = torch.zeros((T + c["pad"], H_Q, D), device=DEV, dtype=torch.float64)
    q[:T] = y[:, :H_Q]
    return [q, pool]


def _stored(c, s, ids, head, kind):
    """Stored keys (kind 0) or values (1) of the given blocks and heads, fp64 [..., bs, D].  A stored element stands
    for its code times its scale, one fp32 product."""
    x = s["pool"][ids, head, kind]
    if c["dtype"] == "bf16":
        return x.double()
    if c["dtype"] == "fp8":
        y = _e4m3_values()[x.view(torch.uint8).long()]
    else:
        b = x.long()
        y = torch.empty(b.shape[:-1] + (c["D"],), device=DEV, dtype=torch.float64)
        y[..., 0::2], y[..., 1::2] = (b % 16 - 8).double(), (b // 16 - 8).double()
    return (y.float() * s["scales"][kind, head].unsqueeze(-2)).double()


def _exact_bounds(c, s):
    bs, H, D = c["bs"], c["H_KV"], c["D"]
    N = s["pool"].shape[0]
    codes = torch.zeros((N, H, 2, D), device=DEV, dtype=torch.int8)
    exps = torch.zeros((N, H), device=DEV, dtype=torch.float64)
    slots = s["slots"].cpu().numpy()
    filled = {}
    for x in slots[slots >= 0]:
        filled[int(x) // bs] = int(x) % bs + 1   # rows come in ascending order
    by_fill = {}
    for block, n in filled.items():
        by_fill.setdefault(n, []).append(block)
    for n, blocks in by_fill.items():
        for a in range(0, len(blocks), 4096):
            ids = torch.tensor(blocks[a:a + 4096], device=DEV)
            k = _stored(c, s, ids[:, None], torch.arange(H, device=DEV)[None], 0)[:, :, :n]
            top = k.abs().amax((2, 3))
            e = torch.full(top.shape, -100, device=DEV, dtype=torch.float64)
            low = torch.ceil(torch.log2(top / 127.0)).clamp(-100, 100)
            for shift in (1, 0, -1):   # the logarithm may land beside a border: take the smallest that holds
                t = (low + shift).clamp(-100, 100)
                e = torch.where(top <= 127.0 * torch.exp2(t), t, e)
            unit = torch.exp2(e)[..., None]
            hi, lo = torch.ceil(k.amax(2) / unit), torch.floor(k.amin(2) / unit)
            codes[ids] = torch.stack([hi, lo], 2).clamp(-127, 127).to(torch.int8)
            exps[ids] = torch.exp2(e)
    return [codes, exps]


def _exact_select(c, s):
    H, g, D, bs, k = c["H_KV"], c["H_Q"] // c["H_KV"], c["D"], c["bs"], c["top_k"]
    lists = torch.zeros((s["q"].shape[0], H, k), device=DEV, dtype=torch.int32)
    rows = _rows(c)
    if sum(_blocks(c, n) * q for n, q in rows) * c["H_Q"] * D > 6_000_000_000:
        return None
    for at, n, b in _groups(c, s, s["q"]):
        nb = _blocks(c, rows[b][0])
        rec = s["codes"][s["table"][b, :nb].long()].double()       # [nb, H, 2, D]
        unit = s["exps"][s["table"][b, :nb].long()].double()
        for h in range(H):
            for i in range(at, at + n):
                q = s["q"][i, h * g:(h + 1) * g].double()
                top, e = float(q.abs().max()), -100
                while e < 100 and top > 127.0 * 2.0 ** e:
                    e += 1
                whole = torch.round(q / 2.0 ** e)
                score = torch.full((nb,), -math.inf, device=DEV, dtype=torch.float64)
                for x in whole:
                    score = torch.maximum(score, torch.maximum(rec[:, h, 0] * x, rec[:, h, 1] * x).sum(-1))   # hi >= lo
                score = (score * unit[:, h]).cpu().numpy()
                last = (rows[b][0] - n + i - at) // bs
                forced = [j for j in range(last + 1) if j < c["sink"] or j > last - c["recent"]]
                rest = np.setdiff1d(np.arange(last + 1), forced)
                rest = rest[np.lexsort((rest, -score[rest]))][:k - len(forced)]
                pick = sorted(forced + rest.tolist())
                lists[i, h] = torch.tensor(pick + [-1] * (k - len(pick)), dtype=torch.int32)
    return [lists]


def _exact_attend(c, s):
    H, g, D, bs = c["H_KV"], c["H_Q"] // c["H_KV"], c["D"], c["bs"]
    out = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], device=DEV, dtype=torch.float64)
    rows = _rows(c)
    step = max(1, (1 << 26) // (c["top_k"] * bs * D))
    for first, n, b in _groups(c, s, s["q"]):
        for h in range(H):
            for a in range(first, first + n, step):
                z = min(first + n, a + step)
                lists = s["lists"][a:z, h].long()
                ids = s["table"][b][lists.clamp(min=0)].long()
                k, v = (_stored(c, s, ids, h, kind).flatten(1, 2) for kind in (0, 1))
                p = rows[b][0] - n + torch.arange(a - first, z - first, device=DEV)
                t = (lists[:, :, None] * bs + torch.arange(bs, device=DEV)).flatten(1)
                no = (t > p[:, None]) | (t < 0)
                x = torch.einsum("ngd,ntd->ngt", s["q"][a:z, h * g:(h + 1) * g].double(), k) / math.sqrt(D)
                x = torch.where(no[:, None], torch.full((), -math.inf, device=DEV, dtype=torch.float64), x)
                l = torch.logsumexp(x, -1)
                out[a:z, h * g:(h + 1) * g] = torch.einsum("ngt,ntd->ngd", torch.exp(x - l[..., None]), v)
                lse[a:z, h * g:(h + 1) * g] = l
    return [out, lse] if c["dtype"] == "bf16" else [out]


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    return {"plan": _exact_plan, "axes": _exact_axes, "bounds": _exact_bounds, "select": _exact_select,
            "attend": _exact_attend}[c["op"]](c, s)
