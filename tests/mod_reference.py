"""Plain 64-bit forms of the rotary write and of attention with modified scores (numpy, one loop per row),
and the error bounds that their fp32 / bf16 / f16 kernels are held to."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}   # relative half steps


@dataclass
class Mod:
    softcap: float = 0.0
    window: int = 0
    sink: int = 0
    prefix: int = 0
    alibi: np.ndarray | None = None       # [H_Q]
    doc_start: np.ndarray | None = None   # [n_q]


def e4m3_table() -> np.ndarray:
    t = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        t[c] = -x if c & 128 else x
    return t


def pool_values(raw: np.ndarray, dtype: str, N: int, H_KV: int, bs: int, D: int) -> np.ndarray:
    """Layer bytes -> fp64 stored elements [N, H_KV, 2, bs, D] (codes, without scales)."""
    if dtype == "bf16":
        v = (raw.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    elif dtype == "fp8":
        v = e4m3_table()[raw]
    else:
        v = np.stack([(raw & 15).astype(np.float64) - 8, (raw >> 4).astype(np.float64) - 8], -1)
    return v.reshape(N, H_KV, 2, bs, D)


def visible(mod: Mod, i: int, p: int, total: int) -> np.ndarray:
    t = np.arange(total)
    d = max(int(mod.doc_start[i]), 0) if mod.doc_start is not None else 0
    see = (t <= p) & (t >= d)
    if mod.window:
        see &= (t > p - mod.window) | (t < d + mod.sink)
    if mod.prefix:
        see |= t < mod.prefix
    return see


# half step of a softmax weight as the operand of the value product: a bf16 high / low pair keeps 16 bits
WEIGHTS = {"pair": 2.0 ** -16, "bf16": HALF["bf16"], "f16": HALF["f16"]}


def attend(q, K, V, p, see, mod: Mod, scale, heads_per_kv, kind="bf16", weights="pair"):
    """One query row: q [H_Q, D], K / V [T, H_KV, D] fp64, position p.  Returns out, lse and their error bounds.

    weights: the type in which the kernel feeds the softmax weights to the value product.  Rounding every weight
    by at most half a step h moves the mixture by at most h * sum w |v|, which is what the bound adds."""
    H_Q, D = q.shape
    out, lse = np.zeros((H_Q, D)), np.full(H_Q, -np.inf)
    tol_o, tol_l = np.zeros((H_Q, D)), np.zeros(H_Q)
    t = np.flatnonzero(see)
    if t.size == 0:
        return out, lse, tol_o, tol_l
    for h in range(H_Q):
        k, v = K[t, h // heads_per_kv], V[t, h // heads_per_kv]
        x = scale * (k @ q[h])
        size = scale * float(np.max(np.abs(k) @ np.abs(q[h])))    # terms that the fp32 sum adds up
        grow = 1.0
        if mod.softcap:
            x = mod.softcap * np.tanh(x / mod.softcap)
        if mod.alibi is not None:
            x = x - float(mod.alibi[h]) * np.abs(p - t)
        m = x.max()
        w = np.exp(x - m)
        L = w.sum()
        out[h] = (w / L) @ v
        lse[h] = m + math.log(L)
        # score error: D fp32 additions (the tensor cores may truncate: a whole step each); for
        # quantised pools q times the key scale is rounded to f16; the cap's tanh is good to a few
        # fp32 steps of the cap, the bias to two steps of itself
        ds = (D + 8) * 2.0 ** -23 * size
        if kind != "bf16":
            ds += HALF["f16"] * size
        if mod.softcap:
            ds += 8 * mod.softcap * 2.0 ** -23
        ds += 4 * 2.0 ** -23 * float(np.max(np.abs(x)) + (np.max(np.abs(p - t)) * abs(float(mod.alibi[h]))
                                                         if mod.alibi is not None else 0.0))
        ds = ds * grow
        # weights: their rounding as an operand, the exponential's few steps, and the sum of t.size fp32
        # terms in any order
        rel = 2 * math.expm1(ds) + WEIGHTS[weights] + 16 * 2.0 ** -23 + min(t.size, 4096) * 2.0 ** -23
        tol_o[h] = HALF["bf16"] * (np.abs(out[h]) + rel * ((w / L) @ np.abs(v))) + rel * ((w / L) @ np.abs(v)) + 2.0 ** -130
        tol_l[h] = math.expm1(ds) + (16 + min(t.size, 4096)) * 2.0 ** -23 + 4 * 2.0 ** -24 * abs(lse[h])
    return out, lse, tol_o, tol_l


def rotate(x, pos, inv_freq, interleaved, weight=None, eps=1e-6):
    """x [T, H, D] fp64 rotated by pos [T] (after the RMS norm); (result, bound of the fp32 result's error)."""
    x = x.astype(np.float64)
    D = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight
    half = len(inv_freq)
    z = x.copy()
    size = np.abs(x)
    if half:
        a = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
        i = np.arange(half)
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(a), np.sin(a)
        z[..., i0], z[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i1] * c + x[..., i0] * s
        both = np.abs(x[..., i0]) + np.abs(x[..., i1])
        size[..., i0], size[..., i1] = both, both
    # the norm's square root and products: (D / 2 + 16) fp32 steps; the angle: 1e-6 radians and three
    # roundings per 2^24 positions beyond; cos, sin, two products and a sum: 8 steps
    far = max(1.0, float(np.max(pos)) / 2 ** 24) if np.size(pos) else 1.0
    return z, size * ((8 + (D / 2 + 16 if weight is not None else 0)) * 2.0 ** -23 + 1e-6 * far)


def bf16(x) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()
