"""Plain forms of planned steps, the rotary write by slots, block bounds, block selection (numpy, one loop per
sequence, row or block; whole numbers and 64 bits)."""
from __future__ import annotations

import numpy as np

from mod_reference import rotate


def plan(table, lens, new, stack, count, n_rows, bs):
    """One step, sequence by sequence: (table, stack, count, lens_out, cu, slots, positions, seq_ids)."""
    table, stack = table.copy(), stack.copy()
    up = lambda n: -(-int(n) // bs)
    top = int(count)
    for b, (a, z) in enumerate(zip(lens, new)):
        for j in range(up(z), up(a)):
            stack[top] = table[b, j]
            top += 1
    out, cu, rows, full, asked = [], [0], [], False, 0
    for b, (a, z) in enumerate(zip(lens, new)):
        if z > a:
            asked += z - a
            full = full or up(z) - up(a) > top or asked > n_rows
            if not full:
                for j in range(up(a), up(z)):
                    top -= 1
                    table[b, j] = stack[top]
                rows += [(table[b, p // bs] * bs + p % bs, p, b) for p in range(a, z)]
        out.append(a if z > a and full else z)
        cu.append(len(rows))
    rows += [(-1, -1, -1)] * (n_rows - len(rows))
    s, p, q = np.array(rows, dtype=np.int32).reshape(n_rows, 3).T
    return table, stack, top, np.array(out, np.int32), np.array(cu, np.int32), s, p, q


def rotate_axes(x, positions, axis_of, inv_freq, interleaved, weight=None, eps=1e-6):
    """rotate() with the angle of frequency i from positions[axis_of[i]]: (result, error bound)."""
    half = len(inv_freq)
    z = tol = None
    for a in range(len(positions)):
        za, ta = rotate(x, np.abs(positions[a]) * 0 + positions[a], inv_freq, interleaved, weight, eps)
        if z is None:
            z, tol = za, ta
            continue
        i = np.array([k for k in range(half) if axis_of[k] == a], dtype=int)
        ch = np.concatenate([2 * i, 2 * i + 1]) if interleaved else np.concatenate([i, i + half])
        z[..., ch] = za[..., ch]
        tol = np.maximum(tol, ta)
    return z, tol


def unit_exponent(top):
    """The smallest e in [-100, 100] with top <= 127 * 2^e."""
    e = -100
    while e < 100 and not top <= 127.0 * 2.0 ** e:
        e += 1
    return e


def bounds_of(k):
    """Codes [2, D] and unit of keys k [n, D] (fp64 of fp32 values)."""
    hi = np.where(np.isnan(k), np.inf, k).max(0)
    lo = np.where(np.isnan(k), -np.inf, k).min(0)
    unit = 2.0 ** unit_exponent(max(np.abs(hi).max(), np.abs(lo).max()))
    return np.clip(np.stack([np.ceil(hi / unit), np.floor(lo / unit)]), -127, 127).astype(np.int8), np.float32(unit)


def whole_queries(q):
    """A group's queries [g, D] (fp64) as the integers that the score takes."""
    q = np.where(np.isnan(q), 0.0, q)
    z = q / 2.0 ** unit_exponent(np.abs(q).max())
    return np.clip(np.rint(z), -127, 127).astype(np.int64)


def block_scores(q, codes, units):
    """score_j of every block: q [g, D], codes [n, 2, D], units [n]."""
    w = whole_queries(q)
    c = codes.astype(np.int64)
    s = np.stack([np.where(x > 0, c[:, 0], c[:, 1]) @ x for x in w]).max(0)
    return s.astype(np.float64) * units.astype(np.float64)


def choose(score, ok, top_k, sink, recent):
    """The listed blocks, ascending, then -1: score [nb], ok [nb] (a readable table entry)."""
    nb = len(score)
    forced = [j for j in range(nb) if ok[j] and (j < sink or j >= nb - recent)]
    rest = sorted((j for j in range(nb) if ok[j] and j not in set(forced)), key=lambda j: (-score[j], j))
    pick = sorted(forced + rest[:max(0, top_k - len(forced))])
    return np.array(pick + [-1] * (top_k - len(pick)), np.int32)
