"""The 8-bit block cache and its attention in numpy, from the definitions:
appends in fp32 steps (bit for bit what the kernels must give), attention in
64 bits with a bound of its error."""
from __future__ import annotations

import numpy as np

BLOCK = 64


def round_away(x):
    x = np.asarray(x, np.float32)
    t = np.trunc(x)
    return t + np.copysign(1.0, x) * (np.abs(x - t) >= 0.5)


def split(codes, dim):
    """Codes [.., 2, heads, 64 * dim] -> keys and values [.., heads, slot, dim] (views)."""
    k = codes[..., 0, :, :].reshape(codes.shape[:-3] + (codes.shape[-2], BLOCK, dim))
    v = codes[..., 1, :, :].reshape(codes.shape[:-3] + (codes.shape[-2], dim, BLOCK))
    return k, np.swapaxes(v, -1, -2)


def rows_of(start, n_seqs, n_tok, max_q):
    """First row and count of each sequence."""
    if start is None:
        return [(s * max_q, max_q) for s in range(n_seqs)]
    out = []
    for s in range(n_seqs):
        a = min(max(int(start[s]), 0), n_tok)
        b = min(max(int(start[s + 1]), a), n_tok)
        out.append((a, min(b - a, max_q)))
    return out


def append(codes, scales, table, lens, start, max_q, k, v):
    """Changes codes and scales in place."""
    n_blocks, _, heads, _ = codes.shape
    dim = k.shape[2]
    for s, (t0, n) in enumerate(rows_of(start, len(lens), k.shape[0], max_q)):
        length = max(int(lens[s]), 0)
        first = max(length - n, 0)
        for b in range(first // BLOCK, min(-(-length // BLOCK), table.shape[1])):
            at = int(table[s, b])
            if not 0 <= at < n_blocks:
                continue
            lo, hi = max(first, b * BLOCK), min(length, (b + 1) * BLOCK)
            if lo >= hi:
                continue
            a, z = lo - b * BLOCK, hi - b * BLOCK
            rows = slice(t0 + lo - (length - n), t0 + hi - (length - n))
            for part, x in ((0, k), (1, v)):
                for h in range(heads):
                    xs = x[rows, h].astype(np.float32)
                    plane = codes[at, part, h].reshape((BLOCK, dim) if part == 0 else (dim, BLOCK))
                    c = plane if part == 0 else plane.T
                    old = scales[at, part, h] if a > 0 else np.float32(0)
                    d = np.maximum(old, np.abs(xs).max() / np.float32(127.0))
                    if old > 0 and d > old:
                        c[:a] = np.clip(round_away(c[:a].astype(np.float32) * (old / d)), -127, 127)
                    c[a:z] = np.clip(round_away(xs / d), -127, 127) if d > 0 else 0
                    scales[at, part, h] = d


def attend(codes, scales, table, lens, start, max_q, q, scale, window):
    """(out, tol, rows): the attention of every row of a sequence in 64 bits,
    how far an fp32 result with 24-bit operands may be from it, and which rows
    belong to a sequence.

    With u = 2^-24: an element of q is off by at most 2 u of its row's largest
    (rounded to half a unit of 1/(127 2^16) of it, and the product before that),
    a score besides by 10 roundings of its own size (integer sums to fp32,
    their fma, the factors dq dk scale log2(e), the difference from the
    maximum) and the exponential by 2.  A weight is rounded to half a unit:
    units are 2/(127 2^16) of what p dv may be 2^1 above and, at the largest of
    its block, 2^-4 below, so half of one is at most 2^4/(127 2^16) < 2^-18.98
    < 33 u of the block's largest.  The sums over T blocks, and the joins of up
    to 68 partial sums, are off by 4 (T + 72) roundings."""
    n_blocks, _, heads, _ = codes.shape
    n_tok, n_heads, dim = q.shape
    group, u = n_heads // heads, 2.0 ** -24
    kk, vv = split(codes, dim)
    out, tol, rows = np.zeros(q.shape), np.zeros(q.shape), np.zeros(n_tok, bool)
    for s, (t0, n) in enumerate(rows_of(start, len(lens), n_tok, max_q)):
        length = max(int(lens[s]), 0)
        width = min(-(-length // BLOCK), table.shape[1])
        ids = table[s, :width]
        ok = (ids >= 0) & (ids < n_blocks)
        pos_of = (np.arange(width)[:, None] * BLOCK + np.arange(BLOCK))[ok].reshape(-1)
        ids = ids[ok]
        sc = scales[ids].astype(np.float64)
        kf = kk[ids].astype(np.float64) * sc[:, 0, :, None, None]
        vf = vv[ids].astype(np.float64) * sc[:, 1, :, None, None]
        for i in range(n):
            rows[t0 + i] = True
            p = length - n + i
            seen = pos_of <= p
            if window:
                seen &= pos_of > p - window
            if p < 0 or not seen.any():
                continue
            for h in range(n_heads):
                kx = kf[:, h // group].reshape(-1, dim)[seen]
                vx = vf[:, h // group].reshape(-1, dim)[seen]
                qx = q[t0 + i, h].astype(np.float64)
                score = scale * (kx @ qx)
                e = np.exp(score - score.max())
                w = e / e.sum()
                out[t0 + i, h] = w @ vx
                ds = 2 * u * abs(scale) * np.abs(qx).max() * np.abs(kx).sum(1)
                ds += 10 * u * (np.abs(score) + np.abs(score - score.max())) + 2 * u
                tiles = pos_of[seen] // BLOCK
                _, inv = np.unique(tiles, return_inverse=True)
                big = np.zeros(inv.max() + 1)
                np.maximum.at(big, inv, w)
                a = np.abs(vx)
                tol[t0 + i, h] = (w * (ds + w @ ds)) @ a + 4 * u * (inv.max() + 73) * (w @ a) + 33 * u * (big[inv] @ a)
    return out, tol, rows
