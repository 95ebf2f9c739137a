"""Plain 64-bit forms of the rotation and the paged-cache operators, and the
error bounds of the library's arithmetic against them.

A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24.
"""

import math

import numpy as np
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def rope(x, pos, freqs, off, half, mscale=1.0, inverse=False):
    """(y, mag): x [T, H, D] turned, and |x_a| + |x_b| at the turned dims."""
    y, mag = x.copy(), np.zeros_like(x)
    n = 2 * len(freqs)
    for i, f in enumerate(freqs):
        a, b = (off + i, off + i + n // 2) if half else (off + 2 * i, off + 2 * i + 1)
        ang = np.asarray(pos, dtype=np.float64) * f * (-1.0 if inverse else 1.0)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y[..., a] = mscale * (x[..., a] * c - x[..., b] * s)
        y[..., b] = mscale * (x[..., b] * c + x[..., a] * s)
        mag[..., a] = mag[..., b] = abs(mscale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, mag


def rope_tol(y, mag, bf16):
    """The reduced angle is a fraction of a turn held to 2^-26 (2^-23.3
    radians), sincospif is off by 2 units (2^-23), times mscale and two
    products and a sum round 3 times by 2^-24: below 2^-21 of |x_a| + |x_b|
    together. bf16 output: 2^-8 of the value on top."""
    t = 2.0 ** -21 * mag
    return t + U16 * (np.abs(y) + t) if bf16 else t


def pool_rows(lengths, page, extra=2, seed=0, keep_from=None):
    """Page table [B, pages] holding `lengths` rows each (-1 past the end and
    below keep_from), pool pages in random order; (table, pool pages)."""
    rng = np.random.default_rng(seed)
    n = [-(-int(x) // page) for x in lengths]
    total = sum(n) + extra
    perm = rng.permutation(total)
    table = np.full((len(lengths), max(1, max(n, default=1))), -1, np.int32)
    at = 0
    for b, k in enumerate(n):
        for p in range(k):
            table[b, p] = perm[at]
            at += 1
            if keep_from is not None and (p + 1) * page <= keep_from[b]:
                table[b, p] = -1
    return table, total


def slot(table, page, b, r):
    """(page, row in page) of row r of sequence b, or None."""
    if r < 0 or r // page >= table.shape[1] or table[b, r // page] < 0:
        return None
    return int(table[b, r // page]), int(r % page)


def gather(cache, table, page, b, rows):
    """(rows present, their values fp64)."""
    keep = [r for r in rows if slot(table, page, b, r) is not None]
    if not keep:
        return keep, np.zeros((0, cache.shape[2]))
    s = np.array([slot(table, page, b, r) for r in keep])
    return keep, f64(cache[torch.from_numpy(s[:, 0]).to(cache.device),
                           torch.from_numpy(s[:, 1]).to(cache.device)])


def indexer(q, cache, w, table, q_seq, q_pos, ratio, topk):
    T = q.shape[0]
    page = cache.shape[1]
    idx = np.full((T, topk), -1, np.int64)
    val = np.full((T, topk), -np.inf)
    qn, wn = f64(q), f64(w)
    for t in range(T):
        if q_pos[t] < 0:
            continue
        n = (int(q_pos[t]) + 1) // ratio
        if n == 0:
            continue
        rows, k = gather(cache, table, page, int(q_seq[t]), range(n))
        assert len(rows) == n
        s = np.maximum(k @ qn[t].T, 0.0) @ wn[t]
        best = np.sort(np.argsort(-s, kind="stable")[:topk])
        idx[t, :len(best)], val[t, :len(best)] = best, s[best]
    return idx, val


def attention(q, ori, cmp, idx, ori_table, cmp_table, q_seq, q_pos, sinks, scale, ratio, win_left):
    """(out, lse, out_tol, lse_tol). With d the largest error of a logit (each
    of 512 products and sums in fp32 rounds once: 512 * 2^-24 of the sum of
    magnitudes; ex2 of a scaled logit adds 2^-22 (|l| + 4)), a weight is off by
    at most 2 d relative before its bf16 rounding (2^-8); out is rounded once."""
    T, H, _ = q.shape
    out = np.zeros((T, H, 512))
    lse = np.full((T, H), -np.inf)
    out_tol, lse_tol = np.zeros((T, H, 512)), np.zeros((T, H))
    qn = f64(q)
    sk = None if sinks is None else f64(sinks)
    for t in range(T):
        if q_pos[t] < 0:
            continue
        b, p = int(q_seq[t]), int(q_pos[t])
        _, keys = gather(ori, ori_table, ori.shape[1], b, range(max(0, p - win_left), p + 1))
        if cmp is not None:
            nv = (p + 1) // ratio
            want = range(nv) if idx is None else [int(j) for j in idx[t] if 0 <= j < nv]
            _, more = gather(cmp, cmp_table, cmp.shape[1], b, want)
            keys = np.concatenate([keys, more])
        logit = scale * (qn[t] @ keys.T)
        full = logit if sk is None else np.concatenate([logit, sk[:, None]], 1)
        if full.shape[1] == 0:
            continue
        m = full.max(1, keepdims=True)
        z = np.exp(full - m).sum(1)
        prob = np.exp(logit - m) / z[:, None]
        out[t] = prob @ keys
        lse[t] = m[:, 0] + np.log(z)
        if keys.shape[0]:
            d = 512 * U32 * scale * (np.abs(qn[t]) @ np.abs(keys).T).max(1)
            d += 2.0 ** -22 * (np.abs(full).max(1) + 4.0)
        else:
            d = 2.0 ** -22 * (np.abs(full).max(1) + 4.0)
        spread = prob @ np.abs(keys)
        tol = (U16 + 2 * d[:, None]) * spread
        out_tol[t] = tol + U16 * (np.abs(out[t]) + tol) + 1e-30
        lse_tol[t] = 2 * d + U32 * 8 * (np.abs(lse[t]) + 1.0)
    return out, lse, out_tol, lse_tol


def check(got, want, tol, what=""):
    g = f64(got)
    same = (g == want)                     # equal infinities
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(g - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / (tol + 1e-300), -1)), g.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, worst at {i}: "
                             f"{g[i]} for {want[i]}, bound {np.broadcast_to(tol, g.shape)[i]}")


def grid(gen, shape, step, dtype):
    x = torch.randn(shape, generator=gen)
    return (torch.round(x / step) * step).to(dtype)


def inv_sqrt(d):
    return 1.0 / math.sqrt(d)
