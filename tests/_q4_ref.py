"""Plain 64-bit forms of the calls around 4-bit rows and eviction.

A held row is 384 bytes: codes of dims 0-447 (eight dims a little-endian word,
even dims in its low half), 28 e4m3 scales, a power of two, dims 448-511 bf16.
"""

import numpy as np
import torch

from tests import _paged_ref as ref

EVICTED = -2 ** 31
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3(code):
    """Value of an e4m3 byte without a sign (0x7f: NaN)."""
    m, e = code & 7, code >> 3
    v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return np.nan if code == 0x7F else v


E4M3 = np.array([e4m3(c) for c in range(128)])


def nearest(x, values):
    """Index of the value nearest to x >= 0, the even index of two."""
    i = int(np.searchsorted(values, x))
    if i == 0:
        return 0
    if i == len(values):
        return len(values) - 1
    lo, hi = x - values[i - 1], values[i] - x
    return i - 1 if lo < hi or (lo == hi and (i - 1) % 2 == 0) else i


def pack_row(x):
    """Bytes of one row x [512] (fp32 values as fp64), rotary dims as they are."""
    out = np.zeros(384, np.uint8)
    g = x[:448].reshape(28, 16)
    fine = np.isfinite(g)
    top = np.where(fine, np.abs(g), 0.0).max(1)
    sixth = (top.astype(np.float32) / np.float32(6)).astype(np.float64)
    unit = sixth.max()
    e = -100 if unit == 0 else int(np.clip(np.frexp(unit)[1] - 1 - 7, -100, 100))
    out[252] = e + 127
    words = np.zeros(56, np.uint32)
    for i in range(28):
        bad = not fine[i].all()
        s = 0x7F if bad else nearest(min(sixth[i] * 2.0 ** -e, 448.0), E4M3[:127])
        out[224 + i] = s
        scale = 0.0 if bad else E4M3[s] * 2.0 ** e
        for d in range(16):
            v = g[i, d]
            code = nearest(abs(v) / scale, VALUES) if scale > 0 and np.isfinite(v) else 0
            code |= 8 if np.signbit(v) else 0
            dim = 16 * i + d
            nib = (dim % 8) // 2 + 4 * (dim % 2)
            words[dim // 8] |= np.uint32(code << (4 * nib))
    out[:224] = words.astype("<u4").view(np.uint8)
    tail = torch.from_numpy(x[448:].astype(np.float32)).bfloat16().view(torch.int16).numpy()
    out[256:] = tail.astype("<i2").view(np.uint8)
    return out


def pack(x):
    return np.stack([pack_row(r) for r in x]) if len(x) else np.zeros((0, 384), np.uint8)


def unpack(b):
    """fp64 rows [N, 512] of bytes [N, 384]."""
    n = b.shape[0]
    words = np.ascontiguousarray(b[:, :224]).view("<u4")
    dim = np.arange(448)
    nib = (dim % 8) // 2 + 4 * (dim % 2)
    code = (words[:, dim // 8] >> (4 * nib).astype(np.uint32)) & 15
    scale = np.where(b[:, 224:252] == 0x7F, np.nan, E4M3[np.minimum(b[:, 224:252], 127)])
    scale = scale * 2.0 ** (b[:, 252].astype(np.float64) - 127)[:, None]
    y = np.empty((n, 512))
    y[:, :448] = np.where(code >= 8, -1.0, 1.0) * VALUES[code & 7] * scale[:, dim // 16]
    tail = np.ascontiguousarray(b[:, 256:]).view("<u2").astype(np.uint32) << 16
    y[:, 448:] = tail.view(np.float32)
    return y


def held(cache):
    """A 4-bit cache's values as a bf16 cache of the same pages (exact)."""
    n, page, _ = cache.shape
    y = unpack(cache.cpu().numpy().reshape(-1, 384))
    v = torch.from_numpy(y).to(torch.bfloat16)
    assert np.array_equal(v.double().numpy(), y, equal_nan=True)
    return v.view(n, page, 512)


def random_cache(gen, pages, page, spread=1.0):
    """4-bit cache [pages, page, 384] with rows of normal values: packed here by
    torch where `pack_row` would take long, scales and codes drawn."""
    n = pages * page
    b = torch.randint(0, 256, (n, 384), generator=gen, dtype=torch.uint8)
    # scales 2^0 .. 2^4.8 (bytes 56 .. 94) under 2^(e - 127): values up to 6
    b[:, 224:252] = torch.randint(56, 95, (n, 28), generator=gen, dtype=torch.uint8)
    b[:, 252] = torch.randint(122, 124, (n,), generator=gen, dtype=torch.uint8)
    b[:, 253:256] = 0
    tail = (torch.randn((n, 64), generator=gen) * spread).bfloat16()
    b[:, 256:] = tail.view(torch.uint8)
    return b.view(pages, page, 384)


def mass(q, lse, cmp, idx, table, q_seq, q_pos, base, scale, ratio):
    """(out, tol). With d the largest error of a logit as in _paged_ref.attention
    (512 * 2^-24 of the sum of magnitudes, scaled) and 2^-22 (|l| + |lse| + 4)
    for the exponent's product, subtraction and ex2, a weight is off by 2 of it
    relative; 64 heads are summed (64 * 2^-24); a fixed-point sum rounds each
    weight by 2^-40 at most; two roundings to 32 bits at the end."""
    out = f64(base) if base is not None else np.zeros((table.shape[0], table.shape[1] * cmp.shape[1]))
    got, err = np.zeros_like(out), np.zeros_like(out)
    qn, ln = f64(q), f64(lse)
    for t in range(q.shape[0]):
        if q_pos[t] < 0:
            continue
        b, nv = int(q_seq[t]), (int(q_pos[t]) + 1) // ratio
        want = range(nv) if idx is None else [int(j) for j in idx[t] if 0 <= j < nv]
        rows, keys = ref.gather(cmp, table, cmp.shape[1], b, want)
        if not len(rows):
            continue
        logit = scale * (qn[t] @ keys.T)                       # [H, n]
        live = np.isfinite(ln[t])
        l = np.where(live, ln[t], 0.0)[:, None]
        w = np.where(live[:, None], np.exp(logit - l), 0.0)
        d = 512 * ref.U32 * scale * (np.abs(qn[t]) @ np.abs(keys).T)
        d = d + 2.0 ** -22 * (np.abs(logit) + np.abs(l) + 4.0)
        np.add.at(got[b], rows, w.sum(0))
        np.add.at(err[b], rows, (w * (2 * d + 64 * ref.U32)).sum(0) + 2.0 ** -40)
    res = out + got
    return res, err + 2 * ref.U32 * (np.abs(res) + np.abs(out))


def f64(t):
    return ref.f64(t)


def evict(mass, pages, rows, page, keep, first=0, last=0):
    out, freed = pages.copy(), np.full(pages.shape, -1, np.int32)
    n_freed = np.zeros(len(pages), np.int32)
    for b in range(len(pages)):
        n = min(max(int(rows[b]), 0), pages.shape[1] * page)
        held, safe = [], 0
        for p in range(-(-n // page)):
            if pages[b, p] < 0:
                continue
            lo, hi = p * page, (p + 1) * page
            if lo < first or hi > max(n - last, 0):
                safe += 1
            else:
                held.append((np.float64(mass[b, lo:min(hi, n)].astype(np.float64).sum()), p))
        held.sort(key=lambda x: (-np.inf if np.isnan(x[0]) else -x[0], x[1]))
        held.sort(key=lambda x: not np.isnan(x[0]))
        gone = sorted(p for _, p in held[max(keep - safe, 0):])
        for i, p in enumerate(gone):
            freed[b, i] = pages[b, p]
            out[b, p] = EVICTED
        n_freed[b] = len(gone)
    return out, freed, n_freed
