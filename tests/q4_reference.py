"""The 4-bit cache restated in 64-bit numpy from its definition, and its pools taken
apart byte by byte (test infrastructure)."""

import numpy as np

GROUP = 32


def quantise(x):
    """x [..., D] -> n (int), s, m (float64 [..., D / 32]); s NaN and m 0 for a group that
    has no finite pair."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        m = lo.astype(np.float16)
        m = np.where(m.astype(np.float64) > lo, np.nextafter(m, np.float16(-np.inf)), m)
        y = (hi - m.astype(np.float64)) / 15.0
        s = y.astype(np.float16)
        # (fp16 has 11 bits, so that 15 s is exact here and decides)
        s = np.where(15.0 * s.astype(np.float64) < hi - m.astype(np.float64),
                     np.nextafter(s, np.float16(np.inf)), s)
        m, s = m.astype(np.float64), s.astype(np.float64)
        bad = ~(np.isfinite(m) & np.isfinite(s) & np.isfinite(lo) & np.isfinite(hi))
        d = (g - m[..., None]) / np.where(s > 0, s, 1.0)[..., None]
        n = np.where((s > 0)[..., None] & ~bad[..., None], np.floor(d + 0.5), 0.0)
    return (n.astype(np.int64).reshape(x.shape), np.where(bad, np.nan, s), np.where(bad, 0.0, m))


def values(n, s, m):
    g = n.reshape(*n.shape[:-1], -1, GROUP).astype(np.float64)
    return (m[..., None] + s[..., None] * g).reshape(n.shape)


def record_bytes(D):
    return D // 2 + D // 8


def unpack(pool, Hkv, D, kind):
    """pool uint8 [num_pages, page_size, row] -> n [N, P, Hkv, D], s, m [N, P, Hkv, D / 32]."""
    N, P, row = pool.shape
    NB = D // GROUP
    rec = pool[:, :, :Hkv * record_bytes(D)].reshape(N, P, Hkv, record_bytes(D))
    code = rec[..., :D // 2]
    nib = np.stack([code & 15, code >> 4], -1).reshape(N, P, Hkv, D)  # in order of the bits
    per = 8 if kind == "k" else 4  # values of a word, which are NB words apart
    n = nib.reshape(N, P, Hkv, GROUP // per, NB, per)
    n = np.moveaxis(n, 4, 3).reshape(N, P, Hkv, D).astype(np.int64)
    pair = np.ascontiguousarray(rec[..., D // 2:]).view(np.float16).reshape(N, P, Hkv, NB, 2)
    with np.errstate(invalid="ignore"):
        return n, pair[..., 0].astype(np.float64), pair[..., 1].astype(np.float64)


def places(lens, table, starts, page):
    """(row, page, slot) of every row that has a place."""
    out = []
    for b, n in enumerate(lens):
        if not 0 <= n <= len(table[b]) * page:
            continue
        for i in range(starts[b], starts[b + 1]):
            pos = n - starts[b + 1] + i
            if 0 <= pos < n:
                out.append((i, table[b][pos // page], pos % page))
    return out
