"""Plain implementations of the 8-bit paged cache for the tests, from the definitions in include/fadkv.h: codes with numpy,
one block of one head after the other; attention through paged_util in 64 bits."""
import numpy as np

from tests import paged_util as U

E4M3, I8 = "e4m3", "i8"
MOST = {E4M3: 448.0, I8: 127.0}


def _e4m3_table():
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


TABLE = _e4m3_table()


def decode(codes, fmt):
    """float64 of codes (uint8)."""
    return TABLE[codes] if fmt == E4M3 else codes.view(np.int8).astype(np.float64)


def encode(y, fmt):
    """The nearest codes (uint8) of values; ties to the even code."""
    y = np.asarray(y, np.float64)
    if fmt == I8:
        y = np.where(np.isnan(y), 0.0, y)
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    sign = (np.signbit(y) * 128).astype(np.uint8)
    a = np.abs(np.where(np.isfinite(y), y, 0.0))
    hi = np.clip(np.searchsorted(TABLE[:127], a), 1, 126)                     # TABLE[hi - 1] < a <= TABLE[hi]
    lo = hi - 1
    down, up = a - TABLE[lo], TABLE[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(y), code | sign, 127).astype(np.uint8)


def least_scale(a, fmt):
    """The least power of two, 2^-126 at least, with a <= MOST * it."""
    t = 2.0 ** -126
    while a > MOST[fmt] * t:
        t *= 2
    return t


def append(x, slots, pool, scales, ps, block, fmt):
    """x [T][Hkv][d] float64; pool [pages][ps][Hkv][d] uint8 and scales [pages][Hkv][ps / block] float32, written in place."""
    P = pool.shape[0]
    ok = [t for t, s in enumerate(slots) if 0 <= s < P * ps]
    groups = {}
    for t in ok:
        groups.setdefault(int(slots[t]) // block, []).append(t)
    for blk, rows in groups.items():
        page, part = blk * block // ps, blk * block % ps // block
        lo = part * block
        first = min(int(slots[t]) % block for t in rows)
        for h in range(x.shape[1]):
            y = x[rows, h]
            t = least_scale(np.abs(y[np.isfinite(y)]).max(initial=0.0), fmt)
            old = float(scales[page, h, part])
            s = max(old, t) if first else t
            if first and s > old:
                was = decode(pool[page, lo:lo + first, h], fmt)
                pool[page, lo:lo + first, h] = encode(was.astype(np.float32) * (np.float32(old) / np.float32(s)), fmt)
            scales[page, h, part] = s
            inv = np.float32(1.0) / np.float32(s)            # (scales that are no powers of two: as the header says, 32 bits)
            for i, row in enumerate(rows):
                pool[page, int(slots[row]) % ps, h] = encode(y[i].astype(np.float32) * inv, fmt)


def gather(pool, scales, row, length, fmt):
    """[length][Hkv][d] float64 of a pool [pages][ps][Hkv][d] through one block-table row, the scale of each token and head, and
    which tokens lie on a page of the pool."""
    P, ps, hkv, d = pool.shape
    block = ps // scales.shape[2]
    out, sc, ok = np.zeros((length, hkv, d)), np.ones((length, hkv)), np.zeros(length, bool)
    for j in range(length):
        page = int(row[j // ps])
        if 0 <= page < P:
            ok[j] = True
            sc[j] = scales[page, :, j % ps // block]
            out[j] = decode(pool[page, j % ps], fmt) * sc[j][:, None]
    return out, sc, ok


def bounds(out, lse, pv, big, n, most, d, eps, least=2.0 ** -24):
    """Largest errors of out and lse that rounding allows.  As paged_util.bounds with 32-bit scores (their error is 2^-23 of
    `big` for each of d products, and eight more for the scales), and:
      - exponents are differences x - m, x + log2 sv - M and M - m, each rounded in 32 bits: 2^-24 of (1.45 big + 140) three
        times, and log2 sv is off by 2^-21 at most;
      - the weights enter as two binary16 terms: 2^-22 of each; one that is below 2^-36 of the largest is lost, for each of n
        keys that much of the largest weight times value, `most`;
      - exponentials, sums and the joins' weights: 2^-19 of the sum.
    out is rounded once, to multiples of `least` at the low end (half of one; binary16's by default, with as much again)."""
    delta = (d + 8) * 2.0 ** -23 * big + 3 * 2.0 ** -24 * (1.45 * big + 140) + 2.0 ** -21
    rel = 2 * delta[..., None] + 2.0 ** -19 + 2.0 ** -22
    e_out = eps / 2 * np.abs(out) * (1 + rel) + 2 * rel * pv + n * 2.0 ** -36 * most[..., None] + least
    e_lse = 2 * delta + 2.0 ** -19 + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22
    return e_out, e_lse


def attend(q, pool_k, pool_v, scales_k, scales_v, table, lengths, window, sinks, scale, fmt, positions=None):
    """q [B][Hq][d] float64: out, lse and the sizes that bounds() takes."""
    B, Hq, d = q.shape
    res = [np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf), np.zeros((B, Hq, d)), np.zeros((B, Hq)), np.zeros((B, Hq))]
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * pool_k.shape[1])
        if n == 0 or (positions is not None and positions[b] < 0):
            continue
        k, _, ok = gather(pool_k, scales_k, table[b], n, fmt)
        v, sv, _ = gather(pool_v, scales_v, table[b], n, fmt)
        got = U.attend_rows(q[b:b + 1], k, np.where(ok[:, None, None], v, 0), ok, [n - 1], window, sinks, scale)
        for r, g in zip(res, got):
            r[b] = g[0]
        # no key has more than all of the weight
        seen = ok & (np.arange(n) <= n - 1) & ((window == 0) | (np.arange(n) > n - 1 - window) | (np.arange(n) < sinks))
        grp = Hq // k.shape[1]
        if seen.any():
            res[4][b] = np.repeat(sv[seen].max(0), grp) * MOST[fmt]
    return res
