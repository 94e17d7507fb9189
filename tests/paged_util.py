"""Plain implementations of the paged-cache operators for the tests: whole
numbers with Python loops, attention and rotation in 64 bits with numpy, from
the definitions in include/fadkv.h."""
import math

import numpy as np


def plan(add, lengths, table, free, count, page_size, max_tokens):
    """One request after the other, one page after the other."""
    ps, mp, P = page_size, table.shape[1], len(free)
    table, free = table.copy(), free.copy()
    lens = [min(max(int(l), 0), mp * ps) for l in lengths]
    count = min(max(int(count), 0), P)
    pages = lambda n: -(-n // ps)
    for b, a in enumerate(add):
        if a < 0:
            for j in range(pages(lens[b])):
                if count < P:
                    free[count] = table[b, j]
                    count += 1
    F, asked, taken, refused = count, 0, 0, 0
    starts, out = [0], list(lens)
    positions, slots = np.full(max_tokens, -1, np.int32), np.full(max_tokens, -1, np.int32)
    for b, a in enumerate(add):
        n = max(int(a), 0)
        s = starts[-1]
        starts.append(min(s + n, 2 ** 31 - 1))
        if a < 0:
            out[b] = 0
        if n == 0:
            continue
        new = lens[b] + n
        if new > mp * ps:
            refused += 1
            continue
        need = pages(new) - pages(lens[b])
        asked += need
        if s + n > max_tokens or (need > 0 and asked > F):
            refused += 1
            continue
        for j in range(need):
            table[b, pages(lens[b]) + j] = free[F - 1 - taken]
            taken += 1
        out[b] = new
        for i in range(n):
            pos = lens[b] + i
            page = int(table[b, pos // ps])
            positions[s + i] = pos
            slots[s + i] = page * ps + pos % ps if 0 <= page < P else -1
    i32 = lambda x: np.array(x, np.int32)
    return dict(table=table, free=free, lengths=i32(out), count=i32([F - taken]), starts=i32(starts), positions=positions,
                slots=slots, refused=i32([refused]))


def frequencies(rd, base=10000.0, scaling="plain", factor=1.0, original=8192.0, slow=1.0, fast=4.0):
    out = []
    for i in range(rd // 2):
        b = base * factor ** (rd / (rd - 2)) if scaling == "stretch" else base
        f = b ** (-2.0 * i / rd)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            g = min(1.0, max(0.0, (original * f / (2 * math.pi) - slow) / (fast - slow)))
            f *= g + (1 - g) / factor
        out.append(f)
    return np.array(out)


def norm_rope(x, w, eps, positions, freq, rd, interleaved, amplitude):
    """float64 [T][H][d], and for each value the size of what was added to
    make it (the scale of its rounding errors)."""
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    ang = positions.astype(np.float64)[:, None] * freq[None]
    c, s = np.cos(ang)[:, None] * amplitude, np.sin(ang)[:, None] * amplitude
    y, mag = x.copy(), np.abs(x)
    ia, ib = (np.arange(0, rd, 2), np.arange(1, rd, 2)) if interleaved else (np.arange(rd // 2), np.arange(rd // 2, rd))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = (np.abs(a) + np.abs(b)) * abs(amplitude)
    dead = positions < 0
    y[dead], mag[dead] = 0, 0
    return y, mag


def gather(pool, row, length, layout):
    """[length][Hkv][d] float64 of a pool through one block-table row, and which tokens lie on a page of the pool."""
    ps = pool.shape[2] if layout == "head" else pool.shape[1]
    hkv, d = (pool.shape[1] if layout == "head" else pool.shape[2]), pool.shape[3]
    out, ok = np.zeros((length, hkv, d)), np.zeros(length, bool)
    for j in range(length):
        page = int(row[j // ps])
        if 0 <= page < pool.shape[0]:
            ok[j] = True
            out[j] = pool[page, :, j % ps] if layout == "head" else pool[page, j % ps]
    return out, ok


def attend_rows(q, k, v, ok, positions, window, sinks, scale):
    """q [n][Hq][d], k, v [len][Hkv][d] float64: out, lse, sum p |v| and the largest sum |q_i k_i| scale of a seen key."""
    n, Hq, d = q.shape
    grp = Hq // k.shape[1]
    out, pv = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, big = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    j = np.arange(k.shape[0])
    for i in range(n):
        p = positions[i]
        seen = (j <= p) & ok
        if window > 0:
            seen &= (j > p - window) | (j < sinks)
        if not seen.any():
            continue
        for h in range(Hq):
            kh, vh = k[seen, h // grp], v[seen, h // grp]
            x = kh @ q[i, h] * scale
            m = x.max()
            e = np.exp(x - m)
            l = e.sum()
            out[i, h], pv[i, h], lse[i, h] = e @ vh / l, e @ np.abs(vh) / l, m + np.log(l)
            big[i, h] = (np.abs(kh) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, pv, big


def bounds(out, lse, pv, big, d, eps, p_terms):
    """Largest errors of out and lse that rounding allows.  Scores: d products summed in 32 bits (2^-23 each, the
    tensor pipe may truncate), then scale and exponent; an error x of a score is a factor within 2x of p.  The
    probabilities are rounded to the 16-bit type (p_terms = 1: half a step, eps / 2) or to two such terms; the
    exponential and the sums of p and p v add 2^-20 of the sum.  out is rounded once."""
    delta = (d + 8) * 2.0 ** -23 * big
    rel = 2 * delta[..., None] + 2.0 ** -20 + (eps / 2 if p_terms == 1 else (eps / 2) ** 2)
    e_out = eps / 2 * np.abs(out) * (1 + rel) + 2 * rel * pv + 2.0 ** -24
    e_lse = 2 * delta + 2.0 ** -20 + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22
    return e_out, e_lse
