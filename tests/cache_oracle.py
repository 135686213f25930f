"""The key/value cache's operators from their definitions, in 64 bits on the
CPU with numpy, position by position.  Shares no code with the library.

A cache here is a dict: k, v uint8 arrays [pages, heads, page, dim] in token
order (to_stored / from_stored convert the library's layouts), scales uint8
[pages, heads, 2], codes "e4m3" or "int8".
"""
import numpy as np

LOWEST = -100
TOP = {"e4m3": 448.0, "int8": 127.0}


def _e4m3_values():
    out = []
    for c in range(128):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    out[127] = np.nan
    return np.array(out)


_E4M3 = _e4m3_values()
_MIDDLES = (_E4M3[:126] + _E4M3[1:127]) / 2


def value(codes, kind):
    codes = np.asarray(codes, np.uint8)
    if kind == "int8":
        return codes.view(np.int8).astype(np.float64)
    x = _E4M3[codes & 127]
    return np.where(codes & 128, -x, x)


def code(x, kind):
    """Nearest code, ties to even; infinities saturate; NaN is E4M3's NaN or 0."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), TOP[kind])
    if kind == "int8":
        return np.where(np.isnan(x), 0, np.copysign(np.rint(a), x)).astype(np.int8).view(np.uint8)
    a0 = np.where(np.isnan(a), 0.0, a)
    below = np.searchsorted(_MIDDLES, a0, side="left")   # middles strictly below a
    tie = (below < 126) & (_MIDDLES[np.minimum(below, 125)] == a0) & (below % 2 == 1)
    c = np.where(np.isnan(x), 127, below + tie)
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def to_stored(k, v):
    p, h, t, d = k.shape
    return (np.ascontiguousarray(k.reshape(p, h, t // 16, 16, d // 16, 16).swapaxes(3, 4)),
            np.ascontiguousarray(v.reshape(p, h, t // 16, 16, d).swapaxes(3, 4)))


def from_stored(k, v):
    p, h, b = k.shape[:3]
    d = v.shape[3]
    return (np.ascontiguousarray(k.swapaxes(3, 4)).reshape(p, h, b * 16, d),
            np.ascontiguousarray(v.swapaxes(3, 4)).reshape(p, h, b * 16, d))


def spans(cu, lengths, rows, capacity):
    """(row0, n, start, ok) of each sequence; a refused one has ok False."""
    if cu is None:
        cu = list(range(len(lengths) + 1))
    out = []
    for i, length in enumerate(lengths):
        c0, c1 = int(cu[i]), int(cu[i + 1])
        ok = 0 <= c0 <= c1 <= rows and 0 <= length <= capacity and length >= c1 - c0
        r0, r1 = min(max(c0, 0), rows), min(max(c1, 0), rows)
        out.append((r0, max(r1 - r0, 0), length - (c1 - c0) if ok else 0, ok))
    return out


def _page(cache, table, i, j):
    p = int(table[i][j])
    return p if 0 <= p < len(cache["scales"]) else None


def write(cache, k, v, table, lengths, cu=None):
    """The cache after the call (a copy) and the status bits."""
    c = {**cache, "k": cache["k"].copy(), "v": cache["v"].copy(), "scales": cache["scales"].copy()}
    kind, P = c["codes"], c["k"].shape[2]
    status = 0
    for i, (r0, n, start, ok) in enumerate(spans(cu, lengths, len(k), len(table[0]) * P)):
        if not ok:
            status |= 2
        if not ok or not n:
            continue
        for j in range(start // P, (start + n - 1) // P + 1):
            p = _page(c, table, i, j)
            if p is None:
                status |= 1
                continue
            lo, hi = max(start, j * P), min(start + n, (j + 1) * P)
            t0, t1 = lo - j * P, hi - j * P
            for which, x in (("k", k), ("v", v)):
                kd = 0 if which == "k" else 1
                y = x[r0 + lo - start:r0 + hi - start].astype(np.float64)  # [t, H, D]
                for h in range(y.shape[1]):
                    a = np.abs(y[:, h])
                    a = a[np.isfinite(a)]
                    largest = a.max() if a.size else 0.0
                    e = LOWEST
                    while largest > TOP[kind] * 2.0 ** e:
                        e += 1
                    if t0:
                        before = int(c["scales"][p, h, kd]) - 127
                        if before > e:
                            e = before
                        elif e > before:
                            c[which][p, h, :t0] = code(value(c[which][p, h, :t0], kind) * 2.0 ** (before - e), kind)
                    with np.errstate(invalid="ignore"):
                        c[which][p, h, t0:t1] = code(y[:, h] / 2.0 ** e, kind)
                    c["scales"][p, h, kd] = e + 127
    return c, status


def _gather(cache, table, i, j0, j1, which):
    """Values [H, (j1 - j0) * P, D] of the sequence's pages, and whether each position has a page."""
    P = cache["k"].shape[2]
    H, D = cache["k"].shape[1], cache["k"].shape[3]
    out, have = np.zeros((H, (j1 - j0) * P, D)), np.zeros((j1 - j0) * P, bool)
    for j in range(j0, j1):
        p = _page(cache, table, i, j)
        if p is None:
            continue
        s = 2.0 ** (cache["scales"][p, :, 0 if which == "k" else 1].astype(np.float64) - 127)
        out[:, (j - j0) * P:(j - j0 + 1) * P] = value(cache[which][p], cache["codes"]) * s[:, None, None]
        have[(j - j0) * P:(j - j0 + 1) * P] = True
    return out, have


def read(cache, table, lengths, cu, rows):
    P, H, D = cache["k"].shape[2], cache["k"].shape[1], cache["k"].shape[3]
    k, v, status = np.zeros((rows, H, D)), np.zeros((rows, H, D)), 0
    for i, (r0, n, start, ok) in enumerate(spans(cu, lengths, rows, len(table[0]) * P)):
        if not ok:
            status |= 2
        if not ok or not n:
            continue
        j0, j1 = start // P, (start + n - 1) // P + 1
        for which, out in (("k", k), ("v", v)):
            x, have = _gather(cache, table, i, j0, j1, which)
            out[r0:r0 + n] = x[:, start - j0 * P:start - j0 * P + n].swapaxes(0, 1)
            status |= 0 if have.all() else 1
    return k, v, status


def attend(cache, q, table, lengths, cu=None, window=0, scale=None):
    """(out, slack, status): slack bounds how far a kernel may be from out
    before its last rounding, from these of its roundings:
      p = exp(s - max) rounded to fp16, 2^-11 of itself or, below fp16's normal
        numbers, 2^-25 of the largest p times its value's scale;
      s in fp32: dim + 8 roundings of 2^-24 of the sum of |q k| (twice: in s
        and in the maximum), and 2^-22 for exp2;
      sums over n positions in fp32: n 2^-24 of the sum of magnitudes, above
        and below the fraction."""
    P, H, D = cache["k"].shape[2], cache["k"].shape[1], cache["k"].shape[3]
    rows, HQ = q.shape[:2]
    G = HQ // H
    scale = D ** -0.5 if scale is None else scale
    out, slack, status = np.zeros((rows, HQ, D)), np.zeros((rows, HQ, D)), 0
    for i, (r0, n, start, ok) in enumerate(spans(cu, lengths, rows, len(table[0]) * P)):
        if not ok:
            status |= 2
        if not ok or not n:
            continue
        j1 = -(-(start + n) // P)
        k, have = _gather(cache, table, i, 0, j1, "k")
        v, _ = _gather(cache, table, i, 0, j1, "v")
        t = np.arange(j1 * P)
        vs = np.zeros((H, j1 * P))
        for j in range(j1):
            p = _page(cache, table, i, j)
            if p is not None:
                vs[:, j * P:(j + 1) * P] = 2.0 ** (cache["scales"][p, :, 1].astype(np.float64) - 127)[:, None]
        for r in range(n):
            pos = start + r
            seen = (t <= pos) & ((t > pos - window) if window else True)
            status |= 0 if have[seen].all() else 1
            seen = seen & have
            if not seen.any():
                continue
            m = int(seen.sum())
            for h in range(HQ):
                qr, kk, vv = q[r0 + r, h].astype(np.float64), k[h // G, seen], v[h // G, seen]
                with np.errstate(invalid="ignore"):
                    s = scale * (kk @ qr)
                    big = scale * (np.abs(kk) @ np.abs(qr)).max()
                    p = np.exp(s - s.max())
                    out[r0 + r, h] = p @ vv / p.sum()
                    mean = p @ np.abs(vv) / p.sum()
                    err = 2.0 ** -11 + 2 * (D + 8) * 2.0 ** -24 * big + 2.0 ** -22 + 2 * m * 2.0 ** -24
                    floor = m * 2.0 ** -25 * (p * vs[h // G, seen]).max() / p.sum() * TOP[cache["codes"]]
                    slack[r0 + r, h] = 1.01 * (err * mean + floor)
    return out, slack, status
