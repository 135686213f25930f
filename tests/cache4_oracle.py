"""The cache of 4-bit codes from its definition, in 64 bits on the CPU with
numpy, token by token.  Shares no code with the library; spans of sequences are
cache_oracle's.

A cache here is a dict: k, v uint8 arrays [pages, heads, page, dim], one code
each, ke, ve uint8 [pages, heads, page] (2^(byte - 127)), drops uint8
[pages, heads, page, dim/32].
"""
import numpy as np

from cache_oracle import LOWEST, _page, spans

TOP, MOST_DROP = 6.0, 15
_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
DROP_BYTES = {64: 1, 96: 2, 128: 2, 192: 4, 256: 4}


def value(codes):
    x = _VALUES[codes & 7]
    return np.where(codes & 8, -x, x)


def code(x):
    """Nearest code, ties to the even one; infinities saturate; NaN is 0."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isnan(x), 0.0, np.minimum(np.abs(x), TOP))
    far = np.abs(a[..., None] - _VALUES)
    best = far.argmin(-1)  # the lower of two that are as near
    tie = (best < 7) & (np.take_along_axis(far, best[..., None], -1)[..., 0] ==
                        np.take_along_axis(far, np.minimum(best + 1, 7)[..., None], -1)[..., 0])
    c = np.where(tie & (best % 2 == 1), best + 1, best)
    return np.where(np.isnan(x), 0, c + 8 * np.signbit(x)).astype(np.uint8)


def exponent(x, lowest):
    """The least e >= lowest with max |x| <= 6 * 2^e over x's finite numbers."""
    a = np.abs(x[np.isfinite(x)])
    largest, e = a.max() if a.size else 0.0, lowest
    while largest > TOP * 2.0 ** e:
        e += 1
    return e


def to_stored(c):
    """(k_codes, v_codes, scales) as the library lays them out."""
    p, h, t, d = c["k"].shape
    k = c["k"].reshape(p, h, t // 16, 16, d // 32, 32).swapaxes(3, 4)
    v = c["v"].reshape(p, h, t // 16, 16, d).swapaxes(3, 4)
    nibbles = np.zeros((p, h, t, 2 * DROP_BYTES[d]), np.uint8)
    nibbles[..., :d // 32] = c["drops"]
    k, v, nibbles = (np.ascontiguousarray(x[..., 0::2] | x[..., 1::2] << 4) for x in (k, v, nibbles))
    return k, v, np.concatenate([c["ke"], c["ve"], nibbles.reshape(p, h, -1)], -1)


def from_stored(k, v, scales):
    def split(x):
        return np.stack([x & 15, x >> 4], -1).reshape(*x.shape[:-1], -1)

    k, v = split(k).swapaxes(3, 4), split(v).swapaxes(3, 4)
    p, h, b, _, d = v.shape
    t = b * 16
    return {"k": np.ascontiguousarray(k).reshape(p, h, t, d), "v": np.ascontiguousarray(v).reshape(p, h, t, d),
            "ke": scales[..., :t].copy(), "ve": scales[..., t:2 * t].copy(),
            "drops": split(scales[..., 2 * t:].reshape(p, h, t, -1))[..., :d // 32].copy()}


def numbers(c, p, which):
    """The values [heads, page, dim] of a page."""
    if which == "v":
        return value(c["v"][p]) * 2.0 ** (c["ve"][p].astype(np.float64) - 127)[..., None]
    e = c["ke"][p].astype(np.float64)[..., None] - 127 - c["drops"][p]
    return value(c["k"][p]) * np.repeat(2.0 ** e, 32, -1)


def write(cache, k, v, table, lengths, cu=None):
    """The cache after the call (a copy) and the status bits."""
    c = {n: x.copy() for n, x in cache.items()}
    P, status = c["k"].shape[2], 0
    for i, (r0, n, start, ok) in enumerate(spans(cu, lengths, len(k), len(table[0]) * P)):
        if not ok:
            status |= 2
            continue
        for r in range(n):
            p, t = _page({"scales": c["ke"]}, table, i, (start + r) // P), (start + r) % P
            if p is None:
                status |= 1
                continue
            for h in range(k.shape[1]):
                x, y = k[r0 + r, h].astype(np.float64), v[r0 + r, h].astype(np.float64)
                e = exponent(x, LOWEST)
                c["ke"][p, h, t] = e + 127
                for j in range(len(x) // 32):
                    b = x[32 * j:32 * j + 32]
                    d = MOST_DROP - (exponent(b, e - MOST_DROP) - (e - MOST_DROP))
                    c["drops"][p, h, t, j] = d
                    with np.errstate(invalid="ignore"):
                        c["k"][p, h, t, 32 * j:32 * j + 32] = code(b / 2.0 ** (e - d))
                e = exponent(y, LOWEST)
                c["ve"][p, h, t] = e + 127
                with np.errstate(invalid="ignore"):
                    c["v"][p, h, t] = code(y / 2.0 ** e)
    return c, status


def _gather(c, table, i, length, which):
    """Values [H, length, D] of a sequence and whether each position has a page."""
    P = c["k"].shape[2]
    H, D = c["k"].shape[1], c["k"].shape[3]
    n = -(-length // P)
    out, have = np.zeros((H, n * P, D)), np.zeros(n * P, bool)
    for j in range(n):
        p = _page({"scales": c["ke"]}, table, i, j)
        if p is not None:
            out[:, j * P:(j + 1) * P] = numbers(c, p, which)
            have[j * P:(j + 1) * P] = True
    return out[:, :length], have[:length]


def read(c, table, lengths, cu, rows):
    P, H, D = c["k"].shape[2], c["k"].shape[1], c["k"].shape[3]
    k, v, status = np.zeros((rows, H, D)), np.zeros((rows, H, D)), 0
    for i, (r0, n, start, ok) in enumerate(spans(cu, lengths, rows, len(table[0]) * P)):
        if not ok:
            status |= 2
        if not ok or not n:
            continue
        for which, out in (("k", k), ("v", v)):
            x, have = _gather(c, table, i, start + n, which)
            out[r0:r0 + n] = x[:, start:].swapaxes(0, 1)
            status |= 0 if have[start:].all() else 1
    return k, v, status


def attend(gather, heads, dim, page, q, table, lengths, cu=None, window=0, scale=None, top=TOP, value_scales=None,
           query_error=0.0):
    """(out, slack, shares, share_slack, status) of attention over positions
    that gather(i, length, which) gives.  shares: a list with, for each
    sequence, the weights [heads, length] its positions got, and how far a
    kernel may be from them.  slack bounds how far a kernel may be from out
    before its last rounding, from these of its roundings:
      p = exp(s - max) rounded to fp16, 2^-11 of itself or, below fp16's normal
        numbers, 2^-25 of the largest p times its value's scale
        (value_scales(i, length), [heads, length]);
      s in fp32: dim + 8 roundings of 2^-24 of the sum of |q k| (twice: in s
        and in the maximum), two more of 2^-24 of |s| and the value's exponent
        with it, and 2^-22 for exp2;
      sums over n positions in fp32: n 2^-24 of the sum of magnitudes, above
        and below the fraction;
      query_error of the row's largest number, of every number of a query.
    A share has the errors of s and of the sum below its fraction, its own
    sum's over the rows, and for each row and query head 2^-126: below that, fp32's
    smallest normal number, the result of exp2 is 0."""
    rows, HQ = q.shape[:2]
    G = HQ // heads
    scale = dim ** -0.5 if scale is None else scale
    out, slack, status = np.zeros((rows, HQ, dim)), np.zeros((rows, HQ, dim)), 0
    shares, share_slack = [], []
    for i, (r0, n, start, ok) in enumerate(spans(cu, lengths, rows, len(table[0]) * page)):
        if not ok:
            status |= 2
        length = start + n if ok else 0
        got, off = np.zeros((heads, length)), np.zeros((heads, length))
        shares.append(got)
        share_slack.append(off)
        if not ok or not n:
            continue
        k, have = gather(i, length, "k")
        v, _ = gather(i, length, "v")
        vs, t = value_scales(i, length), np.arange(length)
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
                    share = p / p.sum()
                    out[r0 + r, h] = share @ vv
                    mean = share @ np.abs(vv)
                    lost = scale * query_error * np.abs(qr).max() * np.abs(kk).sum(-1).max()
                    exp_err = 2 * lost + 2 * (dim + 8) * 2.0 ** -24 * big + 8 * 2.0 ** -24 * (np.abs(s).max() + 300) + 2.0 ** -22
                    err = 2.0 ** -11 + exp_err + 2 * m * 2.0 ** -24
                    floor = m * 2.0 ** -25 * (share * vs[h // G, seen]).max() * top
                    slack[r0 + r, h] = 1.01 * (err * mean + floor)
                    got[h // G, seen] += share
                    off[h // G, seen] += 1.01 * share * (2 * exp_err + 2 * m * 2.0 ** -24)
        off += got * (n * G + 2) * 2.0 ** -24 + n * G * 2.0 ** -126
    return out, slack, shares, share_slack, status


def attend4(c, q, table, lengths, cu=None, window=0, scale=None, query_error=0.0):
    _, H, P, D = c["k"].shape

    def scales(i, length):
        out = np.zeros((H, -(-length // P) * P))
        for j in range(-(-length // P)):
            p = _page({"scales": c["ke"]}, table, i, j)
            if p is not None:
                out[:, j * P:(j + 1) * P] = 2.0 ** (c["ve"][p].astype(np.float64) - 127)
        return out[:, :length]

    return attend(lambda i, length, which: _gather(c, table, i, length, which), H, D, P, q, table, lengths, cu, window,
                  scale, TOP, scales, query_error)
