"""Positions' weights and eviction from their definitions, in 64 bits on the
CPU with numpy.  A cache is cache_oracle's or cache4_oracle's dict."""
import numpy as np

import cache4_oracle as c4
import cache_oracle as co
from cache_oracle import _page, spans


def pages_of(c):
    return len(c["ke"]) if "ke" in c else len(c["scales"])


def page_at(c, table, i, j):
    return _page({"scales": c["ke"] if "ke" in c else c["scales"]}, table, i, j)


def attend(c, q, table, lengths, cu=None, window=0, scale=None):
    """c4.attend's answer for either kind of cache."""
    if "ke" in c:
        return c4.attend4(c, q, table, lengths, cu, window, scale)
    _, H, P, D = c["k"].shape

    def gather(i, length, which):
        x, have = co._gather(c, table, i, 0, -(-length // P), which)
        return x[:, :length], have[:length]

    def value_scales(i, length):
        out = np.zeros((H, -(-length // P) * P))
        for j in range(-(-length // P)):
            p = page_at(c, table, i, j)
            if p is not None:
                out[:, j * P:(j + 1) * P] = 2.0 ** (c["scales"][p, :, 1].astype(np.float64) - 127)[:, None]
        return out[:, :length]

    return c4.attend(gather, H, D, P, q, table, lengths, cu, window, scale, co.TOP[c["codes"]], value_scales)


def weigh(c, weights, shares, share_slack, table, lengths, cu, rows):
    """(weights after a call whose positions got `shares`, how far a kernel may be from them)."""
    P = weights.shape[2]
    out, slack = weights.astype(np.float64), np.zeros(weights.shape)
    for i, (_, n, start, ok) in enumerate(spans(cu, lengths, rows, len(table[0]) * P)):
        if not ok or not n:
            continue
        for t in range(start + n):
            p = page_at(c, table, i, t // P)
            if p is None:
                continue
            before = out[p, :, t % P] if t < start else 0.0
            out[p, :, t % P] = before + shares[i][:, t]
            slack[p, :, t % P] = share_slack[i][:, t] + 2.0 ** -24 * np.abs(out[p, :, t % P])
    return out, slack


def pick(w, keep, recent):
    """The positions that are kept of those of weights w [positions]."""
    n = len(w)
    if n <= keep:
        return list(range(n))
    key = [(-np.inf, 1) if np.isnan(x) else (x, 0) for x in w[:n - recent]]
    order = sorted(range(n - recent), key=lambda t: (key[t][1], -key[t][0], t))
    return sorted(order[:keep - recent]) + list(range(n - recent, n))


def evict(c, weights, table, lengths, to, keep, recent):
    """(cache, weights, lengths, positions, status) after the call."""
    c = {n: x.copy() if isinstance(x, np.ndarray) else x for n, x in c.items()}
    before = {n: x.copy() if isinstance(x, np.ndarray) else x for n, x in c.items()}
    old = weights.copy()
    weights = weights.copy()
    four = "ke" in c
    _, H, P, D = c["k"].shape
    new, positions, status = [], np.full((len(lengths), H, keep), -1, np.int32), 0
    for i, n in enumerate(lengths):
        if not 0 <= n <= len(table[i]) * P:
            status |= 2
            n = 0
        new.append(min(n, keep))
        for h in range(H):
            w = []
            for t in range(n):
                p = page_at(c, table, i, t // P)
                w.append(np.nan if p is None else old[p, h, t % P])
            kept = pick(np.array(w), keep, recent)
            positions[i, h, :len(kept)] = kept
            for j in range(-(-len(kept) // P)):
                part, d = kept[j * P:(j + 1) * P], page_at(c, to, i, j)
                if d is None:
                    status |= 1
                    continue
                sources = [page_at(c, table, i, t // P) for t in part]
                if any(s is None for s in sources):
                    status |= 1
                if not four:
                    top = [max([0] + [int(before["scales"][s, h, x]) for s in sources if s is not None]) for x in range(2)]
                    c["scales"][d, h] = top
                for slot, (t, s) in enumerate(zip(part, sources)):
                    weights[d, h, slot] = 0.0 if s is None else old[s, h, t % P]
                    if four:
                        for name, empty in (("k", 0), ("v", 0), ("ke", 27), ("ve", 27), ("drops", 0)):
                            c[name][d, h, slot] = empty if s is None else before[name][s, h, t % P]
                        continue
                    for x, name in enumerate("kv"):
                        code = np.zeros(D, np.uint8) if s is None else before[name][s, h, t % P]
                        if s is not None and before["scales"][s, h, x] < top[x]:
                            code = co.code(co.value(code, c["codes"]) * 2.0 ** (int(before["scales"][s, h, x]) - top[x]), c["codes"])
                        c[name][d, h, slot] = code
    return c, weights, new, positions, status
