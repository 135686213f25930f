"""The cases that the operators on the 8-bit key/value cache are measured by.

Three operators (`op` of a case):
  write   quantises new keys and values into the pages of a cache
  read    reads cached positions back as 16-bit rows
  attend  attention of new queries over the cached positions

The cache is pages of `page` tokens with one power-of-two scale for each page,
head and kind (key, value):
  k_codes u8 [pages, heads, page/16, dim/16, 16 tokens, 16 dims]
  v_codes u8 [pages, heads, page/16, dim, 16 tokens]
  scales  u8 [pages, heads, 2], a scale is 2^(byte - 127)
Rows cu[i]..cu[i+1] of a call belong to sequence i and stand for its last
positions, lengths[i] - (cu[i+1] - cu[i]) to lengths[i] - 1; its position t is
token t % page of page table[i, t / page].
"""
import random

import torch

own = False

LOWEST = -100  # of a scale's exponent
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, codes, dtype, heads, dim, page, seqs, new, past, q_heads=0, window=0, shape=0):
    """`new` and `past`: "low-high", the rows of a sequence and the positions before them."""
    c = {"op": op, "codes": codes, "dtype": dtype, "heads": heads, "dim": dim, "page": page, "seqs": seqs, "new": new,
         "past": past, "q_heads": q_heads, "window": window, "shape": shape}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a decoding step of 48 sequences writes one token each: latency
        _case("write one token", "write", "e4m3", "bf16", 8, 128, 64, 48, "1-1", "100-1500"),
        # three prompts are written at once, the second half of a long one among them
        _case("write prompts", "write", "e4m3", "bf16", 8, 128, 64, 3, "3000-8200", "0-900", shape=1),
        # pieces of many ragged prompts, small heads, small pages, whole-number codes
        _case("write pieces int8 fp16", "write", "int8", "fp16", 5, 64, 16, 37, "1-190", "0-333", shape=2),
        # one long sequence read back whole, to run a layer on it in 16 bits
        _case("read long", "read", "e4m3", "bf16", 8, 128, 64, 1, "65537-65537", "0-0"),
        # spans of ragged sequences read back
        _case("read spans int8 fp16", "read", "int8", "fp16", 4, 96, 32, 19, "20-501", "0-700", shape=3),
        # one user decodes, short context: latency
        _case("attend one short", "attend", "e4m3", "bf16", 8, 128, 64, 1, "1-1", "776-776", q_heads=32),
        # a serving batch decodes
        _case("attend batch", "attend", "e4m3", "bf16", 8, 128, 64, 64, "1-1", "1000-6000", q_heads=32, shape=4),
        # one user decodes at the end of a very long context: split over the sequence
        _case("attend one long", "attend", "e4m3", "bf16", 8, 128, 64, 1, "1-1", "131070-131070", q_heads=32),
        # a batch of a model with as many key heads as query heads and a sliding window
        _case("attend window int8 fp16", "attend", "int8", "fp16", 12, 64, 32, 23, "1-1", "0-5000", q_heads=12, window=1024,
              shape=5),
        # five drafted tokens a sequence are checked at once
        _case("attend drafts", "attend", "int8", "bf16", 4, 128, 16, 16, "5-5", "300-4001", q_heads=28, shape=6),
        # two prompts are read in, one of them the second piece of a long one
        _case("attend prompts", "attend", "e4m3", "bf16", 8, 128, 64, 2, "2500-4096", "0-4096", q_heads=32, shape=7),
        # short ragged prompts of a model with large heads
        _case("attend pieces int8 fp16", "attend", "int8", "fp16", 2, 256, 64, 9, "33-517", "0-300", q_heads=10, shape=8),
    ]


def draw(rng):
    def spread(low, high):
        return int(round(low * (high / low) ** rng.random()))

    op = rng.choice(["write", "read", "attend", "attend"])
    heads, dim, page = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), rng.choice([64, 96, 128, 192, 256]), rng.choice([16, 32, 64, 128])
    width = heads * dim
    group, window, past_low = 0, 0, 0
    if op == "attend":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        while heads * group > 64:
            group //= 2
        window = rng.choice([0, 0, 0, spread(16, 4096)])
        kind = rng.choice(["one", "one", "few", "many"])
        if kind == "many":  # at most a quarter of the largest listed case's products
            past = spread(1, 4096)
            new = max(9, min(spread(16, 3000), int(2e7 / ((past + 2000) * group * width / 4096))))
            seqs = rng.choice([1, 2, 3])
        else:
            new = 1 if kind == "one" else rng.randint(2, 8)
            past = spread(1, 100000)
            seqs = max(1, min(spread(1, 80), int(1.5e8 / (past * width))))
        new_low = max(1, new // 3) if kind == "many" else new
    elif op == "read":
        past, seqs = spread(1, 3000), spread(1, 40)
        new = max(1, min(spread(1, 30000), int(4e7 / (width * seqs))))
        new_low = max(1, new // 4)
    else:
        past, seqs = spread(1, 3000), spread(1, 100)
        new = rng.choice([1, max(1, min(spread(2, 10000), int(1.5e7 / (width * seqs))))])
        new_low = max(1, new // 4)
    return _case(None, op, rng.choice(["e4m3", "int8"]), rng.choice(["bf16", "fp16"]), heads, dim, page, seqs, "%d-%d" % (new_low, new),
                 "%d-%d" % (past_low, past), heads * group, window, rng.randint(1, 1 << 20))


def _lengths(case):
    """(new rows, length) of each sequence: part of the case, the same for each seed.  The first sequence has the most of both."""
    r = random.Random(case["shape"])
    (nl, nh), (pl, ph) = (map(int, case[k].split("-")) for k in ("new", "past"))
    new = [nh] + [r.randint(nl, nh) for _ in range(case["seqs"] - 1)]
    past = [ph] + [r.randint(pl, ph) for _ in range(case["seqs"] - 1)]
    return new, [a + b for a, b in zip(new, past)]


def _power(e):
    """2^e as float32, exactly, for whole numbers e in -126..127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _round(x, codes):
    """The codes (uint8) of float32 values that are in the codes' range."""
    if codes == "int8":
        return torch.round(x).to(torch.int8).view(torch.uint8)
    e = torch.where(x == 0, -6, torch.frexp(x).exponent - 1).clamp(min=-6)
    n = torch.round(x.abs() * _power(3 - e)).to(torch.int32) + 8 * (e + 6)
    return (n + 128 * torch.signbit(x)).to(torch.uint8)


def _value(c, codes):
    """The float32 values of codes."""
    if codes == "int8":
        return c.view(torch.int8).float()
    c = c.to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).float()
    x = torch.where(e > 0, (m + 8) * _power(e - 10), m * 2.0 ** -9)
    return torch.where(c >= 128, -x, x)


def _typed(c, codes):
    """Codes as the numbers they stand for (a view)."""
    return c.view(torch.float8_e4m3fn if codes == "e4m3" else torch.int8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, total = _lengths(case)
    B, H, D, PT, codes = case["seqs"], case["heads"], case["dim"], case["page"], case["codes"]
    T, widest = sum(new), -(-max(total) // PT)
    need = [-(-n // PT) for n in total]
    n_pages = sum(need) + 3
    dtype = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def held(*shape):  # codes of normal values that fill their range
        x = normal(*shape)
        x *= 110.0 if codes == "e4m3" else 30.0
        top = 448.0 if codes == "e4m3" else 127.0
        return _round(x.clamp_(-top, top), codes)

    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    at = torch.cumsum(torch.tensor([0] + need), 0)[:-1].cuda()[:, None] + torch.arange(widest, device="cuda")
    table = order[at.clamp(max=n_pages - 1)].contiguous()  # what is past a sequence's end is not looked at
    s = {"op": case["op"], "codes": codes, "dim": D, "page": PT, "rows": T, "most_new": max(new), "widest": widest, "window": case["window"],
         "dtype": dtype, "table": table, "lengths": torch.tensor(total, dtype=torch.int32, device="cuda"),
         "cu": torch.cumsum(torch.tensor([0] + new), 0).to(torch.int32).cuda(), "single": max(new) == 1 and min(new) == 1,
         "k_codes": held(n_pages, H, PT // 16, D // 16, 16, 16), "v_codes": held(n_pages, H, PT // 16, D, 16)}
    middle = -7 if codes == "e4m3" else -5
    s["scales"] = (torch.randint(middle - 1, middle + 2, (n_pages, H, 2), generator=g, device="cuda") + 127).to(torch.uint8)
    if case["op"] == "write":
        s["k"] = (normal(T, H, D) * torch.exp(0.5 * normal(1, H, D))).to(dtype)  # some channels of keys are larger than others
        s["v"] = normal(T, H, D).to(dtype)
    elif case["op"] == "attend":
        s["q"] = (2.0 * normal(T, case["q_heads"], D)).to(dtype)
    if own:  # the handle a program keeps; the tensors are the same ones
        import lossless_tensor_compression_amd as ltc
        s["ltc"] = ltc
        s["cache"] = ltc.KVCache.of(s["k_codes"], s["v_codes"], s["scales"], dtype=dtype, codes=codes)
    return s


def run(s):
    if own:
        ltc, cu = s["ltc"], None if s["single"] else s["cu"]
        if s["op"] == "write":
            ltc.cache_write(s["cache"], s["k"], s["v"], s["table"], s["lengths"], cu)
            return _held(s)
        if s["op"] == "read":
            return ltc.cache_read(s["cache"], s["table"], s["lengths"], cu, rows=s["rows"])
        return ltc.cache_attend(s["cache"], s["q"], s["table"], s["lengths"], cu, window=s["window"])
    return {"write": _write, "read": _read, "attend": _attend}[s["op"]](s)


def _held(s):
    return {"k": _typed(s["k_codes"], s["codes"]), "v": _typed(s["v_codes"], s["codes"]), "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _write(s):
    """All pages that new tokens fall on, padded to the most that one sequence has (its last page again and again)."""
    PT, D, codes = s["page"], s["dim"], s["codes"]
    cu, end = s["cu"].long(), s["lengths"].long()
    new = cu[1:] - cu[:-1]
    start = end - new
    most = (s["most_new"] + PT - 2) // PT + 1
    j = torch.minimum((start // PT)[:, None] + torch.arange(most, device=cu.device), ((end - 1) // PT)[:, None])
    page = torch.gather(s["table"].long(), 1, j)
    pos = j[:, :, None] * PT + torch.arange(PT, device=cu.device)
    fresh = (pos >= start[:, None, None]) & (pos < end[:, None, None])
    kept = pos < start[:, None, None]
    row = (pos - start[:, None, None] + cu[:-1, None, None]).clamp(0, s["rows"] - 1)
    begun = kept.any(-1)
    for kind, name in enumerate(("k", "v")):
        x = s[name].float()[row].movedim(3, 2)  # [B, pages, H, PT, D]
        wide = fresh[:, :, None, :, None]
        largest = torch.where(wide, x.abs(), 0.0).amax((3, 4))
        m, e = torch.frexp(largest)
        e = torch.where(m <= 0.875, e - 9, e - 8) if codes == "e4m3" else torch.where(m <= 127 / 128, e - 7, e - 6)
        e = torch.where(largest > 0, e, LOWEST).clamp(min=LOWEST)
        before = s["scales"][page][..., kind].int() - 127
        after = torch.where(begun[:, :, None], torch.maximum(before, e), e)
        store = s[name + "_codes"]
        old = _by_token(store[page], kind, PT, D)
        shrink = _power((before - after).clamp(-126, 0))[..., None, None]
        again = torch.where((after > before)[..., None, None], _round(_value(old, codes) * shrink, codes), old)
        top = 448.0 if codes == "e4m3" else 127.0
        coded = _round((x * _power(-after)[..., None, None]).clamp(-top, top), codes)
        now = torch.where(wide, coded, torch.where(kept[:, :, None, :, None], again, old))
        store[page] = _by_store(now, kind, PT, D)
        s["scales"][page, :, kind] = (after + 127).to(torch.uint8)
    return _held(s)


def _by_token(c, kind, PT, D):
    """[..., PT, D] of the codes of pages as they are stored."""
    if kind == 0:  # [..., PT/16, D/16, 16 tokens, 16 dims]
        return c.transpose(-3, -2).reshape(*c.shape[:-4], PT, D)
    return c.transpose(-2, -1).reshape(*c.shape[:-3], PT, D)


def _by_store(c, kind, PT, D):
    if kind == 0:
        return c.reshape(*c.shape[:-2], PT // 16, 16, D // 16, 16).transpose(-3, -2)
    return c.reshape(*c.shape[:-2], PT // 16, 16, D).transpose(-2, -1)


def _read(s):
    PT, cu, end = s["page"], s["cu"].long(), s["lengths"].long()
    n = cu[1:] - cu[:-1]
    i = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=s["rows"])
    pos = torch.arange(s["rows"], device=n.device) - cu[i] + (end - n)[i]
    page, off = s["table"].long()[i, pos // PT], pos % PT
    scale = _power(s["scales"][page].int() - 127)  # [T, H, 2]
    k = s["k_codes"][page, :, off // 16, :, off % 16].flatten(-2)
    v = s["v_codes"][page, :, off // 16, :, off % 16]
    return ((_value(k, s["codes"]) * scale[:, :, :1]).to(s["dtype"]), (_value(v, s["codes"]) * scale[:, :, 1:]).to(s["dtype"]))


def _attend(s):
    """Every sequence padded to the longest, its rows to the most rows."""
    PT, D, q = s["page"], s["dim"], s["q"]
    H, cu, end = s["k_codes"].shape[1], s["cu"].long(), s["lengths"].long()
    B, N, G = end.numel(), s["most_new"], q.shape[1] // H
    table = s["table"].long()
    scale = _power(s["scales"][table].int() - 127)  # [B, P, H, 2]

    def rows(codes, kind):  # [B, H, L, D]
        x = _value(_by_token(codes[table], kind, PT, D), s["codes"]) * scale[..., kind, None, None]
        return x.transpose(1, 2).reshape(B, H, -1, D)

    n = cu[1:] - cu[:-1]
    at = torch.arange(N, device=q.device)
    row = (cu[:-1, None] + at).clamp(max=s["rows"] - 1)  # [B, N]
    pos = (end - n)[:, None] + at
    t = torch.arange(table.shape[1] * PT, device=q.device)
    seen = t <= pos[..., None]  # [B, N, L]
    if s["window"]:
        seen &= t > pos[..., None] - s["window"]
    seen &= t < end[:, None, None]
    x = q.float()[row].reshape(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    p = torch.matmul(x, rows(s["k_codes"], 0).transpose(-1, -2)) * D ** -0.5
    p = p.view(B, H, G, N, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = rows(s["v_codes"], 1)
    v = torch.where((t < end[:, None])[:, None, :, None], v, 0.0)
    out = torch.matmul(p.view(B, H, G * N, -1), v)
    out = out.view(B, H, G, N, D).permute(0, 3, 1, 2, 4).reshape(B * N, H * G, D)
    i = torch.repeat_interleave(torch.arange(B, device=q.device), n, output_size=s["rows"])
    return out[i * N + torch.arange(s["rows"], device=q.device) - cu[i]].to(s["dtype"])


def work(case):
    new, total = _lengths(case)
    H, D, PT, T = case["heads"], case["dim"], case["page"], sum(new)
    codes, wide = 2 * H * D, 4 * H * D  # bytes of a token's codes, and of its keys and values in 16 bits
    pages = sum(-(-n // PT) for n in total)
    if case["op"] == "write":
        touched = sum((n - 1) // PT - (n - m) // PT + 1 for m, n in zip(new, total))
        return {"bytes": T * (codes + wide) + 2 * 2 * H * touched, "flops": 4 * T * H * D}
    if case["op"] == "read":
        touched = sum((n - 1) // PT - (n - m) // PT + 1 for m, n in zip(new, total))
        return {"bytes": T * (codes + wide) + 2 * H * touched, "flops": 2 * T * H * D}
    w = case["window"]
    pairs, looked = 0, 0
    for m, n in zip(new, total):
        pairs += sum(min(p + 1, w) if w else p + 1 for p in range(n - m, n))
        looked += min(n, w + m - 1) if w else n
    return {"bytes": looked * codes + 2 * H * pages + 2 * 2 * T * case["q_heads"] * D, "flops": 4 * D * case["q_heads"] * pairs}


def exact(case, seed):
    """In 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    new, total = _lengths(case)
    H, D, PT = case["heads"], case["dim"], case["page"]
    float8 = case["codes"] == "e4m3"
    kinds = torch.float8_e4m3fn if float8 else torch.int8
    table = s["table"].tolist()

    def tokens(x, kind):  # [pages, H, PT, D] of stored codes
        x = x.view(kinds).double()
        return (x.permute(0, 1, 2, 4, 3, 5) if kind == 0 else x.permute(0, 1, 2, 4, 3)).reshape(-1, H, PT, D)

    if case["op"] == "write":
        result = {"scales": s["scales"].view(torch.float8_e8m0fnu).double()}
        for kind, name in enumerate("kv"):
            held, source, first = tokens(s[name + "_codes"], kind), s[name].double(), 0
            for b in range(case["seqs"]):
                at = total[b] - new[b]
                while at < total[b]:
                    page, o, end = table[b][at // PT], at % PT, min(total[b], at - at % PT + PT)
                    x = source[first:first + end - at].transpose(0, 1)  # [H, n, D]
                    top = 448.0 if float8 else 127.0
                    size = x.abs().amax((1, 2)).cpu()
                    scale = torch.tensor([next(2.0 ** e for e in range(LOWEST, 128) if a <= top * 2.0 ** e) for a in size.tolist()],
                                         dtype=torch.float64, device="cuda")
                    if o:
                        before = result["scales"][page, :, kind]
                        scale = torch.maximum(scale, before)
                        again = held[page, :, :o] * (before / scale)[:, None, None]
                        held[page, :, :o] = again.float().to(kinds).double() if float8 else again.round()
                    x = x / scale[:, None, None]
                    held[page, :, o:o + end - at] = x.float().to(kinds).double() if float8 else x.round()
                    result["scales"][page, :, kind] = scale
                    first, at = first + end - at, end
            x = held.reshape(-1, H, PT // 16, 16, D)
            result[name] = (x.reshape(-1, H, PT // 16, 16, D // 16, 16).transpose(3, 4) if kind == 0 else x.transpose(3, 4)).contiguous()
        return result
    scale = torch.exp2(s["scales"].double() - 127)
    values = [tokens(s[name + "_codes"], kind) * scale[:, :, kind, None, None] for kind, name in enumerate("kv")]
    outs, first = [], 0
    for b in range(case["seqs"]):
        pages = torch.tensor(table[b][:-(-total[b] // PT)], device="cuda")
        k, v = (x[pages].transpose(0, 1).reshape(H, -1, D)[:, :total[b]] for x in values)  # [H, L, D]
        if case["op"] == "read":
            outs.append([x[:, total[b] - new[b]:].transpose(0, 1) for x in (k, v)])
            continue
        q = s["q"][first:first + new[b]].double()
        first += new[b]
        p = torch.arange(total[b] - new[b], total[b], device="cuda")[:, None]
        t = torch.arange(total[b], device="cuda")
        hidden = (t > p) | (t <= p - (case["window"] or 1 << 30))
        group = case["q_heads"] // H
        one = [torch.softmax((q[:, h] @ k[h // group].T / D ** 0.5).masked_fill(hidden, -float("inf")), -1) @ v[h // group] for h in range(case["q_heads"])]
        outs.append(torch.stack(one, 1))
    return tuple(torch.cat(x) for x in zip(*outs)) if case["op"] == "read" else torch.cat(outs)
