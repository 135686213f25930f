"""Caches of 4-bit codes for the GPU tests: the same on both sides, sequences
with shuffled pages."""
import numpy as np
import torch

import cache4_oracle as c4
from test_gpu_cache import close  # noqa: F401  (got within slack and half a step of want)


class Setup4:
    codes = "e2m1"

    def __init__(self, ltc, seed, heads, dim, page, dtype, new, past, spread=1, single=False, spare=2, most_drop=3):
        rng = self.rng = np.random.default_rng(seed)
        self.dtype, self.H, self.D, self.P = dtype, heads, dim, page
        self.lengths = [a + b for a, b in zip(new, past)]
        self.cu = None if single else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = sum(new)
        need = [-(-n // page) for n in self.lengths]
        self.pages = pages = sum(need) + spare
        width = max(need + [1]) + 1
        self.order = order = rng.permutation(pages)
        self.table = rng.integers(-5, pages + 5, (len(new), width)).astype(np.int32)  # behind the end: anything
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.free = order[at:]  # pages of no sequence
        shape = (pages, heads, page)
        self.o = {"k": c4.code(np.clip(rng.normal(0, 2, (*shape, dim)), -6, 6)),
                  "v": c4.code(np.clip(rng.normal(0, 2, (*shape, dim)), -6, 6)),
                  "ke": rng.integers(126 - spread, 127 + spread, shape).astype(np.uint8),
                  "ve": rng.integers(126 - spread, 127 + spread, shape).astype(np.uint8),
                  "drops": rng.integers(0, most_drop + 1, (*shape, dim // 32)).astype(np.uint8)}
        for i, n in enumerate(self.lengths):  # whatever is behind a sequence's end does not count
            if n % page:
                for name in ("ke", "ve"):
                    self.o[name][self.table[i, n // page], :, n % page:] = 255
        self.upload(ltc)

    def upload(self, ltc):
        k, v, scales = (torch.from_numpy(x).cuda() for x in c4.to_stored(self.o))
        self.cache = ltc.KVCache.of(k, v, scales, dtype=self.dtype, codes="e2m1")
        self.gtable = torch.from_numpy(self.table).cuda()
        self.glengths = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.gcu = None if self.cu is None else torch.from_numpy(self.cu).cuda()

    def rows16(self, heads, size=1.0):
        x = torch.from_numpy(self.rng.normal(0, size, (self.rows, heads, self.D))).to(self.dtype)
        return x.cuda(), x.double().numpy()

    def got(self):
        return c4.from_stored(*(x.cpu().numpy() for x in (self.cache.k_codes, self.cache.v_codes, self.cache.scales)))

    def same(self, want):
        got = self.got()
        for name, x in want.items():
            assert np.array_equal(got[name], x), (name, np.argwhere(got[name] != x)[:5])


def check_attend4(ltc, s, q_heads, window=0, scale=None, size=2.0):
    q, q64 = s.rows16(q_heads, size)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, window=window, scale=scale)
    want, slack, _, _, status = c4.attend4(s.o, q64, s.table, s.lengths, s.cu, window, scale)
    close(out, want, slack, s.dtype)
    assert int(s.cache.status.item()) == status == 0
