"""Calls of the key/value cache with rows of odd strides: single rows of wider
buffers, and one key head, against the oracle."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from gpu_util import banner
from test_gpu_cache import BF, FP, Setup, close, ltc, same_cache  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,dtype", [(2, BF), (1, FP)])
@pytest.mark.parametrize("rows", [1, 3])
def test_odd_widths(ltc, heads, dtype, rows):  # noqa: F811
    banner(f"{rows} rows of a product of odd width, {heads} heads")
    s = Setup(ltc, 81, heads, 64, 16, "e4m3", dtype, [1] * rows, [20 + i for i in range(rows)], single=True)
    D, group = 64, 3
    fused = torch.from_numpy(s.rng.normal(0, 1, (rows + 2, heads * (group + 2) * D + 3))).to(dtype).cuda()[1:1 + rows]
    q, k, v = (fused[:, a * heads * D:b * heads * D].unflatten(1, (-1, D)) for a, b in ((0, group), (group, group + 1), (group + 1, group + 2)))
    if heads == 1:  # and a head stride that is no multiple of anything
        k, v = (torch.as_strided(x, x.shape, (x.stride(0), 13, 1), x.storage_offset()) for x in (k, v))
    ltc.cache_write(s.cache, k, v, s.gtable, s.glengths)
    s.o, _ = co.write(s.o, k.double().cpu().numpy(), v.double().cpu().numpy(), s.table, s.lengths)
    same_cache(s, s.o)
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths)
    want, slack, _ = co.attend(s.o, q.double().cpu().numpy(), s.table, s.lengths)
    close(out, want, slack, dtype)
    assert np.isfinite(want).all()
    s.cache.check()
