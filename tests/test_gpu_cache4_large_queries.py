"""bf16 queries at the end of what calls over 4-bit codes take, 2^107: the
products' sums stay within fp32's numbers, with and without weights."""
import numpy as np
import pytest
import torch

import cache4_oracle as c4
import evict_oracle as eo
from cache4_setup import Setup4, close
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("dim,heads,group,new,past", [(256, 1, 2, [1, 3], [200, 70]), (128, 2, 4, [40, 3], [30, 100]),
                                                      (64, 2, 12, [30, 40], [70, 5]), (256, 1, 40, [9], [60]),
                                                      (128, 8, 16, [9 + i % 3 for i in range(32)], [20 + i for i in range(32)])])
def test_sums_stay_finite(ltc, dim, heads, group, new, past):
    """Numbers of one sign, so that nothing cancels, against keys of large codes at the lowest scale."""
    banner(f"queries of 2^107, dim {dim}")
    s = Setup4(ltc, 151, heads, dim, 16, BF, new, past)
    s.o["k"][:] = s.rng.integers(5, 8, s.o["k"].shape)
    s.o["ke"][:], s.o["drops"][:] = 27, 0
    s.upload(ltc)
    q = torch.from_numpy(s.rng.uniform(1.5, 1.99, (s.rows, heads * group, dim)) * 2.0 ** 106).to(BF).cuda()
    scale = 2.0 ** -6 / dim  # scores of about 5, which differ by the codes
    w = s.cache.no_weights()
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, scale=scale, weights=w)
    some = np.concatenate([h * group + np.arange(min(group, 2)) for h in range(heads)])
    full = len(some) == heads * group or s.rows * heads * group < 3000
    q64 = q.double().cpu().numpy()
    if not full:
        want, slack, _, _, status = c4.attend4(s.o, q64[:, some], s.table, s.lengths, s.cu, 0, scale)
        close(out[:, torch.from_numpy(some).cuda()], want, slack, BF)
        assert torch.isfinite(out).all() and torch.isfinite(w).all()
    else:
        want, slack, shares, off, status = c4.attend4(s.o, q64, s.table, s.lengths, s.cu, 0, scale)
        close(out, want, slack, BF)
        want_w, slack_w = eo.weigh(s.o, np.zeros(tuple(w.shape)), shares, off, s.table, s.lengths, s.cu, s.rows)
        assert (np.abs(w.double().cpu().numpy() - want_w) <= slack_w).all()
    assert np.abs(want).max() > 0 and int(s.cache.status.item()) == status == 0
