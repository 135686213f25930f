"""Positions without a page that eviction keeps: they become zeros, and what
reads them afterwards is attention over zeros."""
import numpy as np
import pytest
import torch

import evict_oracle as eo
from cache4_setup import close
from gpu_util import banner
from test_gpu_cache_evict import BF, FP, prepared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("codes,dtype,dim,page", [("int8", FP, 64, 64), ("e4m3", BF, 128, 128), ("int8", BF, 64, 16), ("e2m1", BF, 64, 64)])
@pytest.mark.parametrize("rows", [1, 3])
def test_pages_of_zeros_are_attended_to(ltc, codes, dtype, dim, page, rows):
    """Whole pages of zeros in front of the others, as many as a step of the
    attention takes: their weights are those of scores of 0."""
    banner(f"pages of zeros, {codes}, {dim} dims, pages of {page}")
    n = 6 * 64
    s = prepared(ltc, 81, 2, dim, page, codes, dtype, [n, n], n)
    lost = max(64 // page, 1)
    s.table[0, :lost] = -1
    s.gtable = torch.from_numpy(s.table).cuda()
    w, to = torch.from_numpy(s.w.copy()).cuda(), torch.from_numpy(s.to).cuda()
    new, _ = ltc.cache_evict(s.cache, w, s.gtable, s.glengths, to, n)
    assert new.tolist() == [n, n]
    s.o, _, _, _, status = eo.evict(s.o, s.w, s.table, s.lengths, s.to, n, 0)
    assert int(s.cache.status.item()) == status == 1
    s.cache.status.zero_()
    s.rows, cu = 2 * rows, np.array([0, rows, 2 * rows], np.int32)
    q, q64 = s.rows16(4, 0.2)
    weights, before = s.cache.no_weights(), np.zeros(s.w.shape)
    out = ltc.cache_attend(s.cache, q, to, new, torch.from_numpy(cu).cuda(), weights=weights)
    want, slack, shares, off, status = eo.attend(s.o, q64, s.to, [n, n], cu)
    assert status == 0 and np.abs(want[0]).max() > 0
    close(out, want, slack, dtype)
    want_w, slack_w = eo.weigh(s.o, before, shares, off, s.to, [n, n], cu, 2 * rows)
    assert (np.abs(weights.double().cpu().numpy() - want_w) <= slack_w).all()
    s.cache.check()
