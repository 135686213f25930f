"""Eviction by one workgroup a sequence and head from more positions than it
counts at a time (65,536): random weights, and ties on both sides of that."""
import numpy as np
import pytest
import torch

from gpu_util import banner
from test_gpu_cache_evict import FP, _few_hundreds, _ties, check, prepared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def _ones(rng, shape):
    return np.ones(shape, np.float32)


# of four weights as many positions each: 40,000 are those of two, and the first ones of a third; 55,000 reach past
# position 65,536 for the last of them
@pytest.mark.parametrize("weights,keep,recent", [(None, 40000, 100), (_few_hundreds, 55000, 0), (_ties, 40000, 100), (_ties, 55000, 64),
                                                 (_ones, 70000, 100), (_ones, 65536, 0), (_ones, 65637, 100)])
def test_more_positions_than_are_counted_at_a_time(ltc, weights, keep, recent):
    banner(f"evict 75,001 positions to {keep}")
    lengths = [1 + (i * 37) % 250 for i in range(66)]
    lengths[40] = 75001
    # pages for what is kept of the long one are those of a sequence that the call does not name; the others come to
    # the first of their targets alone
    pages = -(-keep // 256)
    s = prepared(ltc, 121, 1, 64, 256, "int8", FP, lengths + [pages * 256], 1, weights)
    to = np.full((66, pages), -1, np.int32)
    to[:, 0] = s.to[:66, 0]
    to[40] = s.table[66, :pages]
    s.table, s.lengths, s.rows, s.to = s.table[:66], lengths, 66, to
    s.gtable, s.glengths = s.gtable[:66], s.glengths[:66]
    check(ltc, s, keep, recent)
