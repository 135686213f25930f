"""Queries with one number that is larger than all others by far and meets keys
of zero, in calls of many rows over 4-bit codes: the others make the scores, and
keep their bits."""
import numpy as np
import pytest
import torch

import cache4_oracle as c4
from cache4_setup import Setup4, close
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# heads, query heads of each, new rows: enough for the kernel whose waves share positions
MANY = {128: (8, 16, [5 + i % 9 for i in range(32)]), 256: (8, 16, [5 + i % 9 for i in range(16)])}


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def far_rows(ltc, dim, seed):
    heads, group, new = MANY[dim]
    s = Setup4(ltc, seed, heads, dim, 32, BF, new, [20 + 3 * i for i in range(len(new))])
    s.o["k"][..., 7] = 0
    s.upload(ltc)
    return s, heads * group


@pytest.mark.parametrize("dim,far,weights", [(128, 10, False), (128, 20, False), (128, 20, True), (128, 40, False), (256, 14, False),
                                             (256, 20, False)])
def test_small_numbers_keep_their_bits(ltc, dim, far, weights):
    """Some heads of some rows have such a number, 2^far; 2^-14 of the largest of
    eight numbers is what they may lose, 2^-16 of them being left out and the largest
    of another eight perhaps four times smaller."""
    banner(f"far queries, {dim} dims, 2^{far}, weights {weights}")
    s, q_heads = far_rows(ltc, dim, 92)
    q, q64 = s.rows16(q_heads, 1.0)
    which = torch.from_numpy(s.rng.random((s.rows, q_heads)) < 0.01).cuda()
    q[which, 7] = 2.0 ** far
    w = s.cache.no_weights() if weights else None
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu, weights=w)
    small = q.clone()
    small[..., 7] = 0  # the number has no part in the scores, and none in the oracle's slack
    want, slack, shares, off, status = c4.attend4(s.o, small.double().cpu().numpy(), s.table, s.lengths, s.cu, query_error=2.0 ** -16)
    close(out, want, slack, BF)
    if weights:
        import evict_oracle as eo
        want_w, slack_w = eo.weigh(s.o, np.zeros(tuple(w.shape)), shares, off, s.table, s.lengths, s.cu, s.rows)
        assert (np.abs(w.double().cpu().numpy() - want_w) <= slack_w).all()
    assert int(s.cache.status.item()) == status == 0


def test_tiles_without_such_a_number_are_as_they_were(ltc):
    """One row's changes its tile's way into the products, and no other's."""
    s, q_heads = far_rows(ltc, 128, 93)
    q, _ = s.rows16(q_heads, 1.0)
    plain = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    q[s.rows - 1, 3, 7] = 2.0 ** 30
    out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    last = s.rows - int(s.cu[-1] - s.cu[-2])
    assert torch.equal(out[:last], plain[:last])
    assert torch.allclose(out[last:].float(), plain[last:].float(), atol=6 * 2.0 ** -7)


def test_captured(ltc):
    """Replays with queries that take the one way, and the other."""
    s, q_heads = far_rows(ltc, 128, 94)
    q, _ = s.rows16(q_heads, 1.0)
    ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)
    for i in range(5):
        q.copy_(s.rows16(q_heads, 1.0)[0])
        if i % 2:
            q[::3, ::5, 7] = 2.0 ** 20
        graph.replay()
        assert torch.equal(out, ltc.cache_attend(s.cache, q, s.gtable, s.glengths, s.gcu)) and bool(out.any())
        torch.cuda.synchronize()
