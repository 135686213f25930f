"""Caches that share a stream's workspace: their calls in turn, and from several
threads, give what they give alone."""
import threading

import pytest
import torch

from cache4_setup import Setup4
from test_gpu_cache import Setup

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def layers(ltc):
    """Layers of unlike sizes, each with a cache of its own, and what a call on each gives."""
    out = [Setup4(ltc, 101, 2, 128, 32, BF, [1] * 5, [600, 5, 70, 3000, 31], single=True),
           Setup(ltc, 102, 1, 64, 64, "e4m3", FP, [1, 3], [9000, 20]), Setup(ltc, 103, 8, 256, 16, "int8", BF, [5, 1, 9], [300, 900, 10])]
    for s in out:
        s.q = s.rows16(s.H * 4)[0]
        s.w = s.cache.no_weights()
        s.want = ltc.cache_attend(s.cache, s.q, s.gtable, s.glengths, s.gcu)
        ltc.cache_attend(s.cache, s.q, s.gtable, s.glengths, s.gcu, weights=s.w)
        s.want_w = s.w.clone()
        s.w.zero_()
    return out


def call(ltc, s):
    s.w.zero_()
    got = [ltc.cache_attend(s.cache, s.q, s.gtable, s.glengths, s.gcu, weights=s.w), s.w.clone(),
           ltc.cache_attend(s.cache, s.q, s.gtable, s.glengths, s.gcu)]
    return [torch.equal(x, y) for x, y in zip(got, (s.want, s.want_w, s.want))]


def test_in_turn(ltc):
    a = layers(ltc)
    for _ in range(5):
        for s in a:
            assert all(call(ltc, s))


def test_from_threads(ltc):
    """All on one stream, so that calls of different caches come between each other."""
    a, wrong = layers(ltc), []
    torch.cuda.synchronize()

    def run(s):
        for _ in range(20):
            if not all(call(ltc, s)):
                wrong.append(s)

    threads = [threading.Thread(target=run, args=(s,)) for s in a]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
