"""The example that serves a layer from the 8-bit cache."""
import importlib.util
import os

import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_cache.py")


def test_example():
    """Codes of numbers within 4.5 are off by at most 2^-4 of them, the values'
    part of a row's difference is at most that of their largest; the weights
    differ by exp of the scores' differences, which are sums of 128 such
    relative errors of random sign, 0.03 on average: together below 0.3."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    banner("serve_cache example")
    spec = importlib.util.spec_from_file_location("serve_cache", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    worst, share = m.main(steps=9)
    assert worst < 0.3
    assert 0.5 < share < 1.01
