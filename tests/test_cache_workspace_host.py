"""What workspaces hold on to, without a GPU."""
import pytest
import torch

from cache_cpu import cpu_cache, sequences
from lossless_tensor_compression_amd import kv_cache as kc


@pytest.mark.parametrize("need,most", [(1, 1), (100000, 1 << 17), (1 << 24, 1 << 24), ((1 << 24) + 1, 18 << 20), (70 << 20, 72 << 20),
                                       ((1 << 27) + (1 << 20), 144 << 20), (1 << 30, 1 << 30)])
def test_room(need, most):
    """Large workspaces are at most an eighth larger than asked for."""
    assert need <= kc._room(need) <= most


def _attending(monkeypatch, need, taken):
    def attend(cache_ref, s, q, q_heads, window, scale, out, ws, size, stream):
        taken.append((ws, size))
        return 0

    return cpu_cache(monkeypatch, ltc_cache_attend=attend, ltc_cache_attend_workspace_size=lambda *a: need[0])


def test_caches_of_a_stream_share_one(monkeypatch):
    """A cache for each layer, one stream: one workspace, the largest that was asked for; gone with the caches."""
    need, taken = [200000], []
    caches = [_attending(monkeypatch, need, taken) for _ in range(4)]
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    for n in (200000, 900000, 30000):
        need[0] = n
        for c in caches:
            kc.cache_attend(c, q, *sequences([5]))
    assert len({ws for ws, _ in taken[:4]}) == len({ws for ws, _ in taken[4:]}) == 1
    assert [size for _, size in taken] == [1 << 18] * 4 + [1 << 20] * 8
    held = {id(ws) for c in caches for ws in c._workspaces.values()}
    assert len(held) == 1 and not next(iter(caches[0]._workspaces.values()))[:kc.WS_ZEROS].any()
    assert len({id(c._lock) for c in caches}) == 1  # a call's launches are not to be parted by another cache's
    del caches, c
    assert (kc_index, 0) not in kc._workspaces


kc_index = -1  # what the CPU tensors of these tests have for a GPU


def test_streams_have_their_own(monkeypatch):
    need, taken = [200000], []
    c = _attending(monkeypatch, need, taken)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    for stream in (0, 7, 0, 7):
        monkeypatch.setattr(kc, "_raw_stream", lambda index, stream=stream: stream)
        kc.cache_attend(c, q, *sequences([5]))
    a, b = taken[0][0], taken[1][0]
    assert a != b and [ws for ws, _ in taken] == [a, b, a, b]


def test_captured_calls_have_their_own(monkeypatch):
    need, taken = [200000], []
    c = _attending(monkeypatch, need, taken)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    kc.cache_attend(c, q, *sequences([5]))
    kept = dict(c._workspaces)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: True, raising=False)
    kc.cache_attend(c, q, *sequences([5]))
    assert taken[0][0] != taken[1][0] and c._workspaces == kept
