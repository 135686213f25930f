"""A cache whose codes pass 4 GiB: every operator on its last pages gives the
bits that it gives on the first ones of a small cache."""
import pytest
import torch

from gpu_util import banner

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HEADS, DIM, PAGE = 8, 256, 256


@pytest.fixture(scope="module")
def ltc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import lossless_tensor_compression_amd as m
    m.lib()
    return m


def serve(ltc, codes, cache, weights, first, new, past, seed):
    """Sequences on pages first, first + 1, ..: written, read, attended to with weights, cut, attended to again."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    total = [n + p for n, p in zip(new, past)]
    width = -(-max(total) // PAGE)
    table = first + torch.arange(len(new) * width, **i32).view(len(new), width)
    to = int(table.max()) + 1 + torch.arange(len(new), **i32)[:, None]
    lengths = torch.tensor(total, **i32)
    out = []
    x = lambda rows, heads: torch.randn((rows, heads, DIM), generator=g, device="cuda").to(BF)  # noqa: E731
    cu = torch.cumsum(torch.tensor([0] + total), 0).to(torch.int32).cuda()
    ltc.cache_write(cache, x(sum(total), HEADS), x(sum(total), HEADS), table, lengths, cu)
    out += ltc.cache_read(cache, table, lengths, cu, rows=sum(total))
    cu = torch.cumsum(torch.tensor([0] + new), 0).to(torch.int32).cuda()
    q = x(sum(new), 2 * HEADS)
    out.append(ltc.cache_attend(cache, q, table, lengths, cu, weights=weights))
    kept, positions = ltc.cache_evict(cache, weights, table, lengths, to, 100, 9)
    out += [kept, positions, ltc.cache_attend(cache, q[:len(new)], to, kept, weights=weights), *ltc.cache_read(cache, to, kept)]
    cache.check()
    used = slice(first, int(to.max()) + 1)
    return out + [t[used].clone() for t in (cache.k_codes, cache.v_codes, cache.scales, weights)]


@pytest.mark.parametrize("new,past", [([1, 3, 2], [300, 700, 90]), ([200, 3], [60, 500])])
@pytest.mark.parametrize("codes", ["e2m1", "int8"])
def test_last_pages(ltc, codes, new, past):
    banner(f"last pages of a cache past 4 GiB, {codes}")
    bytes_ = HEADS * PAGE * DIM // (2 if codes == "e2m1" else 1)
    pages = (5 << 30) // bytes_
    need = len(new) * (-(-max(n + p for n, p in zip(new, past)) // PAGE) + 1)
    small = ltc.KVCache.empty(need, HEADS, DIM, page=PAGE, codes=codes)
    want = serve(ltc, codes, small, small.no_weights(), 0, new, past, 7)
    large = ltc.KVCache.empty(pages, HEADS, DIM, page=PAGE, codes=codes)
    assert large.k_codes.numel() > 1 << 32
    got = serve(ltc, codes, large, large.no_weights(), pages - need, new, past, 7)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert not large.k_codes[:pages - need].any() and not large.v_codes[:pages - need].any()
    del large, got
    torch.cuda.empty_cache()
