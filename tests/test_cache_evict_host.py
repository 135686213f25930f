"""Eviction's new lengths in the place of the old ones, without a GPU: refused,
since a sequence's heads would read what one of them writes."""
import pytest

from test_cache4_host import evict
from test_cache_host import P, cache, seqs


@pytest.mark.parametrize("new", [P, P + 4, P + 8, P - 8])
@pytest.mark.parametrize("codes", [0, 1, 3])
def test_lengths_in_their_own_place(codes, new):
    s = seqs(cu=0, n=3, rows=3)
    assert evict(cache(codes=codes), s, lengths=new) == -1
