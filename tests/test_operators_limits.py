"""Counts near 2^31, which the operators over the state cache step through in 31 bits, are refused on the host
(no GPU: nothing here gets as far as a launch)."""
import pytest

from test_operators_host import FAKE, L  # noqa: F401

TOP = 2**31 - 1
ROOM = 1 << 62


@pytest.mark.parametrize("num,n", [(2**30 + 1, 3), (TOP - 8191, 3), (TOP, 3), (8, 2**30 + 1), (8, TOP - 1023),
                                   (8, TOP), (TOP, TOP)])
def test_cache_counts_past_30_bits(L, num, n):  # noqa: F811
    head, ws = (FAKE, 2, num, 16), (FAKE, ROOM, None)
    assert L.gdn_cache_copy(*head, n, FAKE, FAKE, *ws) == 2
    assert L.gdn_cache_fork(*head, FAKE, n, FAKE, FAKE, 0, *ws) == 2
    assert L.gdn_cache_compact(*head, FAKE, n, FAKE, None, None, *ws) == 2
    assert L.gdn_cache_free(num, FAKE, n, FAKE, *ws) == 2
    W = L.gdn_cache_workspace_bytes
    assert W(num, n) == 0 and W(2**30, 0) > 0 and W(1, 2**30) > 0
