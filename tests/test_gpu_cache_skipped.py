"""Pairs that gdn_cache_copy skips (a negative dst) take no part in the call: a list padded to the
fixed length of a captured graph holds stale sources. Every comparison is exact."""
import pytest
import torch

from context_scan_gb300 import gdn
from test_gpu_cache import _lib, err, ints, make  # noqa: F401

pytestmark = pytest.mark.gpu

LISTS = [
    ([3, 1], [1, -1]),                         # the skipped pair's source is written
    ([1, 3], [-7, 1]),                         # ... from in front
    ([1, 1, 3, 1], [-1, -2, 1, -1]),           # named by several
    ([3, 4, 2, 1, 0], [1, 2, -1, -1, 0]),      # beside a page onto itself
    ([-1, 5, 6], [5, -1, 7]),                  # zeros
    ([5] * 2000, [-1] * 1999 + [6]),           # more pairs than the block has threads
    ([6] * 2000 + [2], [-1] * 2000 + [6]),
]


def plain(pages, src, dst):
    after = pages.clone()
    for a, b in zip(src, dst):
        if b >= 0:
            after[:, b] = pages[:, a] if a >= 0 else 0
    return after


@pytest.mark.parametrize("src,dst", LISTS)
def test_skipped_pairs_read_nothing(src, dst):
    pages, _ = make(2, 12, (6, 8))
    d, ws = pages.cuda(), gdn.alloc_cache_workspace(12, len(src))
    gdn.gdn_cache_copy(d, ints(src), ints(dst), ws)
    assert err(ws) == 0
    assert torch.equal(d.cpu(), plain(pages, src, dst))


def test_pairs_that_do_something_are_refused_as_before():
    pages, _ = make(2, 12, (6, 8))
    d, ws = pages.cuda(), gdn.alloc_cache_workspace(12, 4)
    # (page 1 is read by the second pair, and named by a skipped one)
    gdn.gdn_cache_copy(d, ints([3, 1, 1, 0]), ints([1, 2, -1, 4]), ws)
    want = pages.clone()
    want[:, 2], want[:, 4] = pages[:, 1], pages[:, 0]
    assert err(ws) == 1 and torch.equal(d.cpu(), want)


def test_captured_list_of_fixed_length():
    pages, _ = make(3, 10, (4, 16))
    d, ws = pages.cuda(), gdn.alloc_cache_workspace(10, 4)
    src, dst = ints([0, 1, 2, 3]), ints([4, 5, 6, 7])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gdn.gdn_cache_copy(d, src, dst, ws)
        for a, b in LISTS[:1] + [([9, 8, 7, 4], [4, -1, -1, -1]), ([-1, 0, 2, 3], [2, 3, -1, -1])]:
            a, b = a + [5] * (4 - len(a)), b + [-1] * (4 - len(b))
            d.copy_(pages)
            src.copy_(ints(a))
            dst.copy_(ints(b))
            graph.replay()
            side.synchronize()
            assert err(ws) == 0 and torch.equal(d.cpu(), plain(pages, a, b))
