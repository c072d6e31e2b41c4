"""The state cache's page operations against their plain forms. Bytes move as they are: every
comparison is exact."""
import pytest
import torch

import plain64
from context_scan_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def make(layers, num, page, seed=0, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn((layers, num, *page), generator=gen).to(dtype), gen
    return torch.randint(0, 256, (layers, num, *page), generator=gen).to(dtype), gen


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def err(ws):
    return gdn.gdn_check_device_error(ws)[0]


# layers, pages, shape of a page, type: pages from 16 bytes to beyond several pieces, not a multiple
# of a piece, thousands of pages (more than one round of the block that makes the jobs)
SHAPES = {
    "one_page": (1, 1, (4,), torch.float32),
    "sixteen_bytes": (3, 20, (16,), torch.uint8),
    "odd_page": (2, 33, (7, 1052), torch.float32),
    "state_page": (2, 12, (4, 128, 128), torch.float32),
    "bf16_page": (5, 9, (3, 8, 24), torch.bfloat16),
    "many_pages": (2, 9001, (4, 4), torch.float32),
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("seed", [1, 2])
def test_copy(name, seed):
    layers, num, page, dtype = SHAPES[name]
    pages, gen = make(layers, num, page, seed, dtype)
    order = torch.randperm(num, generator=gen).tolist()
    half = (num + 1) // 2
    src = [order[i % half] if i % 5 else -1 for i in range(num - half)]     # sources repeat
    dst = [x if i % 7 != 6 else -1 for i, x in enumerate(order[half:])]
    src += [order[0], -3]
    dst += [order[0], -1]                  # a page onto itself, a pair of nothing
    if name == "one_page":
        src, dst = [-1], [0]
    elif order[0] in src:
        src, dst = src[:-2], dst[:-2]      # (a page that others read is no dst)
    d, ws = pages.cuda(), gdn.alloc_cache_workspace(num, len(src))
    gdn.gdn_cache_copy(d, ints(src), ints(dst), ws)
    want, bad = plain64.cache_copy(pages, src, dst) if num < 1000 else (None, False)
    if want is None:
        want = pages.clone()
        keep = [i for i, b in enumerate(dst) if b >= 0]
        s = torch.tensor([src[i] for i in keep])
        want[:, [dst[i] for i in keep]] = pages[:, s.clamp(min=0)] * (s >= 0).view(1, -1, 1, 1)
    assert err(ws) == 0 and not bad
    assert torch.equal(d.cpu(), want)


@pytest.mark.parametrize("src,dst", [
    ([0, 1, 2], [5, 5, 6]),          # one page twice
    ([0, 1, 2], [1, 7, 8]),          # a page that another pair reads
    ([0, 1], [1, 0]),                # a swap
    ([0, 1, 3, 3], [1, 2, 3, 4]),    # a chain; a page onto itself that another pair reads
    ([0, 12, 1], [4, 5, 6]),         # past the cache
    ([0, 1], [12, 6]),
    ([2**31 - 1, 1], [-1, 6]),
    ([-1, -1, 4], [3, 3, 3]),
])
def test_copy_refusals(src, dst):
    pages, _ = make(2, 12, (6, 8))
    d, ws = pages.cuda(), gdn.alloc_cache_workspace(12, 4)
    gdn.gdn_cache_copy(d, ints(src), ints(dst), ws)
    want, bad = plain64.cache_copy(pages, src, dst)
    assert bad and err(ws) == 1
    assert torch.equal(d.cpu(), want)
    gdn.gdn_cache_copy(d, ints([]), ints([]), ws)      # nothing to do
    assert err(ws) == 0 and torch.equal(d.cpu(), want)


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("kind", ["room", "full", "refused"])
def test_fork(name, kind):
    layers, num, page, dtype = SHAPES[name]
    pages, gen = make(layers, num, page, 3, dtype)
    refs = torch.randint(0, 3, (num,), generator=gen).tolist()
    used = [p for p, r in enumerate(refs) if r > 0]
    free = num - len(used)
    n = free // 2 if kind == "room" else free + 3
    parents = [used[i % len(used)] if used and i % 4 else -1 for i in range(n)]
    if kind == "refused":
        parents[::3] = [num + 5 if i % 2 else (refs.index(0) if 0 in refs else num)
                        for i in range(len(parents[::3]))]
    d, r = pages.cuda(), ints(refs)
    children = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    ws = gdn.alloc_cache_workspace(num, n)
    gdn.gdn_cache_fork(d, r, ints(parents), children, ws)
    want, refs2, kids, code = plain64.cache_fork(pages, refs, parents)
    assert err(ws) == code
    assert children.tolist() == kids and r.tolist() == refs2
    assert torch.equal(d.cpu(), want)


def test_fork_shared_and_freed():
    pages, _ = make(2, 10, (8, 4))
    refs = [1, 0, 2, 0, 1, 0, 0, 0, 0, -1]
    d, r, ws = pages.cuda(), ints(refs), gdn.alloc_cache_workspace(10, 6)
    kids = ints([2, 2, 0, 1, -1, 10])
    gdn.gdn_cache_fork(d, r, kids, kids, ws, share=True)      # in place
    assert err(ws) == 1                                       # a free page, none, one past the end
    assert kids.tolist() == [2, 2, 0, -1, -1, -1]
    assert r.tolist() == [2, 0, 4, 0, 1, 0, 0, 0, 0, -1] and torch.equal(d.cpu(), pages)
    gdn.gdn_cache_free(r, kids, ws)
    assert err(ws) == 0 and r.tolist() == refs
    # freed more often than used, beyond the end, again
    gdn.gdn_cache_free(r, ints([2, 2, 2, 4, -5, 2, 10]), ws)
    assert err(ws) == 1 and r.tolist() == [1, 0, 0, 0, 0, 0, 0, 0, 0, -1]
    gdn.gdn_cache_free(r, ints([0] * 1000), ws)
    assert err(ws) == 1 and r.tolist() == [0, 0, 0, 0, 0, 0, 0, 0, 0, -1]


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("kind", ["mixed", "none", "all", "front", "back"])
def test_compact(name, kind):
    layers, num, page, dtype = SHAPES[name]
    pages, gen = make(layers, num, page, 5, dtype)
    refs = torch.randint(0, 3, (num,), generator=gen).tolist()
    if kind == "none":
        refs = [0] * num
    elif kind == "all":
        refs = [2] * num
    elif kind in ("front", "back"):
        refs = [1 if (p < num // 2) == (kind == "front") else 0 for p in range(num)]
    used = [p for p, r in enumerate(refs) if r > 0]
    table = used[::-1][:300] + [-1, -9]
    want, refs2, table2, remap2, live2 = plain64.cache_compact(pages, refs, table)
    d, r, t = pages.cuda(), ints(refs), ints(table)
    remap = torch.full((num,), 77, dtype=torch.int32, device="cuda")
    live = ints([-1])
    ws = gdn.alloc_cache_workspace(num)
    gdn.gdn_cache_compact(d, r, t, remap, live, ws)
    assert err(ws) == 0
    assert live.item() == live2 and r.tolist() == refs2
    assert remap.tolist() == remap2 and t.tolist() == table2
    assert torch.equal(d.cpu(), want)
    # once more, with nothing to move and without the optional arrays
    gdn.gdn_cache_compact(d, r, None, None, None, ws)
    assert err(ws) == 0 and r.tolist() == refs2 and torch.equal(d.cpu(), want)


def test_compact_refuses_table_entries_of_free_pages():
    pages, _ = make(1, 6, (16,))
    refs = [0, 1, 0, 1, 0, 1]
    d, r, t = pages.cuda(), ints(refs), ints([5, 4, 6, 1, -1, 3])
    ws = gdn.alloc_cache_workspace(6)
    gdn.gdn_cache_compact(d, r, t, None, None, ws)
    assert err(ws) == 1
    assert t.tolist() == [2, -1, -1, 1, -1, 0]


def test_captured_cycle_on_a_side_stream():
    # fork, free and compact captured in two graphs that share one workspace, replayed in turn
    pages, gen = make(3, 40, (4, 64))
    refs = [1 if p % 3 else 0 for p in range(40)]
    base, r0 = pages.cuda(), ints(refs)
    parents = ints([1, 2, 4, -1, 5])
    d, r = base.clone(), r0.clone()
    kids, live = ints([0] * 5), ints([0])
    ws = gdn.alloc_cache_workspace(40, 5)

    def cycle(drop):
        gdn.gdn_cache_fork(d, r, parents, kids, ws)
        gdn.gdn_cache_free(r, drop, ws)
        gdn.gdn_cache_compact(d, r, kids, None, live, ws)

    drops = [ints([7, 8]), ints([20])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs = []
        for drop in drops:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                cycle(drop)
            graphs.append(graph)
        for i in range(4):
            d.copy_(base)
            r.copy_(r0)
            graphs[i % 2].replay()
            side.synchronize()
            w, rr, kk, code = plain64.cache_fork(pages, refs, parents.tolist())
            for p in drops[i % 2].tolist():
                rr[p] -= 1
            w, rr, kk, _, ll = plain64.cache_compact(w, rr, kk)
            assert code == 0 and gdn.gdn_check_device_error(ws) == (0, 0)
            assert torch.equal(d.cpu(), w) and r.tolist() == rr and kids.tolist() == kk
            assert live.item() == ll


def test_cache_past_four_gigabytes():
    # layer and page offsets past 2^32 bytes, in a cache with a count a page beyond one round
    layers, num, page = 2, 20000, 65536
    d = torch.empty((layers, num, page // 4), device="cuda")
    mark = torch.arange(page // 4, dtype=torch.float32, device="cuda")
    d[1, num - 1] = mark
    d[0, num - 1] = -mark
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    refs[num - 1] = 1
    ws = gdn.alloc_cache_workspace(num, 1)
    gdn.gdn_cache_copy(d, ints([num - 1]), ints([num - 3]), ws)
    table = ints([num - 1])
    gdn.gdn_cache_compact(d, refs, table, None, None, ws)
    assert err(ws) == 0 and table.tolist() == [0]
    for p in (0, num - 3):
        assert torch.equal(d[1, p], mark) and torch.equal(d[0, p], -mark)
