"""Packed batches of a thousand sequences and more: the plan goes over them in several rounds of its block, with sequences that
are cut in each of them. Tolerances: those of test_gpu_linear.py."""
import pytest
import torch

from context_scan_gb300 import gdn
from test_gpu_linear import BF, F32, absolute, close, make, reference, run_bwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def lengths(n, long):
    lens = [(5 * i) % 4 for i in range(n)]
    for at, length in long.items():
        lens[at] = length
    return lens


BATCHES = {
    "1024": lengths(1024, {3: 3000, 1023: 2000}),
    "1025": lengths(1025, {1023: 1500, 1024: 3001}),
    "1100": lengths(1100, {500: 2900, 1030: 1700, 1099: 2600}),
    "2500": lengths(2500, {0: 1300, 1100: 2500, 2048: 2000, 2499: 1}),
    "empty": lengths(600, {}) + [0] * 700 + [2200],
}


def table(ws, nseq):
    """The sequences in the order in which their first pieces start; the pieces behind first ones."""
    order = ws[256:256 + 16 * nseq].view(torch.int32).view(nseq, 4)[:, 0].cpu().tolist()
    return order, int(ws[132:136].view(torch.int32).cpu())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_forward(name, dtype):
    lens = BATCHES[name]
    d = make(lens, 1, 1, 64, 64, dtype=dtype, packed=True)
    ws = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"])
    o, ht, st = run_fwd(d, ws=ws)
    order, pieces = table(ws, len(lens))
    assert st == 0 and pieces > 0
    assert sorted(order) == list(range(len(lens)))
    chunks = [-(-lens[s] // 128) for s in order]
    assert chunks == sorted(chunks, reverse=True)
    o_ref, h_ref = reference(d)
    o_abs, h_abs = reference(absolute(d))
    close(d, o, o_ref, o_abs, "o")
    close(d, ht, h_ref, h_abs, "h", state=True)
    again = run_fwd(d, ws=ws)
    assert torch.equal(again[0], o) and torch.equal(again[1], ht)


@pytest.mark.parametrize("name", ["1024", "1100", "2500"])
def test_backward(name):
    lens = BATCHES[name]
    d = make(lens, 2, 1, 64, 64, packed=True)
    ws = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"], backward=True)
    *got, st = run_bwd(d, ws=ws)
    assert st == 0 and table(ws, len(lens))[1] > 0
    ref, bound = reference(d, True), reference(absolute(d), True)
    for what, g, r, b in zip(("dq", "dk", "dv"), got, ref, bound):
        close(d, g, r, b, what, rep=2)
    close(d, got[3], ref[3], bound[3], "dh0", state=True)


def test_very_many():
    # 70000 sequences of none to three tokens and one of 4000, in the last rounds: against the same sequences in two calls
    lens = [(5 * i) % 4 for i in range(70000)]
    lens[69000] = 4000
    d = make(lens, 1, 1, 64, 64, packed=True, start=False)
    o, ht, st = run_fwd(d)
    assert st == 0 and torch.isfinite(o).all()
    lo, at = sum(lens[:69000]), 69000
    alone = {**d, **{n: d[n][:, lo:lo + 4000].contiguous() for n in ("q", "k", "v")}, "lens": [4000], "n": 4000, "cu": None}
    ref, h_ref = reference(alone)
    bound, h_bound = reference(absolute(alone))
    close(alone, o[:, lo:lo + 4000], ref, bound, "o")
    close(alone, ht[at:at + 1], h_ref, h_bound, "h", state=True)
    short = {**d, **{n: d[n][:, :2000].contiguous() for n in ("q", "k", "v")}}
    few = next(i for i in range(70000) if sum(lens[:i]) >= 1990)
    short.update(lens=lens[:few], n=sum(lens[:few]), cu=d["cu"][:few + 1].contiguous())
    ref, h_ref = reference(short)
    bound, h_bound = reference(absolute(short))
    close(short, o[:, :2000], ref, bound, "o")
    close(short, ht[:few], h_ref, h_bound, "h", state=True)
