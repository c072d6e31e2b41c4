"""Calls of the chunked linear attention one behind the other, with other inputs each time and nothing in the workspace that an
earlier call could have left for the next one: what a call reads of its workspace is its own."""
import pytest
import torch

from context_scan_gb300 import gdn
from test_gpu_linear import BF, F32, make, nans, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

# lengths, heads, heads of q and k, K, V; whether the plan cuts the batch
BATCHES = {
    "whole": ([320, 0, 5, 635, 640, 1500, 0, 165], 16, 8, 128, 128, False),
    "whole_k64": ([1500, 3, 700, 250, 1100, 90, 640], 16, 4, 64, 128, False),
    "cut": ([9000, 85, 4500, 0, 7500], 2, 1, 128, 128, True),
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def entries_of_phase_2(ws):
    return int(ws[132:136].view(torch.int32).cpu())


@pytest.mark.parametrize("name", sorted(BATCHES))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_of_other_inputs_each_time(name, dtype):
    lens, H, Hqk, K, V, cut = BATCHES[name]
    sets = [make(lens, H, Hqk, K, V, dtype=dtype, seed=s) for s in (1, 2, 3)]
    wants = [run_bwd(d) for d in sets]
    assert all(w[4] == 0 for w in wants)
    ws = gdn.alloc_linear_workspace(sets[0]["k"], sets[0]["v"], sets[0]["cu"], backward=True)
    got = []
    for i in range(24):
        d = sets[i % 3]
        ws[256:] = 255          # NaN in every sum and state of the call before
        g = [nans(*w.shape, dtype=w.dtype) for w in wants[0][:4]]
        gdn.gdn_linear_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["do"], d["dht"], *g, ws, cu_seqlens=d["cu"])
        got.append(g)
    assert gdn.gdn_check_device_error(ws)[0] == 0
    for i, g in enumerate(got):
        for a, b in zip(g, wants[i % 3]):
            assert torch.equal(a, b), i
    if dtype == BF:
        assert (entries_of_phase_2(ws) > 0) == cut


@pytest.mark.parametrize("name", sorted(BATCHES))
def test_forward_of_other_inputs_each_time(name):
    # and a kernel of the caller's right behind each call
    lens, H, Hqk, K, V, _ = BATCHES[name]
    sets = [make(lens, H, Hqk, K, V, seed=s) for s in (1, 2, 3)]
    wants = [run_fwd(d) for d in sets]
    ws = gdn.alloc_linear_workspace(sets[0]["k"], sets[0]["v"], sets[0]["cu"])
    o, ht = nans(*wants[0][0].shape, dtype=BF), nans(*wants[0][1].shape, dtype=F32)
    got = []
    for i in range(24):
        d = sets[i % 3]
        ws[256:] = 255
        o.fill_(float("nan"))
        gdn.gdn_linear_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], o, ht, ws, cu_seqlens=d["cu"])
        got.append((o.clone(), ht.clone()))
    assert gdn.gdn_check_device_error(ws)[0] == 0
    for i, (a, b) in enumerate(got):
        assert torch.equal(a, wants[i % 3][0]) and torch.equal(b, wants[i % 3][1]), i


def test_captured_gradients_of_a_whole_batch():
    lens, H, Hqk, K, V, _ = BATCHES["whole"]
    sets = [make(lens, H, Hqk, K, V, seed=s) for s in (1, 2)]
    wants = [run_bwd(d) for d in sets]
    d = {n: None if x is None else x.clone() for n, x in sets[0].items() if n in ("q", "k", "v", "do", "decay", "h0", "dht", "cu")}
    ws = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"], backward=True)
    g = [nans(*w.shape, dtype=w.dtype) for w in wants[0][:4]]
    copies = [torch.empty_like(x) for x in g]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ws[256:].fill_(255)
        gdn.gdn_linear_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["do"], d["dht"], *g, ws, cu_seqlens=d["cu"])
        for c, x in zip(copies, g):
            c.copy_(x)
    for i in range(10):
        for n in d:
            d[n].copy_(sets[i % 2][n])
        graph.replay()
        torch.cuda.synchronize()
        for c, b in zip(copies, wants[i % 2]):
            assert torch.equal(c, b), i
    assert gdn.gdn_check_device_error(ws)[0] == 0
