"""An infinity or a NaN in one value of one token of the chunked linear attention reaches what the formulas let it reach, and
nothing else: where the plain 64-bit form of the same inputs is finite, the results have the bits of the clean call, and
nowhere else are they finite. (Of a batch padded behind each sequence's last token, say, whose padding holds anything.)"""
import pytest
import torch

from context_scan_gb300 import gdn
from test_gpu_linear import BF, F32, make, reference, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# lengths, H, Hqk, K, V; the places (tensor, row of all tokens, head, channel)
BATCHES = {
    "chunk": ([128, 128], 2, 2, 128, 128),
    "short": ([300, 300], 4, 2, 128, 128),
    "packed": ([70, 200, 131], 2, 1, 128, 128),
    "k64": ([200, 7, 129], 2, 2, 64, 64),
    "k64_v128": ([200, 131], 4, 2, 64, 128),
    "k128_v64": ([200, 131], 2, 1, 128, 64),
    "pieces": ([1700], 1, 1, 128, 128),
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def same_but_there(got, clean, ref, what):
    got, clean, ref = got.float().cpu(), clean.float().cpu(), ref.reshape(got.shape)
    bad = ~torch.isfinite(ref)
    assert torch.isfinite(clean).all(), what
    assert not torch.isfinite(got[bad]).any(), what
    assert torch.equal(got[~bad], clean[~bad]), what
    return int(bad.sum())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tensor", ["q", "k", "v", "do"])
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_one_value(name, tensor, dtype):
    lens, H, Hqk, K, V = BATCHES[name]
    d = make(lens, H, Hqk, K, V, dtype=dtype, seed=11)
    clean_f, clean_b = run_fwd(d), run_bwd(d)
    n, heads, channels = d["n"], d[tensor].shape[2], d[tensor].shape[3]
    keep = d[tensor].clone()
    for i, (row, value) in enumerate([(0, NAN), (n // 2 + 3, INF), (n // 3, -INF), (n - 1, NAN), (63, NAN), (64, INF)]):
        d[tensor] = keep.clone()
        d[tensor].view(-1, heads, channels)[row, i % heads, (37 * i + 5) % channels] = value
        o, ht, st = run_fwd(d)
        g = run_bwd(d)
        assert st == 0 and g[4] == 0
        there = 0
        for what, a, b, r in zip(("o", "h"), (o, ht), clean_f, reference(d)):
            there += same_but_there(a, b, r, (what, row))
        for what, a, b, r in zip(("dq", "dk", "dv", "dh0"), g, clean_b, reference(d, True)):
            there += same_but_there(a, b, r, (what, row))
        assert there > 0


@pytest.mark.parametrize("name", ["short", "k64", "k64_v128", "k128_v64", "pieces"])
def test_many_values(name):
    # several in a chunk, in chunks one behind the other, in every tensor
    lens, H, Hqk, K, V = BATCHES[name]
    d = make(lens, H, Hqk, K, V, seed=12)
    clean_f, clean_b = run_fwd(d), run_bwd(d)
    gen = torch.Generator().manual_seed(3)
    for tensor in ("q", "k", "v", "do"):
        keep = d[tensor].clone()
        flat = d[tensor].view(-1, *d[tensor].shape[2:])
        # (one head, late tokens: what comes before them, and the other heads' columns, are there to be kept)
        lo = d["n"] // 2 if tensor != "do" else 0
        hi = d["n"] if tensor != "do" else d["n"] // 2
        for _ in range(12):
            row = int(torch.randint(lo, hi, (1,), generator=gen))
            c = int(torch.randint(0, flat.shape[2] // 2, (1,), generator=gen))
            flat[row, 0, c] = (NAN, INF, -INF)[int(torch.randint(0, 3, (1,), generator=gen))]
        o, ht, _ = run_fwd(d)
        g = run_bwd(d)
        for what, a, b, r in zip(("o", "h"), (o, ht), clean_f, reference(d)):
            same_but_there(a, b, r, (tensor, what))
        for what, a, b, r in zip(("dq", "dk", "dv", "dh0"), g, clean_b, reference(d, True)):
            same_but_there(a, b, r, (tensor, what))
        d[tensor] = keep


@pytest.mark.parametrize("dtype", [BF, F32])
def test_garbage_behind_each_sequence_of_a_batch(dtype):
    # sequences of 200, 70 and 130 tokens in rows of 300
    d = make([300, 300, 300], 2, 1, 128, 128, dtype=dtype, seed=13)
    clean = run_fwd(d)[0]
    for n in ("q", "k", "v"):
        for s, length in enumerate((200, 70, 130)):
            d[n][s, length:] = NAN if s < 2 else INF
    o = run_fwd(d)[0]
    for s, length in enumerate((200, 70, 130)):
        assert torch.equal(o[s, :length], clean[s, :length])
        assert not torch.isfinite(o[s, length:]).any()


def same_bits(a, b):
    return torch.equal(torch.nan_to_num(a, nan=7.0), torch.nan_to_num(b, nan=7.0)) and torch.equal(torch.isnan(a), torch.isnan(b))


def test_clean_and_bad_calls_in_turn():
    # many blocks at work, pieces and whole sequences, one call behind the other without a wait on the host
    lens = [3000, 0, 85, 640, 2500, 1, 1500]
    clean = make(lens, 16, 8, 128, 128, seed=14)
    bad = {**clean, "v": clean["v"].clone(), "do": clean["do"].clone()}
    for row in (5, 2999, 3080, 4000, 6222):
        bad["v"][0, row, :, row % 128] = NAN
        bad["do"][0, row + 1, row % 16, 3] = INF
    wants = [(run_fwd(d), run_bwd(d)) for d in (clean, bad)]
    wf = gdn.alloc_linear_workspace(clean["k"], clean["v"], clean["cu"])
    wb = gdn.alloc_linear_workspace(clean["k"], clean["v"], clean["cu"], backward=True)
    o, ht = torch.empty_like(wants[0][0][0]), torch.empty_like(wants[0][0][1])
    g = [torch.empty_like(x) for x in wants[0][1][:4]]
    for i in range(60):
        d, (f, b) = (clean, bad)[i % 2], wants[i % 2]
        gdn.gdn_linear_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], o, ht, wf, cu_seqlens=d["cu"])
        gdn.gdn_linear_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["do"], d["dht"], *g, wb, cu_seqlens=d["cu"])
        assert same_bits(o, f[0]) and same_bits(ht, f[1]) and all(same_bits(x, y) for x, y in zip(g, b)), i
    for _ in range(100):
        gdn.gdn_linear_bwd(bad["q"], bad["k"], bad["v"], bad["decay"], bad["h0"], bad["do"], bad["dht"], *g, wb, cu_seqlens=bad["cu"])
    assert all(same_bits(x, y) for x, y in zip(g, wants[1][1]))
    assert gdn.gdn_check_device_error(wf)[0] == 0 and gdn.gdn_check_device_error(wb)[0] == 0
