"""GPU parity of the chunked linear attention with a decay for each head (gdn_linear_fwd, gdn_linear_bwd) against the
plain 64-bit forms, its refusals on the device, other streams, graphs, padded batches.

Tolerances, derived: every result is a sum of products whose absolute values add up to A, the same form on absolute
values (inputs, and the states they start from). In fp32 a term passes at most K roundings in its product, 64 in a
step of 32 tokens and four for each later step: with n tokens, (K + 64 + 4 (n / 32 + 1)) 2^-24 A. With bf16 inputs
and outputs the products are exact, and a term of an output is rounded once to bf16 (the weighted attention, or the state
it reads), half a step or 2^-8 of it; a term of a state is good to 2^-17; both then pass the fp32 sums above. A bf16 result adds
half a step of itself. Beside these bounds, which no input can exceed, the RMS error of bf16 results stays under 2^-8 of their
RMS: three roundings of at most 2^-8 / sqrt(3) each.
"""
import numpy as np
import pytest
import torch

import plain64_linear as plain
from context_scan_gb300 import gdn
from gpu_util import record

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def slopes(H, gen):
    s = -(2.0 ** (-8.0 * (torch.arange(H) + 1) / H))
    return s * torch.empty(H).uniform_(0.8, 1.2, generator=gen)


def make(lens, H, Hqk, K, V, dtype=BF, out=None, start=True, packed=None, pad=0, seed=0, decay=None):
    gen = torch.Generator().manual_seed(77 + seed)
    out = out or dtype
    n, nseq = sum(lens), len(lens)
    if packed is None:
        packed = len(set(lens)) > 1
    lead = (1, n + pad) if packed else (nseq, lens[0])
    normal = lambda *s, sd=1.0: torch.randn(*s, generator=gen) * sd  # noqa: E731
    unit = torch.nn.functional.normalize
    d = {"q": unit(normal(*lead, Hqk, K), dim=-1).to(dtype), "k": unit(normal(*lead, Hqk, K), dim=-1).to(dtype),
         "v": normal(*lead, H, V).to(dtype), "do": normal(*lead, H, V).to(out)}
    d = {name: x.cuda() for name, x in d.items()}
    d["decay"] = (slopes(H, gen) if decay is None else torch.tensor(decay, dtype=F32)).cuda()
    d["h0"] = normal(nseq, H, K, V, sd=0.3).cuda() if start else None
    d["dht"] = normal(nseq, H, K, V, sd=0.3).cuda() if start else None
    d["cu"] = None
    if packed:
        d["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    d["lens"], d["n"], d["out"], d["dtype"] = list(lens), n, out, dtype
    return d


def nans(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def run_fwd(d, ws=None, stream=None, final=True):
    nseq, (H, V), K = len(d["lens"]), d["v"].shape[2:], d["k"].shape[3]
    o = nans(*d["v"].shape, dtype=d["out"])
    ht = nans(nseq, H, K, V, dtype=F32) if final else None
    ws = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"]) if ws is None else ws
    gdn.gdn_linear_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], o, ht, ws, cu_seqlens=d["cu"], stream=stream)
    torch.cuda.synchronize()
    return o, ht, gdn.gdn_check_device_error(ws)[0]


def run_bwd(d, ws=None, want_dh0=True):
    g = {n: torch.full_like(d[n], float("nan")) for n in ("q", "k", "v")}
    nseq, (H, V), K = len(d["lens"]), d["v"].shape[2:], d["k"].shape[3]
    dh0 = nans(nseq, H, K, V, dtype=F32) if want_dh0 else None
    ws = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"], backward=True) if ws is None else ws
    gdn.gdn_linear_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["do"], d["dht"], g["q"], g["k"], g["v"], dh0, ws,
                       cu_seqlens=d["cu"])
    torch.cuda.synchronize()
    return g["q"], g["k"], g["v"], dh0, gdn.gdn_check_device_error(ws)[0]


def flat(d, *names):
    return [None if d[n] is None else d[n].reshape(-1, *d[n].shape[2:])[:d["n"]] for n in names]


def absolute(d):
    a = dict(d)
    for n in ("q", "k", "v", "do", "h0", "dht"):
        a[n] = None if d[n] is None else d[n].abs()
    return a


def reference(d, bwd=False):
    if bwd:
        q, k, v, do = flat(d, "q", "k", "v", "do")
        return plain.backward(q, k, v, d["decay"], d["h0"], do, d["dht"], d["lens"])
    return plain.forward(*flat(d, "q", "k", "v"), d["decay"], d["h0"], d["lens"])


def close(d, got, ref, bound, what, state=False, rep=1):
    if not ref.numel():
        return
    got = got.double().cpu()
    got = got if state else got.reshape(-1, *got.shape[2:])[:d["n"]]
    K, longest = d["k"].shape[3], max(d["lens"])
    tc = d["dtype"] == BF and d["out"] == BF
    term = (K + 64 + 4 * (longest // 32 + 1) + rep) * 2.0 ** -24 + (0 if not tc else 2.0 ** -17 if state else 2.0 ** -8)
    half = 0.0 if state or got.dtype == F32 else 2.0 ** -8
    out_half = half if (d["out"] if what == "o" else d["dtype"]) == BF else 0.0
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), what
    record(float((off / (term * bound + out_half * ref.abs() + 1e-30)).max()), what)
    assert (off <= term * bound + out_half * ref.abs() + 1e-30).all(), (what, float(off.max()))
    if not state:
        rms = float(off.square().mean().sqrt() / ref.square().mean().sqrt().clamp(min=1e-30))
        assert rms <= (2.0 ** -8 if tc else 2.0 ** -8 if out_half else 1e-5), (what, rms)
    else:
        rms = float(off.square().mean().sqrt() / ref.square().mean().sqrt().clamp(min=1e-30))
        assert rms <= 1e-5, (what, rms)


CASES = {
    # lengths, H, Hqk, K, V, options
    "one_token": ([1], 4, 2, 128, 128, {}),
    "one_token_batch": ([1] * 9, 3, 3, 128, 128, {}),
    "one_chunk": ([128], 2, 2, 128, 128, {}),
    "a_chunk_and_one": ([129], 2, 1, 128, 128, dict(start=False)),
    "two_sequences": ([300, 300], 3, 3, 128, 128, {}),
    "ragged": ([64, 0, 1, 127, 128, 300, 0, 33], 4, 2, 128, 128, {}),
    "ragged_no_start": ([5, 260, 131], 4, 1, 128, 128, dict(start=False)),
    "in_pieces": ([2900], 2, 2, 128, 128, {}),
    "in_pieces_no_start": ([3001], 1, 1, 128, 128, dict(start=False)),
    "packed_pieces": ([1800, 17, 900, 0, 1500], 2, 1, 128, 128, {}),
    "long_among_many_short": ([1 + i % 3 for i in range(300)] + [20000], 2, 1, 64, 128, {}),
    "k64": ([200, 7, 129], 3, 3, 64, 64, {}),
    "k64_v128": ([130, 0, 257], 4, 2, 64, 128, {}),
    "k128_v64": ([130, 1, 257], 4, 2, 128, 64, {}),
    "k64_v128_pieces": ([2500], 2, 1, 64, 128, {}),
    "k128_v64_pieces": ([2500], 2, 2, 128, 64, dict(start=False)),
    "many_short": ([(i * 7) % 23 for i in range(60)], 3, 3, 64, 64, {}),
    "fp32": ([130, 33], 2, 2, 64, 64, dict(dtype=F32)),
    "fp32_k128": ([70, 0, 95], 3, 1, 128, 128, dict(dtype=F32)),
    "fp32_pieces": ([2000], 1, 1, 128, 64, dict(dtype=F32)),
    "fp32_in_bf16_out": ([70, 131], 2, 1, 128, 128, dict(dtype=F32, out=BF)),
    "bf16_in_fp32_out": ([70, 131], 2, 1, 128, 128, dict(out=F32)),
    "no_decay": ([300], 2, 2, 128, 128, dict(decay=[0.0, -1e-6])),
    "strong_decay": ([300, 5], 5, 5, 128, 128, dict(decay=[-1.0, -6.0, -30.0, -1e30, float("-inf")])),
    "strong_decay_fp32": ([100, 5], 5, 5, 64, 64, dict(dtype=F32, decay=[-1.0, -6.0, -30.0, -1e30, float("-inf")])),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name):
    lens, H, Hqk, K, V, kw = CASES[name]
    d = make(lens, H, Hqk, K, V, **kw)
    o, ht, st = run_fwd(d)
    assert st == 0
    o_ref, h_ref = reference(d)
    o_abs, h_abs = reference(absolute(d))
    close(d, o, o_ref, o_abs, "o")
    close(d, ht, h_ref, h_abs, "h", state=True)


@pytest.mark.parametrize("name", sorted(CASES))
def test_backward(name):
    lens, H, Hqk, K, V, kw = CASES[name]
    d = make(lens, H, Hqk, K, V, **kw)
    *got, st = run_bwd(d)
    assert st == 0
    ref, bound = reference(d, True), reference(absolute(d), True)
    for what, g, r, b in zip(("dq", "dk", "dv"), got, ref, bound):
        close(d, g, r, b, what, rep=H // Hqk)
    close(d, got[3], ref[3], bound[3], "dh0", state=True)


def test_gradients_against_differences():
    # L = <dO, o> + <dht, h_final> along random directions, in fp32 with the 64-bit form for L: L is linear in each of
    # q, (k), (v) and h0, so a difference is exact up to the 64-bit form's roundings
    d = make([37, 90], 2, 1, 64, 64, dtype=F32)
    dq, dk, dv, dh0, _ = run_bwd(d)
    do, = flat(d, "do")

    def loss(**moved):
        e = {**d, **moved}
        o, h = reference(e)
        return float((o * do.double().cpu()).sum() + (h * d["dht"].double().cpu()).sum())

    gen = torch.Generator().manual_seed(5)
    for name, grad in (("q", dq), ("k", dk), ("v", dv), ("h0", dh0)):
        step = torch.randn(d[name].shape, generator=gen).cuda()
        diff = loss(**{name: d[name].double() + step.double()}) - loss()
        along = float((grad.double() * step.double()).sum())
        size = float(grad.double().norm() * step.double().norm())
        assert abs(diff - along) <= 1e-5 * size, name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padded_rows_stay(dtype):
    d = make([200, 0, 131], 2, 1, 128, 128, dtype=dtype, pad=150)
    for n in ("q", "k", "v", "do"):
        d[n][:, d["n"]:] = float("nan")       # read into nothing
    o, ht, st = run_fwd(d)
    assert st == 0 and torch.isnan(o[:, d["n"]:]).all() and torch.isfinite(o[:, :d["n"]]).all()
    o_ref, h_ref = reference(d)
    close(d, o, o_ref, reference(absolute(d))[0], "o")
    *g, st = run_bwd(d)
    assert st == 0
    for x in g[:3]:
        assert torch.isnan(x[:, d["n"]:]).all() and torch.isfinite(x[:, :d["n"]]).all()
    assert torch.isfinite(g[3]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_sequence_stays_alone(dtype, value):
    d = make([130, 70, 3, 200], 2, 2, 128, 128, dtype=dtype)
    clean = run_fwd(d), run_bwd(d)
    for n in ("q", "k", "v", "do"):
        d[n][:, 130:200] = value
    o, ht, _ = run_fwd(d)
    g = run_bwd(d)
    keep = [i for i in range(d["n"]) if not 130 <= i < 200]
    assert torch.equal(o[:, keep], clean[0][0][:, keep])
    for a, b in zip(g[:3], clean[1][:3]):
        assert torch.equal(a[:, keep], b[:, keep])
    others = [0, 2, 3]
    assert torch.equal(ht[others], clean[0][1][others]) and torch.equal(g[3][others], clean[1][3][others])
    assert not torch.isfinite(o[:, 199]).all()


@pytest.mark.parametrize("cu", [[1, 5, 9], [0, 7, 5], [0, 5, 10], [0, -3, 9], [0, 2**31 - 1, 9]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_lengths_write_nothing(cu, dtype):
    d = make([5, 4], 2, 1, 64, 64, dtype=dtype)
    d["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    o, ht, st = run_fwd(d)
    assert st == 1 and torch.isnan(o).all() and torch.isnan(ht).all()
    *g, st = run_bwd(d)
    assert st == 1 and all(torch.isnan(x).all() for x in g)


def test_no_tokens():
    d = make([0, 0, 0], 2, 1, 128, 64, packed=True)
    o, ht, st = run_fwd(d)
    assert st == 0 and torch.equal(ht, d["h0"])
    assert torch.equal(run_bwd(d)[3], d["dht"])
    d = make([0, 0], 2, 1, 128, 64, packed=False, start=False)
    assert torch.count_nonzero(run_fwd(d)[1]) == 0 and torch.count_nonzero(run_bwd(d)[3]) == 0


def test_optional_outputs():
    d = make([200, 131], 2, 2, 128, 128)
    o, _, _ = run_fwd(d, final=False)
    assert torch.equal(o, run_fwd(d)[0])
    a, b = run_bwd(d, want_dh0=False), run_bwd(d)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_same_bits_every_time(dtype):
    d = make([700, 3, 900], 4, 2, 128, 128, dtype=dtype)
    a, b = run_fwd(d), run_bwd(d)
    ws = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"], backward=True)
    ws[256:] = 255       # what an earlier call left
    for _ in range(3):
        for x, y in zip(run_fwd(d, ws=ws)[:2], a[:2]):
            assert torch.equal(x, y)
        for x, y in zip(run_bwd(d, ws=ws)[:4], b[:4]):
            assert torch.equal(x, y)


def test_graph_and_other_stream():
    # captured with one batch's lengths, replayed with others, in padded buffers
    d = make([300, 120, 80], 2, 1, 128, 128, pad=100)
    nseq, (H, V), K = 3, d["v"].shape[2:], 128
    side = torch.cuda.Stream()
    o, ht = nans(*d["v"].shape, dtype=BF), nans(nseq, H, K, V, dtype=F32)
    ws = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        gdn.gdn_linear_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], o, ht, ws, cu_seqlens=d["cu"])
    for lens in ([300, 120, 80], [10, 0, 590], [0, 0, 600]):
        d["lens"], d["n"] = lens, sum(lens)
        d["cu"].copy_(torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32))
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        again = run_fwd(d, stream=side)
        assert torch.equal(o[:, :d["n"]], again[0][:, :d["n"]]) and torch.equal(ht, again[1])
        assert torch.isnan(o[:, d["n"]:]).all()
    assert gdn.gdn_check_device_error(ws)[0] == 0


@pytest.mark.parametrize("name", ["packed_pieces", "in_pieces", "ragged"])
def test_many_calls_in_a_row(name):
    # one behind the other, without a wait on the host: no wait in a kernel runs out, every call gives the same
    lens, H, Hqk, K, V, kw = CASES[name]
    lens = [5 * n for n in lens]
    d = make(lens, 16, 8, K, V, **kw)
    o, ht, _ = run_fwd(d)
    g = run_bwd(d)
    wf = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"])
    wb = gdn.alloc_linear_workspace(d["k"], d["v"], d["cu"], backward=True)
    o2, ht2, g2 = torch.empty_like(o), torch.empty_like(ht), [torch.empty_like(x) for x in g[:4]]
    for _ in range(400):
        gdn.gdn_linear_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], o2, ht2, wf, cu_seqlens=d["cu"])
    for _ in range(100):
        gdn.gdn_linear_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["do"], d["dht"], *g2, wb, cu_seqlens=d["cu"])
    assert gdn.gdn_check_device_error(wf)[0] == 0 and gdn.gdn_check_device_error(wb)[0] == 0
    assert torch.equal(o, o2) and torch.equal(ht, ht2) and all(torch.equal(x, y) for x, y in zip(g, g2))


def test_split_and_joined_prompts_agree():
    # a prompt in one call, and in three that hand the state on
    d = make([1000], 3, 3, 128, 128, packed=False)
    whole, ht, _ = run_fwd(d)
    ref, h_ref = reference(d)
    h, parts = d["h0"], []
    for a, b in ((0, 333), (333, 334), (334, 1000)):
        e = {**d, **{n: d[n][:, a:b].contiguous() for n in ("q", "k", "v")}, "h0": h, "lens": [b - a], "n": b - a}
        o, h, _ = run_fwd(e)
        parts.append(o)
    bound, h_bound = reference(absolute(d))
    close(d, torch.cat(parts, 1), ref, bound, "o")
    close(d, h, h_ref, h_bound, "h", state=True)
