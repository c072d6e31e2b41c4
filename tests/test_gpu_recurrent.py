"""GPU parity of the recurrent rule over a state cache (gdn_recurrent_fwd) against its plain 64-bit
form, its refusals on the device, and its use with the other entry points.

Tolerance, derived: the kernel's fp32 sum over K = 128 rows joins at most 22 additions in a chain
(16 pairs in a lane, the pair, up to four lanes' exchanges), so a product with the state is off by at
most 22 * 2^-24 |H column| = 1.3e-6 |H column|, and |H column| is sqrt(K) = 11.3 times the RMS of
q^T H for unit q. With decays around 0.85 the errors of earlier tokens add up to 1 / (1 - 0.85) = 7
of these: 1.0e-4 of the RMS, the bar of the library's fp32 paths (TOL_F32). A bf16 output adds half
a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle
import plain64
from context_scan_gb300 import gdn, synth
from gpu_util import TOL_BF16, TOL_F32, np64, record, rel_err

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def make(lens, H, Hqk, K, V, dtype=BF, out=F32, gate_k=False, packed=None, seed=0, extra=3):
    """Tokens of these sequences and a cache with a slot per sequence and token and some more."""
    gen = torch.Generator().manual_seed(1000 + seed)
    n, nseq = sum(lens), len(lens)
    if packed is None:
        packed = len(set(lens)) > 1
    lead = (1, n) if packed else (nseq, lens[0])

    def normal(*shape, mean=0.0, sd=1.0):
        return torch.randn(shape, generator=gen) * sd + mean

    unit = torch.nn.functional.normalize
    d = {
        "q": unit(normal(*lead, Hqk, K), dim=-1),
        "k": unit(normal(*lead, Hqk, K), dim=-1),
        "v": normal(*lead, H, V),
        "g": torch.nn.functional.logsigmoid(normal(*lead, H, *((K,) if gate_k else ()), mean=2.0)),
        "beta": torch.sigmoid(normal(*lead, H)),
    }
    d = {name: x.to(dtype).cuda() for name, x in d.items()}
    d["state"] = normal(nseq + n + extra, H, K, V, sd=0.3).cuda()
    d["order"] = torch.randperm(nseq + n + extra, generator=gen).tolist()
    d["cu"] = None
    if packed:
        d["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    d["o"] = torch.full((*lead, H, V), float("nan"), dtype=out, device="cuda")
    d["lens"] = list(lens)
    return d


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32).cuda()


def call(d, slots_in, slots_out, per_token=False, decay_first=False, ws=None, state=None):
    state = d["state"].clone() if state is None else state
    ws = gdn.alloc_recurrent_workspace(state.shape[0]) if ws is None else ws
    gdn.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], state, ints(slots_in),
                          ints(slots_out), d["o"], ws, cu_seqlens=d["cu"], per_token=per_token,
                          decay_first=decay_first)
    torch.cuda.synchronize()
    return state, gdn.gdn_check_device_error(ws)


def reference(d, slots_in, slots_out, per_token=False, decay_first=False):
    flat = [d[n].reshape(-1, *d[n].shape[2:]) for n in ("q", "k", "v", "g", "beta")]
    return plain64.recurrence(*flat, d["state"], slots_in, slots_out, d["lens"], per_token, decay_first)


def check_o(d, o_ref):
    o = d["o"].double().cpu().reshape(o_ref.shape)
    if not o.numel():
        return
    rms = o_ref.square().mean().sqrt()
    half = torch.finfo(d["o"].dtype).eps / 2 if d["o"].dtype == BF else 0.0
    off = (o - o_ref).abs() - half * o_ref.abs()
    record(float(off.max() / rms), "o")
    assert (off <= TOL_F32 * rms).all(), float(off.max() / rms)


def check_state(d, after, ref, written):
    """Written slots to the tolerance, every other slot bit for bit as it was."""
    rest = [i for i in range(ref.shape[0]) if i not in set(written)]
    assert torch.equal(after[rest], d["state"][rest])
    if written:
        w = sorted(set(written))
        assert rel_err(np64(after[w]), ref[w].numpy(), label="state") <= TOL_F32


CASES = {
    # lengths, H, Hqk, K, V, options; the split of the state's columns goes by the number of
    # sequences and heads, so small and large batches run different instances
    "one_token_one_seq": ([1], 4, 2, 128, 128, {}),
    "one_token_batch": ([1] * 7, 4, 4, 128, 128, dict(out=BF)),
    "one_token_large_batch": ([1] * 340, 4, 1, 128, 128, {}),
    "two_tokens_mid_batch": ([2] * 170, 1, 1, 128, 128, {}),
    "past_the_block_check": ([1] * 515, 1, 1, 64, 64, {}),
    "ragged": ([3, 0, 17, 1, 8, 9, 0], 6, 2, 128, 128, {}),
    "ragged_large": ([(i * 5) % 11 for i in range(330)], 4, 2, 128, 128, {}),
    "ragged_v64_large": ([(i * 5) % 4 for i in range(400)], 8, 8, 128, 64, {}),
    "ragged_k64_v128_large": ([(i * 5) % 4 for i in range(400)], 8, 8, 64, 128, {}),
    "ragged_k64_large": ([(i * 5) % 4 for i in range(700)], 8, 4, 64, 64, {}),
    "long": ([200, 63, 65], 2, 1, 128, 128, {}),
    "k64": ([5, 16, 33], 3, 3, 64, 64, {}),
    "k64_v128": ([5, 0, 8], 3, 1, 64, 128, {}),
    "k128_v64": ([5, 7, 9], 3, 1, 128, 64, dict(out=BF)),
    "fp32": ([4, 11, 64], 3, 3, 128, 128, dict(dtype=F32)),
    "fp32_k64": ([4, 11, 64], 5, 5, 64, 64, dict(dtype=F32, out=BF)),
    "fp32_large": ([2] * 320, 4, 4, 128, 128, dict(dtype=F32)),
    "gate_k": ([4, 0, 30, 9], 4, 2, 128, 128, dict(gate_k=True)),
    "gate_k_fp32_k64": ([4, 10, 9], 4, 2, 64, 64, dict(gate_k=True, dtype=F32)),
    "gate_k_large": ([3] * 320, 4, 4, 128, 128, dict(gate_k=True)),
    "many_tokens_wide": ([30, 2, 17] * 30, 8, 4, 128, 128, {}),
    "many_tokens_wide_fp32_gate_k": ([24] * 64, 8, 8, 128, 128, dict(gate_k=True, dtype=F32)),
    "no_tokens_at_all": ([0, 0], 2, 1, 128, 128, dict(packed=True)),
    "no_tokens_unpacked": ([0, 0, 0], 2, 1, 64, 64, dict(packed=False)),
    # (2, 4 and 8 columns a warp by the number of warps, on some 150 SMs)
    "few_gate_k": ([9, 31], 3, 1, 128, 128, dict(gate_k=True)),
    "few_fp32": ([25], 8, 8, 128, 128, dict(dtype=F32)),
    "some_k64": ([5, 16, 33, 0, 12], 5, 1, 64, 64, dict(gate_k=True)),
    "some_k128_v64": ([5, 16, 33, 0, 12], 8, 2, 128, 64, {}),
    "some_fp32": ([40, 7], 16, 8, 128, 128, dict(dtype=F32)),
    "more_k64": ([8, 3, 17, 26] * 5, 4, 4, 64, 64, {}),
    "more_gate_k": ([8, 3, 17, 26] * 2, 8, 2, 128, 128, dict(gate_k=True)),
    "one_packed": ([10], 2, 1, 128, 128, dict(packed=True)),
}


@pytest.mark.parametrize("decay_first", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_plain_form(name, decay_first):
    lens, H, Hqk, K, V, opt = CASES[name]
    d = make(lens, H, Hqk, K, V, seed=len(name), **opt)
    n = len(lens)
    # every third sequence fresh; each writes a slot of its own, every fifth none
    slots_in = [-1 if i % 3 == 2 else d["order"][i] for i in range(n)]
    slots_out = [-7 if i % 5 == 4 else d["order"][n + i] if n + i < len(d["order"]) else -1
                 for i in range(n)]
    after, err = call(d, slots_in, slots_out, decay_first=decay_first)
    assert err == (0, 0)
    o_ref, ref = reference(d, slots_in, slots_out, decay_first=decay_first)
    check_o(d, o_ref)
    check_state(d, after, ref, [x for x in slots_out if x >= 0])


@pytest.mark.parametrize("name", ["one_token_one_seq", "ragged", "ragged_large", "gate_k", "long",
                                  "past_the_block_check", "no_tokens_at_all"])
def test_in_place(name):
    lens, H, Hqk, K, V, opt = CASES[name]
    d = make(lens, H, Hqk, K, V, seed=3, **opt)
    slots = d["order"][:len(lens)]
    after, err = call(d, slots, slots)
    assert err == (0, 0)
    o_ref, ref = reference(d, slots, slots)
    check_o(d, o_ref)
    check_state(d, after, ref, slots)


def test_long_sequences_start_first():
    # lengths that the order of long sequences covers: ties, empty ones, more than one warp's worth of them, one far
    # beyond the last bucket; every sequence is run exactly once
    for lens in ([(i * 37) % 61 for i in range(300)], [0] * 40 + [500] + [20] * 200, [12] * 200 + [13] * 100):
        d = make(lens, 3, 1, 64, 64, seed=len(lens), packed=True)
        n = len(lens)
        slots = d["order"][:n]
        after, err = call(d, slots, slots)
        assert err == (0, 0)
        o_ref, ref = reference(d, slots, slots)
        check_o(d, o_ref)
        check_state(d, after, ref, slots)


@pytest.mark.parametrize("name", ["one_token_one_seq", "one_token_batch", "ragged", "ragged_large",
                                  "k64_v128", "gate_k", "no_tokens_at_all", "one_packed"])
def test_state_after_every_token(name):
    lens, H, Hqk, K, V, opt = CASES[name]
    d = make(lens, H, Hqk, K, V, seed=5, **opt)
    n, t = len(lens), sum(lens)
    slots_in = d["order"][:n]
    slots_out = [-1 if i % 4 == 3 else d["order"][n + i] for i in range(t)]
    after, err = call(d, slots_in, slots_out, per_token=True)
    assert err == (0, 0)
    o_ref, ref = reference(d, slots_in, slots_out, per_token=True)
    check_o(d, o_ref)
    check_state(d, after, ref, [x for x in slots_out if x >= 0])


def test_one_slot_for_all_tokens_of_a_sequence_keeps_the_last():
    d = make([4, 3], 2, 1, 128, 128)
    a, b = d["order"][:2]
    slots_out = [a] * 4 + [b] * 3       # the slots they read, too
    after, err = call(d, [a, b], slots_out, per_token=True)
    assert err == (0, 0)
    _, ref = reference(d, [a, b], slots_out, per_token=True)
    check_state(d, after, ref, [a, b])


def test_shared_prefix_and_absent_arrays():
    d = make([2] * 6, 2, 2, 128, 128)
    shared = d["order"][0]
    slots_out = d["order"][1:7]
    after, err = call(d, [shared] * 6, slots_out)   # six sequences read one slot
    assert err == (0, 0)
    o_ref, ref = reference(d, [shared] * 6, slots_out)
    check_o(d, o_ref)
    check_state(d, after, ref, slots_out)
    after, err = call(d, None, None)                # zero states, none kept
    assert err == (0, 0) and torch.equal(after, d["state"])
    check_o(d, reference(d, None, None)[0])
    # without a cache at all
    ws = gdn.alloc_recurrent_workspace(0)
    d["o"].fill_(float("nan"))
    gdn.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], None, None, None, d["o"], ws)
    torch.cuda.synchronize()
    check_o(d, reference(d, None, None)[0])


@pytest.mark.parametrize("n", [4, 600])   # compared by every block; by the claims
@pytest.mark.parametrize("per_token", [False, True])
def test_shared_writes_are_refused(n, per_token):
    d = make([1] * n, 1, 1, 64, 64)
    o = d["order"]
    slots_in = o[:n]
    slots_out = o[n:2 * n]
    slots_out[2] = slots_out[0]         # two sequences write one slot
    slots_out[1] = slots_in[3]          # one writes what another one reads
    after, (code, detail) = call(d, slots_in, slots_out, per_token=per_token)
    assert (code, detail) == (1, 0x43)
    o_ref, _ = reference(d, slots_in, slots_out)
    check_o(d, o_ref)                   # the outputs are whole
    good = list(slots_out)
    for i in (0, 1, 2):
        good[i] = -1
    _, ref = reference(d, slots_in, good, per_token=per_token)
    check_state(d, after, ref, [x for x in good if x >= 0])   # the refused slots as they were


@pytest.mark.parametrize("n", [3, 520])
@pytest.mark.parametrize("per_token", [False, True])
def test_slots_out_of_range_are_refused(n, per_token):
    d = make([1] * n, 1, 1, 64, 64)
    o = d["order"]
    slots_in, slots_out = o[:n], o[n:2 * n]
    bad_out = list(slots_out)
    bad_out[1] = len(o)
    after, err = call(d, slots_in, bad_out, per_token=per_token)
    assert err == (1, 0x42)
    good = list(slots_out)
    good[1] = -1
    o_ref, ref = reference(d, slots_in, good, per_token=per_token)
    check_o(d, o_ref)
    check_state(d, after, ref, [x for x in good if x >= 0])
    # a start past the cache: the sequence is left out
    bad_in = list(slots_in)
    bad_in[2] = 2**31 - 1
    d["o"].fill_(7.0)
    after, err = call(d, bad_in, slots_out, per_token=per_token)
    assert err == (1, 0x42)
    assert (d["o"].reshape(n, -1)[2] == 7.0).all()
    keep = [i for i in range(n) if i != 2]
    check_state(d, after, reference(d, slots_in, slots_out, per_token=per_token)[1],
                [slots_out[i] for i in keep])


@pytest.mark.parametrize("cu", [[1, 4, 9], [0, 5, 4, 9], [0, 4, 8], [0, 4, 10], [0, -3, 9],
                                [0, 2**31 - 1, 9]])
@pytest.mark.parametrize("claims", [False, True])
def test_bad_lengths_write_nothing(cu, claims):
    d = make([3, 6], 2, 1, 128, 128, packed=True)
    d["o"].fill_(7.0)
    d["cu"] = ints(cu)
    n = len(cu) - 1
    slots_out = d["order"][4:13] if claims else d["order"][4:4 + n]
    after, err = call(d, d["order"][:n], slots_out, per_token=claims)
    assert err == (1, 0x41)
    assert (d["o"] == 7.0).all() and torch.equal(after, d["state"])
    # the workspace serves the next call
    d = make([3, 6], 2, 1, 128, 128, packed=True)
    after, err = call(d, None, d["order"][:2])
    assert err == (0, 0)


def test_token_by_token_equals_one_call():
    # one call over 20 tokens (in blocks of eight), and 20 calls of one token in place. The two round in
    # another order; each lies within TOL_F32 of the same 64-bit values (the arithmetic at the top), so
    # they lie within twice that of one another.
    d = make([20] * 3, 4, 2, 128, 128)
    slots = d["order"][:3]
    whole, err = call(d, slots, slots)
    assert err == (0, 0)
    state, ws = d["state"].clone(), gdn.alloc_recurrent_workspace(d["state"].shape[0])
    o = torch.empty_like(d["o"])
    for t in range(20):
        part = {n: d[n][:, t:t + 1].contiguous() for n in ("q", "k", "v", "g", "beta")}
        part.update(o=torch.empty_like(o[:, :1]), cu=None, state=d["state"])
        call(part, slots, slots, ws=ws, state=state)
        o[:, t:t + 1] = part["o"]
    assert rel_err(np64(o), np64(d["o"])) <= 2 * TOL_F32
    assert rel_err(np64(state[slots]), np64(whole[slots])) <= 2 * TOL_F32
    o_ref, ref = reference(d, slots, slots)
    check_state(d, state, ref, slots)
    d["o"] = o
    check_o(d, o_ref)


def test_decay_of_zero_and_poisoned_slots():
    # exp(-inf) = 0 forgets the state; pages that nobody names hold NaN and stay out of every result
    d = make([3, 2], 2, 1, 128, 128)
    d["g"][:, 1] = float("-inf")
    slots = d["order"][:2]
    rest = [i for i in range(d["state"].shape[0]) if i not in slots]
    d["state"][rest] = float("nan")
    state, err = call(d, slots, slots)
    assert err == (0, 0)
    o_ref, ref = reference(d, slots, slots)
    check_o(d, o_ref)
    assert rel_err(np64(state[slots]), ref[slots].numpy()) <= TOL_F32
    # a fresh sequence does not read slot 0 or any other
    d["state"].fill_(float("nan"))
    state, err = call(d, [-1, -1], slots)
    assert err == (0, 0)
    d["state"].zero_()
    o_ref, ref = reference(d, [-1, -1], slots)
    check_o(d, o_ref)
    assert rel_err(np64(state[slots]), ref[slots].numpy()) <= TOL_F32


@pytest.mark.parametrize("claims", [False, True])
def test_captured_and_on_another_stream(claims):
    # two graphs of the same call share a workspace and are replayed in turn, on a side stream
    d = make([4] * 5, 4, 2, 128, 128)
    slots = d["order"][:5]
    out = [x for s in range(5) for x in [slots[s]] * 4] if claims else slots
    eager, _ = call(d, slots, out, per_token=claims)
    want = d["o"].clone()
    state, ws = d["state"].clone(), gdn.alloc_recurrent_workspace(d["state"].shape[0])
    sin, sout = ints(slots), ints(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                gdn.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], state, sin, sout,
                                      d["o"], ws, per_token=claims)
            graphs.append(graph)
        for i in range(4):
            state.copy_(d["state"])
            d["o"].fill_(float("nan"))
            graphs[i % 2].replay()
            side.synchronize()
            assert torch.equal(d["o"], want) and torch.equal(state, eager), i
        assert gdn.gdn_check_device_error(ws) == (0, 0)


def test_slot_numbers_past_31_bits_of_bytes():
    # a page of 128 KiB at slot 70000: its offset is past 2^33 bytes, 2^31 elements
    n, H = 70001, 2
    state = torch.empty((n, H, 128, 128), device="cuda")
    d = make([2], H, 1, 128, 128)
    d["order"] = [0]
    page = d["state"][:1].clone()
    state[n - 1] = page[0]
    ws = gdn.alloc_recurrent_workspace(n)
    after, err = call(d, [n - 1], [n - 2], ws=ws, state=state)
    assert err == (0, 0)
    d["state"] = torch.cat([page, page])
    o_ref, ref = reference(d, [0], [1])
    check_o(d, o_ref)
    assert rel_err(np64(after[n - 2]), ref[1].numpy()) <= TOL_F32
    assert torch.equal(after[n - 1], page[0])


def test_after_the_prompt_in_chunks():
    # a serving step: prompts by the chunked packed forward, whose final states are cache pages, then
    # the next tokens by the recurrent form; against the fp64 oracle over all of the tokens
    lens, more, H = (130, 64, 77), 5, 4
    full = synth.scaled(synth.WORKLOADS["varlen5_h16_t7300"], H=H, T=sum(lens) + 3 * more,
                        seq_lens=tuple(n + more for n in lens))
    x = synth.make_inputs(full)
    cu = synth.cu_seqlens(full)
    names = ("q", "k", "v", "g", "beta")
    tok = {n: torch.from_numpy(x[n]).cuda().to(BF) for n in names}
    prompt = np.concatenate([np.arange(cu[i], cu[i] + n) for i, n in enumerate(lens)])
    tail = np.concatenate([np.arange(cu[i] + n, cu[i + 1]) for i, n in enumerate(lens)])
    a = {n: tok[n][:, prompt].contiguous() for n in names}
    b = {n: tok[n][:, tail].reshape(3, more, *tok[n].shape[2:]).contiguous() for n in names}
    cu_p = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    o_p = torch.empty((1, sum(lens), H, 128), device="cuda")
    pages = torch.full((8, H, 128, 128), float("nan"), device="cuda")
    prob = gdn.problem(a["k"], a["v"], o_p)
    h0 = torch.from_numpy(x["h0"]).cuda() if x["h0"] is not None else None
    gdn.gdn_varlen_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], h0, o_p, pages[2:5], cu_p,
                       gdn.alloc_varlen_workspace(prob, 3), prob=prob)
    o_t = torch.empty((3, more, H, 128), device="cuda")
    ws = gdn.alloc_recurrent_workspace(8)
    slots = ints([2, 3, 4])
    gdn.gdn_recurrent_fwd(b["q"], b["k"], b["v"], b["g"], b["beta"], pages, slots, slots, o_t, ws)
    torch.cuda.synchronize()
    assert gdn.gdn_check_device_error(ws) == (0, 0)
    o_ref, hf_ref = oracle.varlen_recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, x["h0"])
    assert rel_err(np64(o_t).reshape(1, -1, H, 128), o_ref[:, tail]) <= TOL_BF16
    assert rel_err(np64(pages[2:5]), hf_ref) <= TOL_BF16


@pytest.mark.parametrize("gate_k", [False, True])
@pytest.mark.parametrize("lens,H", [([7, 6], 2), ([7, 6, 12], 8), ([15, 14] * 40, 8)])
@pytest.mark.parametrize("bad", [4, 5])   # the first and the second token of a pair
def test_later_tokens_and_other_sequences_do_not_matter(lens, H, gate_k, bad):
    d = make(lens, H, H, 128, 128, seed=11, gate_k=gate_k)
    n = len(lens)
    slots_in, slots_out = d["order"][:n], d["order"][n:2 * n]
    state, err = call(d, slots_in, slots_out)
    o = d["o"].clone()
    for name, value in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("g", float("-inf")),
                        ("beta", float("nan"))):
        d[name].view(-1, *d[name].shape[2:])[bad] = value
    after, err2 = call(d, slots_in, slots_out)
    assert err[0] == 0 and err2[0] == 0
    new, old = (x.view(-1, *x.shape[2:]) for x in (d["o"], o))
    assert torch.equal(new[:bad], old[:bad]) and torch.equal(new[lens[0]:], old[lens[0]:])
    assert new[bad].isnan().any()
    rest = [i for i in range(state.shape[0]) if i != slots_out[0]]
    assert torch.equal(after[rest], state[rest])
