"""GPU parity of the recurrent linear attention over a state cache (gdn_linear_recurrent_fwd) against its plain 64-bit form.

Tolerance, derived: a state's term passes one rounding a token, an output's at most K / 4 + 6 more in its sum over the rows:
with n tokens (K / 4 + 6 + 2 n) 2^-24 of the same form on absolute values; a bf16 output adds half a step, 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

import plain64_linear as plain
from context_scan_gb300 import gdn
from gpu_util import record
from test_gpu_linear import slopes

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def make(lens, H, Hqk, K, V, dtype=BF, out=BF, packed=None, pad=0, decay=None, seed=0):
    gen = torch.Generator().manual_seed(500 + seed)
    n, nseq = sum(lens), len(lens)
    if packed is None:
        packed = len(set(lens)) > 1
    lead = (1, n + pad) if packed else (nseq, lens[0])
    normal = lambda *s, sd=1.0: torch.randn(*s, generator=gen) * sd  # noqa: E731
    unit = torch.nn.functional.normalize
    d = {"q": unit(normal(*lead, Hqk, K), dim=-1).to(dtype).cuda(), "k": unit(normal(*lead, Hqk, K), dim=-1).to(dtype).cuda(),
         "v": normal(*lead, H, V).to(dtype).cuda()}
    d["decay"] = (slopes(H, gen) if decay is None else torch.tensor(decay, dtype=F32)).cuda()
    slots = nseq + n + 3
    d["state"] = normal(slots, H, K, V, sd=0.3).cuda()
    d["order"] = torch.randperm(slots, generator=gen).tolist()
    d["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda() if packed else None
    d["o"] = torch.full((*lead, H, V), float("nan"), dtype=out, device="cuda")
    d["lens"], d["n"] = list(lens), n
    return d


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32).cuda()


def call(d, slots_in, slots_out, per_token=False, ws=None):
    state = d["state"].clone()
    ws = gdn.alloc_recurrent_workspace(state.shape[0]) if ws is None else ws
    gdn.gdn_linear_recurrent_fwd(d["q"], d["k"], d["v"], d["decay"], state, ints(slots_in), ints(slots_out), d["o"], ws,
                                 cu_seqlens=d["cu"], per_token=per_token)
    torch.cuda.synchronize()
    return state, gdn.gdn_check_device_error(ws)


def form(d, slots_in, absolute=False):
    f = (lambda x: x.abs()) if absolute else (lambda x: x)
    h0 = torch.stack([f(d["state"][s]) if s >= 0 else torch.zeros_like(d["state"][0]) for s in slots_in])
    q, k, v = (f(d[n]).reshape(-1, *d[n].shape[2:])[:d["n"]] for n in ("q", "k", "v"))
    keep = []
    o, h = plain.forward(q, k, v, d["decay"], h0, d["lens"], keep)
    return o, h, keep


def check(d, got_o, state, slots_in, slots_out, per_token):
    o, h, keep = form(d, slots_in)
    oa, ha, keepa = form(d, slots_in, True)
    K, n = d["k"].shape[3], max(d["lens"] + [0])
    step = 2.0 ** -24
    if o.numel():
        got = got_o.double().cpu().reshape(-1, *got_o.shape[2:])[:d["n"]]
        tol = (K / 4 + 6 + 2 * n) * step * oa + (2.0 ** -8 if d["o"].dtype == BF else 2.0 ** -24) * o.abs() + 1e-30
        record(float(((got - o).abs() / tol).max()), "o")
        assert ((got - o).abs() <= tol).all()
    states, bounds = (keep, keepa) if per_token else (list(h), list(ha))
    written = set()
    for i, slot in enumerate(slots_out[:len(states)]):
        if slot >= 0:
            written.add(slot)
            last = max(j for j, x in enumerate(slots_out[:len(states)]) if x == slot)
            assert ((state[slot].double().cpu() - states[last]).abs() <= (2 * n + 1) * step * bounds[last] + 1e-30).all()
    rest = [i for i in range(state.shape[0]) if i not in written]
    assert torch.equal(state[rest], d["state"][rest])


CASES = {
    "one": ([1], 4, 2, 128, 128, {}),
    "batch": ([1] * 7, 4, 4, 128, 128, dict(out=F32)),
    "large_batch": ([1] * 340, 4, 1, 128, 128, {}),
    "past_the_block_check": ([1] * 515, 1, 1, 64, 64, {}),
    "ragged": ([3, 0, 17, 1, 8, 9, 0], 6, 2, 128, 128, dict(out=F32)),
    "ragged_large": ([(i * 5) % 11 for i in range(330)], 4, 2, 128, 128, {}),
    "tails_large": ([(i * 29) % 64 for i in range(60)], 8, 4, 128, 128, {}),
    "long": ([200, 63, 65], 2, 1, 128, 128, dict(out=F32)),
    "long_even": ([100, 100], 3, 3, 128, 64, {}),
    "k64": ([5, 16, 33], 3, 3, 64, 64, {}),
    "k64_v128": ([5, 0, 8], 3, 1, 64, 128, {}),
    "k64_large": ([(i * 5) % 14 for i in range(700)], 4, 4, 64, 64, {}),
    "k64_v128_large": ([(i * 5) % 14 for i in range(400)], 4, 4, 64, 128, {}),
    "k128_v64_large": ([(i * 5) % 14 for i in range(400)], 8, 4, 128, 64, {}),
    "fp32": ([4, 11, 64], 3, 3, 128, 128, dict(dtype=F32, out=F32)),
    "fp32_bf16_out": ([4, 11, 70], 5, 5, 64, 64, dict(dtype=F32)),
    "fp32_large": ([20] * 100, 4, 4, 128, 128, dict(dtype=F32, out=F32)),
    "padded": ([9, 0, 20], 2, 2, 128, 128, dict(pad=13)),
    "strong": ([40, 3], 4, 4, 128, 128, dict(out=F32, decay=[0.0, -30.0, -1e30, float("-inf")])),
}


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_against_the_plain_form(name, per_token):
    lens, H, Hqk, K, V, kw = CASES[name]
    if per_token and sum(lens) * H * K * V > 3e8:
        pytest.skip("a cache of many GB")
    d = make(lens, H, Hqk, K, V, **kw)
    nseq, n, order = len(lens), sum(lens), d["order"]
    slots_in = [-1 if i % 4 == 3 else order[i] for i in range(nseq)]
    rows = d["q"].shape[0] * d["q"].shape[1]
    outs = order[nseq:nseq + (n if per_token else nseq)] + [order[nseq]] * (rows - n if per_token else 0)
    state, (st, _) = call(d, slots_in, outs, per_token)
    assert st == 0
    check(d, d["o"], state, slots_in, outs, per_token)
    if d["n"] < rows:
        assert torch.isnan(d["o"][:, d["n"]:]).all()


def test_in_place_and_without_slots():
    d = make([5, 1, 12], 4, 2, 128, 128)
    slots = d["order"][:3]
    state, (st, _) = call(d, slots, slots)
    assert st == 0
    check(d, d["o"], state, slots, slots, False)
    state, (st, _) = call(d, None, None)
    assert st == 0 and torch.equal(state, d["state"])
    check(d, d["o"], state, [-1, -1, -1], [-1, -1, -1], False)


def test_refusals_on_the_device():
    d = make([5, 1, 12], 2, 2, 64, 64)
    a, b, c, e = d["order"][:4]
    # two sequences write one slot: neither does, the third is whole
    state, (st, detail) = call(d, [a, b, c], [e, e, c])
    assert st == 1 and detail == 0x43 and torch.equal(state[e], d["state"][e]) and not torch.equal(state[c], d["state"][c])
    big = d["state"].shape[0]
    d["o"].fill_(float("nan"))
    state, (st, detail) = call(d, [a, big, c], [-1, -1, big + 7])
    assert st == 1 and detail == 0x42 and torch.isnan(d["o"][0, 5]).all() and torch.isfinite(d["o"][0, 6:]).all()
    for cu in ([1, 5, 6, 18], [0, 6, 5, 18], [0, 5, 6, 19], [0, 5, 6, -2]):
        d["cu"], d["o"] = ints(cu), torch.full_like(d["o"], float("nan"))
        state, (st, detail) = call(d, [a, b, c], [a, b, c])
        assert st == 1 and detail == 0x41 and torch.isnan(d["o"]).all() and torch.equal(state, d["state"])


def test_continues_the_chunked_form():
    # a prompt through the chunked form, its state into a page of the cache, three tokens from there
    d = make([503], 4, 2, 128, 128, out=F32)
    ht = torch.empty(1, 4, 128, 128, device="cuda")
    part = lambda a, b: [d[n][:, a:b].contiguous() for n in ("q", "k", "v")]  # noqa: E731
    q, k, v = part(0, 500)
    o = torch.empty_like(v)
    gdn.gdn_linear_fwd(q, k, v, d["decay"], None, o, ht, gdn.alloc_linear_workspace(k, v))
    cache = d["state"]
    page = d["order"][0]
    cache[page] = ht[0]
    q, k, v = part(500, 503)
    o = torch.empty_like(v, dtype=F32)
    ws = gdn.alloc_recurrent_workspace(cache.shape[0])
    gdn.gdn_linear_recurrent_fwd(q, k, v, d["decay"], cache, ints([page]), ints([page]), o, ws)
    ref, h, _ = form({**d, "state": torch.zeros_like(cache)}, [-1])
    bound, hb, _ = form({**d, "state": torch.zeros_like(cache)}, [-1], True)
    term = 2.0 ** -17 + 700 * 2.0 ** -24    # the chunked form's state, then the recurrent form's sums
    assert ((o[0].double().cpu() - ref[500:]).abs() <= term * bound[500:]).all()
    assert ((cache[page].double().cpu() - h[0]).abs() <= term * hb[0]).all()
