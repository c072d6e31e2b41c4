"""The operators of a serving loop together: prompts by the chunked packed forward into cache pages, new tokens by the
recurrent form, every output through the gated norm, sequences forked, ended and compacted in between; the
same in 64 bits beside it. And the calls that the binding refuses.

Tolerances: the first states come from bf16 prompts run on the tensor cores (TOL_BF16, as the parity tests have it for
h_final); the plain loop starts from the states that the device holds after the prompts, so that everything
behind them is held to the fp32 bar of the recurrent form, 1e-4 of the RMS. The norm of a row divides its
error by the row's own RMS, which for these outputs is at least a twentieth of the whole's: 20 times that for y.
"""
import numpy as np
import pytest
import torch

import oracle
import plain64
from context_scan_gb300 import gdn, synth
from gpu_util import TOL_BF16, TOL_F32, np64, rel_err

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def tokens(gen, n, t, H, K):
    unit = torch.nn.functional.normalize
    d = {"q": unit(torch.randn(n, t, H, K, generator=gen), dim=-1),
         "k": unit(torch.randn(n, t, H, K, generator=gen), dim=-1),
         "v": torch.randn(n, t, H, K, generator=gen),
         "g": torch.nn.functional.logsigmoid(torch.randn(n, t, H, generator=gen) + 2.0),
         "beta": torch.sigmoid(torch.randn(n, t, H, generator=gen))}
    return {name: x.to(BF) for name, x in d.items()}


def test_prompts_decode_fork_end_compact():
    L, PAGES, H, K = 2, 9, 4, 128
    lens = (70, 130, 64)
    gen = torch.Generator().manual_seed(11)
    pages = torch.full((L, PAGES, H, K, K), float("nan"), device="cuda")
    refs = ints([0] * PAGES)
    ws = gdn.alloc_recurrent_workspace(PAGES)
    wc = gdn.alloc_cache_workspace(PAGES, 4)
    w = torch.rand(K, generator=gen) + 0.5

    # three pages of zeros for the three prompts, then the prompts' states into them
    table = ints([0, 0, 0])
    gdn.gdn_cache_fork(pages, refs, ints([-1, -1, -1]), table, wc)
    torch.cuda.synchronize()
    assert table.tolist() == [0, 1, 2] and not pages[:, :3].any() and torch.isnan(pages[:, 3:]).all()
    wl = synth.scaled(synth.WORKLOADS["varlen5_h16_t7300"], H=H, T=sum(lens), seq_lens=lens)
    cu = synth.cu_seqlens(wl)
    for layer in range(L):
        x = synth.make_inputs(synth.scaled(wl, seed=wl.seed + layer))
        t = {n: torch.from_numpy(x[n]).cuda().to(BF) for n in ("q", "k", "v", "g", "beta")}
        o = torch.empty((1, wl.T, H, K), device="cuda")
        prob = gdn.problem(t["k"], t["v"], o)
        h0 = None if x["h0"] is None else torch.from_numpy(x["h0"]).cuda()
        gdn.gdn_varlen_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], h0, o, pages[layer, :3],
                           torch.from_numpy(cu).cuda(), gdn.alloc_varlen_workspace(prob, 3), prob=prob)
        torch.cuda.synchronize()
        _, hf = oracle.varlen_recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, x["h0"])
        assert rel_err(np64(pages[layer, :3]), hf) <= TOL_BF16
    plain = pages.double().cpu()        # the plain loop goes on from here, page by page
    refs64, table64 = refs.tolist(), table.tolist()

    def step(n_tokens):
        """n_tokens more of every sequence in the table, in every layer, and the norm of the outputs."""
        n = len(table64)
        for layer in range(L):
            d = tokens(gen, n, n_tokens, H, K)
            z = torch.randn(n, n_tokens, H, K, generator=gen).to(BF)
            c = {name: x.cuda() for name, x in d.items()}
            o = torch.empty((n, n_tokens, H, K), device="cuda")
            y = torch.empty((n, n_tokens, H, K), dtype=BF, device="cuda")
            gdn.gdn_recurrent_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], pages[layer], table, table, o, ws)
            gdn.gdn_norm_fwd(o, w.cuda(), None, z.cuda(), y, eps=EPS)
            torch.cuda.synchronize()
            flat = [d[name].flatten(0, 1) for name in ("q", "k", "v", "g", "beta")]
            o64, plain[layer] = plain64.recurrence(*flat, plain[layer], table64, table64, [n_tokens] * n)
            assert rel_err(np64(o).reshape(o64.shape), o64.numpy()) <= TOL_F32
            y64 = plain64.norm(o64, w.double(), None, z.double().reshape(o64.shape), True, EPS)
            off = (y.double().cpu().reshape(y64.shape) - y64).abs() - torch.finfo(BF).eps / 2 * y64.abs()
            assert float(off.max() / y64.square().mean().sqrt()) <= 20 * TOL_F32

    def same():
        used = [p for p, r in enumerate(refs64) if r > 0]
        assert refs.tolist() == refs64 and table.tolist() == table64
        assert rel_err(np64(pages[:, used]), plain[:, used].numpy()) <= TOL_F32

    step(1)
    step(3)
    same()
    # sequence 1 forks in two, sequence 2 in one more: pages 3, 4, 5
    kids = ints([0, 0, 0])
    parents = [table64[1], table64[1], table64[2]]
    gdn.gdn_cache_fork(pages, refs, ints(parents), kids, wc)
    plain, refs64, kids64, code = plain64.cache_fork(plain, refs64, parents)
    assert code == 0 and kids.tolist() == kids64 == [3, 4, 5]
    table, table64 = torch.cat([table, kids]), table64 + kids64
    step(2)
    same()
    # sequences 0 and 3 end, the rest move to the front
    ended = [table64[0], table64[3]]
    gdn.gdn_cache_free(refs, ints(ended), wc)
    table, table64 = table[[1, 2, 4, 5]].contiguous(), [table64[i] for i in (1, 2, 4, 5)]
    for p in ended:
        refs64[p] -= 1
    live = ints([0])
    gdn.gdn_cache_compact(pages, refs, table, None, live, wc)
    plain, refs64, table64, _, live64 = plain64.cache_compact(plain, refs64, table64)
    assert live.item() == live64 == 4
    same()
    step(1)
    same()
    # draft tokens: the state after each in a page of its own, then the one behind the accepted ones copied over
    seq, keep = table64[0], 2
    drafts = ints([0, 0, 0])
    gdn.gdn_cache_fork(pages, refs, ints([-1, -1, -1]), drafts, wc)
    for layer in range(L):
        d = tokens(gen, 1, 3, H, K)
        c = {name: x.cuda() for name, x in d.items()}
        o = torch.empty((1, 3, H, K), device="cuda")
        gdn.gdn_recurrent_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], pages[layer], ints([seq]), drafts, o, ws,
                              per_token=True)
        flat = [d[name].flatten(0, 1)[:keep] for name in ("q", "k", "v", "g", "beta")]
        _, plain[layer] = plain64.recurrence(*flat, plain[layer], [seq], [seq], [keep])
    gdn.gdn_cache_copy(pages, drafts[keep - 1:keep], ints([seq]), wc)
    gdn.gdn_cache_free(refs, drafts, wc)
    same()
    assert gdn.gdn_check_device_error(ws) == (0, 0) and gdn.gdn_check_device_error(wc) == (0, 0)


def test_two_streams_at_once():
    # two decode batches on two streams, on disjoint pages of one cache, each with its own workspace
    gen = torch.Generator().manual_seed(5)
    n, H, K = 64, 4, 128
    state = torch.randn(2 * n, H, K, K, generator=gen)
    both = state.cuda()
    parts = []
    for i in range(2):
        d = tokens(gen, n, 4, H, K)
        parts.append(dict(d=d, c={name: x.cuda() for name, x in d.items()}, s=torch.cuda.Stream(),
                          slots=ints(list(range(i, 2 * n, 2))), o=torch.empty((n, 4, H, K), device="cuda"),
                          ws=gdn.alloc_recurrent_workspace(2 * n)))
    torch.cuda.synchronize()
    for _ in range(3):
        for p in parts:
            c = p["c"]
            gdn.gdn_recurrent_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], both, p["slots"], p["slots"], p["o"],
                                  p["ws"], stream=p["s"])
    torch.cuda.synchronize()
    ref = state
    for p in parts:
        flat = [p["d"][name].flatten(0, 1) for name in ("q", "k", "v", "g", "beta")]
        slots = p["slots"].tolist()
        for _ in range(3):
            o64, ref = plain64.recurrence(*flat, ref, slots, slots, [4] * n)
        assert rel_err(np64(p["o"]).reshape(o64.shape), o64.numpy()) <= TOL_F32
        assert gdn.gdn_check_device_error(p["ws"]) == (0, 0)
    assert rel_err(np64(both), ref.numpy()) <= TOL_F32


def test_binding_refusals():
    q, v = torch.zeros(2, 3, 1, 64, device="cuda", dtype=BF), torch.zeros(2, 3, 2, 64, device="cuda", dtype=BF)
    g = torch.zeros(2, 3, 2, device="cuda", dtype=BF)
    state, slots = torch.zeros(5, 2, 64, 64, device="cuda"), ints([0, 1])
    o, ws = torch.full_like(v, 7.0), gdn.alloc_recurrent_workspace(5)

    def call(**kw):
        a = dict(q=q, k=q, v=v, g=g, beta=g, state=state, slots_in=slots, slots_out=slots, o=o, workspace=ws)
        a.update(kw)
        gdn.gdn_recurrent_fwd(**a)

    wide = torch.zeros(2, 3, 2, 64, device="cuda", dtype=BF)
    for kw, why in [
        (dict(q=wide[:, :, :1]), "not contiguous"), (dict(v=v.transpose(0, 1)), "not contiguous"),
        (dict(k=q.cpu()), "is on cpu"), (dict(q=q.float()), "q is torch.float32"),
        (dict(q=q[:1]), "q is"), (dict(beta=g[:, :2].contiguous()), "beta is"),
        (dict(g=torch.zeros(2, 3, 2, 32, device="cuda", dtype=BF)), "g is"),
        (dict(state=state[:, :1].contiguous()), "state is"), (dict(state=state.to(BF)), "state is"),
        (dict(slots_in=slots.long()), "slots_in is"), (dict(slots_out=slots[:1]), "slots_out is"),
        (dict(per_token=True), "slots_out is"), (dict(o=o[:1]), "o is"),
        (dict(cu_seqlens=ints([0, 3])), "slots_in is"), (dict(cu_seqlens=torch.zeros(3, device="cuda")), "cu_seqlens is"),
    ]:
        with pytest.raises(ValueError, match=why):
            call(**kw)
    for kw, status in [(dict(workspace=ws[:256]), 5), (dict(o=o.half()), 3), (dict(cu_seqlens=ints([0, 3, 6])), 1)]:
        with pytest.raises(gdn.GdnError) as e:
            call(**kw)
        assert e.value.status == status
    pages = torch.zeros(1, 4, 16, device="cuda")
    idx, wc = ints([0]), gdn.alloc_cache_workspace(4, 1)
    for bad in (lambda: gdn.gdn_cache_copy(pages, idx.long(), idx, wc),
                lambda: gdn.gdn_cache_copy(pages, idx, ints([0, 1]), wc),
                lambda: gdn.gdn_cache_copy(pages[0], idx, idx, wc),
                lambda: gdn.gdn_cache_fork(pages, idx, idx, idx, wc),
                lambda: gdn.gdn_cache_fork(pages, ints([0] * 4), idx, ints([0, 1]), wc),
                lambda: gdn.gdn_cache_compact(pages, ints([0] * 4), idx, idx, None, wc),
                lambda: gdn.gdn_cache_compact(pages[:, ::2], ints([0] * 2), idx, None, None, wc)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_cache_copy(pages, ints([0, 1, 2] * 64), ints([-1] * 192), wc)   # more pairs than the workspace holds
    assert e.value.status == 5
    x, w = torch.zeros(3, 64, device="cuda"), torch.zeros(64, device="cuda")
    for bad in (lambda: gdn.gdn_norm_fwd(x, w[:32], None, None, x.clone()),
                lambda: gdn.gdn_norm_fwd(x, w.to(BF), None, None, x.clone()),
                lambda: gdn.gdn_norm_fwd(x, w, None, x.to(BF), x.clone()),
                lambda: gdn.gdn_norm_fwd(x, w, None, None, x[:2]),
                lambda: gdn.gdn_norm_fwd(x.t(), None, None, None, x.t()),
                lambda: gdn.gdn_norm_bwd(x, w, None, None, x, x.to(BF), None, w, None, wc)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_norm_fwd(x, w, None, None, x.half())
    assert e.value.status == 3
    torch.cuda.synchronize()
    assert (o == 7.0).all()
