"""The normalisation of the rule's outputs and its gradients against their plain 64-bit forms.

Tolerances, derived (u = 2^-24, half a step of fp32):
 - the sums over a row: a thread adds at most 16 terms, the exchanges join 5 + 4 more levels, so a sum
   is off by at most 25 u of the sum of its terms' sizes. For the variance all terms have one sign: s is off by
   at most 25 u / 2 plus rsqrt's 2 u and the mean's own error (25 u |x|max-scale, folded into 64 u of
   the row's largest |x| s), and y adds a handful of roundings: |y - y64| <= 64 u (|xh|max |w| + |b|) |z sg|,
   which is under 128 u of the row's largest |y| scale; bf16 outputs add half a step, 2^-8 |y|.
 - the sigmoid: expf 2 u, the quotient 4 u, and for z the products: under 16 u |value|.
 - dx: three terms of the row's largest |d w| s, each off by under 64 u (1 + |xh|max): bounded by
   256 u (1 + max|xh|^2) max|d w| s.
 - dw, db: a column's sum joins its terms in chains of at most rows / (threads' rows) + 40 additions:
   for the sizes here at most 400, so 400 u of the sum of the terms' sizes at the very most.
"""
import pytest
import torch

import oracle
import plain64
from context_scan_gb300 import gdn, synth
from gpu_util import record

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def make(rows, n, xt, yt, gated, w=True, b=True, seed=0, mean=0.3):
    gen = torch.Generator().manual_seed(seed + 7 * n + rows)

    def normal(*shape, mu=0.0, sd=1.0):
        return torch.randn(shape, generator=gen) * sd + mu

    return dict(x=normal(rows, n, mu=mean).to(xt), z=normal(rows, n, sd=2.0).to(yt) if gated else None,
                dy=normal(rows, n).to(yt), w=normal(n, mu=1.0, sd=0.3) if w else None,
                b=normal(n, sd=0.3) if b else None)


def cuda(t):
    return None if t is None else t.cuda()


def half(t):
    return torch.finfo(t).eps / 2 if t == BF else 0.0


def check(got, ref, bound, label):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    off = (got - ref).abs() - half(BF if label.endswith("bf16") else F32) * ref.abs() * (1 + 1e-6)
    if off.numel():
        record(float((off / bound.clamp(min=1e-300)).max()), label)
        assert (off <= bound).all(), (label, float((off / bound.clamp(min=1e-300)).max()))


def bounds(d, rms):
    """The row's scales that the tolerances are stated in."""
    x, dy = d["x"].double(), d["dy"].double()
    w = torch.ones(x.shape[-1]).double() if d["w"] is None else d["w"].double()
    b = torch.zeros(x.shape[-1]).double() if d["b"] is None else d["b"].double()
    xm = x if rms else x - x.mean(-1, keepdim=True)
    s = 1 / torch.sqrt((xm * xm).mean(-1, keepdim=True) + EPS)
    # (with a mean, the subtraction is off by the mean's own rounding: u |x|max s)
    top = (x.abs().amax(-1, keepdim=True) * s).clamp(min=1.0)
    y0 = top * w.abs() + b.abs()
    z = None if d["z"] is None else d["z"].double()
    sg = None if z is None else torch.sigmoid(z)
    zs = 1.0 if z is None else (z * sg).abs()
    dd = dy.abs() * zs
    return dict(y=128 * U * y0 * zs + 1e-37,
                dz=None if z is None else 128 * U * y0 * (dy * sg).abs() * (1 + z.abs()) + 1e-37,
                dx=256 * U * (1 + top * top) * (dd * w.abs()).amax(-1, keepdim=True) * s + 1e-37,
                dw=400 * U * (dd * top).sum(0) + 1e-37, db=400 * U * dd.sum(0) + 1e-37)


def run_both(d, rms, xt, yt):
    c = {k: cuda(v) for k, v in d.items()}
    rows, n = d["x"].shape
    y = torch.full((rows, n), float("nan"), dtype=yt, device="cuda")
    gdn.gdn_norm_fwd(c["x"], c["w"], c["b"], c["z"], y, eps=EPS, rms=rms)
    dx = torch.full((rows, n), float("nan"), dtype=xt, device="cuda")
    dz = None if d["z"] is None else torch.full((rows, n), float("nan"), dtype=yt, device="cuda")
    dw, db = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    gdn.gdn_norm_bwd(c["x"], c["w"], c["b"], c["z"], c["dy"], dx, dz, dw, db,
                     gdn.alloc_norm_bwd_workspace(rows, n), eps=EPS, rms=rms)
    torch.cuda.synchronize()
    return y, dx, dz, dw, db


def compare(d, rms, xt, yt):
    y, dx, dz, dw, db = run_both(d, rms, xt, yt)
    lim = bounds(d, rms)
    w, b, z = (None if d[k] is None else d[k].double() for k in ("w", "b", "z"))
    xn, yn = ("bf16" if t == BF else "f32" for t in (xt, yt))
    check(y, plain64.norm(d["x"].double(), w, b, z, rms, EPS), lim["y"], "y " + yn)
    rdx, rdz, rdw, rdb = plain64.norm_grads(d["x"], d["w"], d["b"], d["z"], d["dy"], rms, EPS)
    check(dx, rdx, lim["dx"].expand_as(rdx), "dx " + xn)
    if dz is not None:
        check(dz, rdz, lim["dz"], "dz " + yn)
    check(dw, rdw, lim["dw"], "dw f32")
    check(db, rdb, lim["db"], "db f32")


# every way a row is dealt out: 8 to 32 threads, a block of 64 to 512, two eights a thread; vectors and
# single values; more rows than one round of the grid holds
SIZES = [(1, 1), (5, 2), (3, 7), (9, 8), (33, 40), (700, 64), (257, 100), (1000, 128), (12, 129), (3000, 16),
         (77, 255), (400, 256), (5, 257), (64, 512), (41, 1000), (300, 1999), (700, 2048), (3, 4095),
         (170, 4096), (9, 4097), (400, 5000), (5, 8191), (330, 8192), (12000, 128), (2600, 300), (50, 20), (61, 1996), (40, 1998)]


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,n", SIZES)
def test_fp32_in_bf16_out(rows, n, gated, rms):
    d = make(rows, n, F32, BF, gated)
    compare(d, rms, F32, BF)


@pytest.mark.parametrize("xt,yt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,n", [(37, 128), (65, 96), (20, 131), (33, 1032), (17, 999), (9, 6000), (7, 4999),
                                    (50, 20), (61, 1996), (40, 1998), (400, 2001), (700, 125)])
def test_types(rows, n, xt, yt):
    for gated in (True, False):
        for rms in (True, False):
            compare(make(rows, n, xt, yt, gated, seed=3), rms, xt, yt)


@pytest.mark.parametrize("n", [64, 200, 5120])
@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_absent_parameters(n, w, b):
    for gated in (True, False):
        compare(make(19, n, F32, F32, gated, w=w, b=b), not b, F32, F32)


@pytest.mark.parametrize("n", [128, 130, 2048, 8192])
def test_against_differences(n):
    # the gradient along a random direction is the slope of <y, dy>: in 64 bits the formulas hold to
    # 1e-6, so what the kernel returns is compared with the slope itself
    d = {k: None if v is None else v.double() for k, v in make(4, n, F32, F32, True, seed=9).items()}
    _, dx, dz, dw, db = run_both({k: None if v is None else v.float() for k, v in d.items()}, False, F32, F32)
    got = dict(x=dx, z=dz, w=dw, b=db)
    gen = torch.Generator().manual_seed(1)
    for name, grad in got.items():
        way = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5

        def loss(t):
            a = dict(d)
            a[name] = d[name] + t * way
            return (plain64.norm(a["x"], a["w"], a["b"], a["z"], False, EPS) * d["dy"]).sum()

        slope = float((loss(h) - loss(-h)) / (2 * h))
        mine = float((grad.double().cpu() * way).sum())
        scale = float((grad.double().cpu() * way).abs().sum())
        assert abs(mine - slope) <= 1e-6 * scale, (name, mine, slope)


def test_values_at_the_edge():
    # equal values (variance 0), zeros, a large mean, one spike, gates that saturate; eps = 0 where the row
    # allows it
    n = 256
    x = torch.zeros(6, n)
    x[0] = 3.0
    x[2] = torch.randn(n, generator=torch.Generator().manual_seed(0)) + 1000.0
    x[3, 5] = 1e4
    x[4:] = torch.randn(2, n, generator=torch.Generator().manual_seed(1))
    z = torch.randn(6, n, generator=torch.Generator().manual_seed(2))
    z[4], z[5] = 200.0, -200.0
    d = dict(x=x, z=z, dy=torch.randn(6, n, generator=torch.Generator().manual_seed(3)), w=None, b=None)
    for rms in (True, False):
        compare(d, rms, F32, F32)
    c = {k: cuda(v) for k, v in d.items()}
    y = torch.empty_like(c["x"])
    gdn.gdn_norm_fwd(c["x"][4:].clone(), None, None, None, y[4:].clone(), eps=0.0)
    gdn.gdn_norm_fwd(c["x"], None, None, None, y, eps=0.0, rms=True)
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all()             # 0 / 0, as the formula has it
    assert torch.isfinite(y[[0, 2, 3, 4, 5]]).all()
    # NaN and infinity stay in their row; with eps = 0 and rows that do not fill the grid the sums stay finite
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    gdn.gdn_norm_fwd(x.cuda(), None, None, None, y, eps=EPS)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 3, 4, 5]]).all()
    dx, dw, db = torch.empty(3, 128).cuda(), torch.empty(128).cuda(), torch.empty(128).cuda()
    g = torch.randn(3, 128, generator=torch.Generator().manual_seed(4)).cuda()
    gdn.gdn_norm_bwd(g, None, None, None, g, dx, None, dw, db, gdn.alloc_norm_bwd_workspace(3, 128), eps=0.0)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    gdn.gdn_norm_fwd(e, w, None, None, e.clone())
    dw, db = torch.full((64,), 7.0, device="cuda"), torch.full((64,), 7.0, device="cuda")
    gdn.gdn_norm_bwd(e, w, None, None, e.clone(), e.clone(), None, dw, db, gdn.alloc_norm_bwd_workspace(0, 64))
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("n", [128, 127, 1999, 2048, 6000])
def test_in_place_partial_and_repeated(n):
    d = {k: cuda(v) for k, v in make(900, n, BF, BF, True).items()}
    y, dx, dz, dw, db = run_both({k: v for k, v in make(900, n, BF, BF, True).items()}, True, BF, BF)
    ws = gdn.alloc_norm_bwd_workspace(900, n)
    # each output by itself, the others skipped; twice the same bits
    for keep in ("dx", "dz", "dw", "db"):
        out = dict(dx=torch.empty_like(d["x"]), dz=None, dw=None, db=None)
        if keep != "dx":
            out[keep] = torch.empty_like(dict(dz=dz, dw=dw, db=db)[keep])
        gdn.gdn_norm_bwd(d["x"], d["w"], d["b"], d["z"], d["dy"], out["dx"], out["dz"], out["dw"], out["db"],
                         ws, eps=EPS)
        torch.cuda.synchronize()
        assert torch.equal(out["dx"], dx)
        assert torch.equal(out[keep], dict(dx=dx, dz=dz, dw=dw, db=db)[keep])
    # on top of the inputs
    a, z = d["x"].clone(), d["z"].clone()
    gdn.gdn_norm_bwd(a, d["w"], d["b"], z, d["dy"], a, z, None, None, ws, eps=EPS)
    assert torch.equal(a, dx) and torch.equal(z, dz)
    for target in ("x", "z"):
        a = {k: d[k].clone() for k in ("x", "z")}
        gdn.gdn_norm_fwd(a["x"], d["w"], d["b"], a["z"], a[target], eps=EPS)
        assert torch.equal(a[target], y)


def test_captured_and_on_another_stream():
    d = {k: cuda(v) for k, v in make(500, 128, F32, BF, True).items()}
    want = run_both(make(500, 128, F32, BF, True), True, F32, BF)
    out = [torch.empty_like(t) for t in want]
    ws = gdn.alloc_norm_bwd_workspace(500, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                gdn.gdn_norm_fwd(d["x"], d["w"], d["b"], d["z"], out[0], eps=EPS)
                gdn.gdn_norm_bwd(d["x"], d["w"], d["b"], d["z"], d["dy"], *out[1:], ws, eps=EPS)
            graphs.append(graph)
        for i in range(4):
            for t in out:
                t.fill_(float("nan"))
            graphs[i % 2].replay()
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_rows_past_31_bits():
    # more than 2^31 values: the last rows come out as they do alone
    rows, n = 17_000_001, 128
    x = torch.ones((rows, n), dtype=BF, device="cuda")
    x[-3:] = torch.randn(3, n, generator=torch.Generator().manual_seed(0)).to(BF).cuda()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_norm_fwd(x, None, None, None, y, eps=EPS)
    y3, dx3 = torch.empty_like(x[-3:]), torch.empty_like(x[-3:])
    gdn.gdn_norm_fwd(x[-3:].clone(), None, None, None, y3, eps=EPS)
    assert torch.equal(y[-3:], y3)
    db = torch.empty(n, device="cuda")
    gdn.gdn_norm_bwd(x, None, None, None, x, dx, None, None, db, gdn.alloc_norm_bwd_workspace(rows, n), eps=EPS)
    gdn.gdn_norm_bwd(x[-3:].clone(), None, None, None, x[-3:].clone(), dx3, None, None, None,
                     gdn.alloc_norm_bwd_workspace(3, n), eps=EPS)
    assert torch.equal(dx[-3:], dx3)
    assert ((db - rows).abs() <= 400 * U * rows + 20).all()


def test_training_step_through_the_rule():
    # forward of the rule, gated norm, a loss; the norm's dx is the dO of the rule's backward. Against the
    # fp64 oracle's backward fed with the plain norm's gradient of the oracle's own outputs.
    w0 = synth.scaled(synth.WORKLOADS["tiny_f32_k64_cp4"], B=2, H=2, T=256)
    x = synth.make_inputs(w0)
    names = ("q", "k", "v", "g", "beta")
    t = {n: torch.from_numpy(x[n]).cuda() for n in names}
    B, T, H, V = x["v"].shape
    K = x["k"].shape[-1]
    h0 = torch.from_numpy(x["h0"]).cuda()
    o = torch.empty((B, T, H, V), device="cuda")
    prob = gdn.problem(t["k"], t["v"], o)
    gdn.gdn_segmented_fwd(*(t[n] for n in names), h0, o, None, 4, gdn.alloc_workspace(prob, 4), prob=prob)
    gen = torch.Generator().manual_seed(0)
    z, dy = (torch.randn((B, T, H, V), generator=gen) for _ in range(2))
    weight = torch.rand(V, generator=gen) + 0.5
    y, dO, dz = torch.empty_like(o), torch.empty_like(o), torch.empty_like(o)
    dw = torch.empty(V, device="cuda")
    gdn.gdn_norm_fwd(o, weight.cuda(), None, z.cuda(), y, eps=EPS)
    gdn.gdn_norm_bwd(o, weight.cuda(), None, z.cuda(), dy.cuda(), dO, dz, dw, None,
                     gdn.alloc_norm_bwd_workspace(B * T * H, V), eps=EPS)
    grads = [torch.empty_like(t[n]) for n in names] + [torch.empty_like(h0)]
    gdn.gdn_chunk_bwd(*(t[n] for n in names), h0, dO, None, *grads, 4, gdn.alloc_bwd_workspace(prob, 4), prob=prob)
    torch.cuda.synchronize()
    o_ref, _, _ = oracle.recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], x["h0"])
    o64 = torch.from_numpy(o_ref).double().reshape(-1, V)
    dO64, dz64, dw64, _ = plain64.norm_grads(o64, weight, None, z.reshape(-1, V), dy.reshape(-1, V), True, EPS)
    ref = oracle.backward(x["q"], x["k"], x["v"], x["g"], x["beta"],
                          dO64.reshape(B, T, H, V).numpy(), x["h0"], None)
    # fp32 throughout: the library's bar of 1e-4 of the RMS for o grows by the norm's slope, s = 1/rms(o_row), on
    # rows whose outputs are small against the others: 10 times is allowed for the parts
    for got, want in zip(grads, ref):
        want = torch.as_tensor(want).double()
        off = (got.double().cpu() - want).abs().max() / want.square().mean().sqrt()
        assert float(record(float(off), "grad")) <= 1e-3
    for got, want in ((dz, dz64), (dw, dw64)):
        want = want.reshape(got.shape)
        assert float((got.double().cpu() - want).abs().max() / want.square().mean().sqrt()) <= 1e-3
