"""Layer norm of rows whose mean is large against their spread, down to rows of one value: the second
exchange over a row, for every group of threads, in both directions.

Tolerances, derived (u = 2^-24; s = 1 / sqrt(var + eps); X = max|x| s, C = max|x - m| s; a row's sum
joins at most 16 + 9 terms in a chain, with its share of 1 / N off by at most 27 u of the mean size):
 - a mean formed first is off by at most 30 u max|x|; the values less that mean are exact to u, and
   their own mean, which is then taken off, is off by 27 u of their size: x - m is off by at most
   28 u (C + 30 u X) / s.
 - a row whose mean lies within two standard deviations goes without: its mean is off by 30 u 2.3 / s, its
   variance by 27 u (1 + 4) of itself, so s by 68 u.
   Either way |xh - xh64| <= 128 u (1 + C + 30 u X), and y adds a handful of roundings of xh w + b.
 - the gate: z sigmoid(z) to 16 u (1 + |z|) of itself.
 - dx = s (d w - mean(d w) - xh mean(d w xh)): with D = max|d w| of the row, the first two are off by
   30 u D, mean(d w xh) by 120 u D and twice s's 68 u, and xh by the above: 400 u (1 + C + 30 u X) D s.
   That is linear in C: for the rows here under 1/500 of the row's largest |dx|, which is checked.
 - dw, db: at most 64 additions in a chain for these rows, and xh's error: 256 u.
A bf16 output adds half a step, 2^-8 of the value."""
import pytest
import torch

import plain64
from context_scan_gb300 import gdn
from test_gpu_norm import BF, EPS, F32, U, _lib, cuda, half, run_both  # noqa: F401
from gpu_util import record

pytestmark = pytest.mark.gpu


def rows_of(n, xt, seed):
    """Rows with means of 0 to 3000 standard deviations and rows of one value, mixed."""
    gen = torch.Generator().manual_seed(seed + n)
    base = torch.randn(21, n, generator=gen)
    means = [0.0, 3.0, 0.3, 10.0, -30.0, 1.0, 3.0, -3.0, 30.0, 0.0, 300.0, 2.5, 1.5, -1000.0, 3000.0]
    x = base[:len(means)] + torch.tensor(means)[:, None]
    constant = torch.tensor([100.0, 1000.0, -3.0, 0.1, 0.0, 7.7])[:, None].expand(6, n)
    x = torch.cat([x, constant])[torch.randperm(21, generator=gen)]
    return x.to(xt), gen


def make(n, xt, yt, gated, seed=0):
    x, gen = rows_of(n, xt, seed)
    rows = x.shape[0]
    return dict(x=x, z=(2 * torch.randn(rows, n, generator=gen)).to(yt) if gated else None,
                dy=torch.randn(rows, n, generator=gen).to(yt), w=1 + 0.3 * torch.randn(n, generator=gen),
                b=0.3 * torch.randn(n, generator=gen))


def limits(d):
    x, dy, w, b = (d[k].double() for k in ("x", "dy", "w", "b"))
    m = x.mean(-1, keepdim=True)
    s = 1 / torch.sqrt((x - m).square().mean(-1, keepdim=True) + EPS)
    one_c = 1 + (x - m).abs().amax(-1, keepdim=True) * s + 30 * U * x.abs().amax(-1, keepdim=True) * s
    z = None if d["z"] is None else d["z"].double()
    sg = 1.0 if z is None else torch.sigmoid(z)
    zs, zz = (1.0, 0.0) if z is None else ((z * sg).abs(), z.abs())
    dd = dy.abs() * zs
    dmax = (dd * w.abs()).amax(-1, keepdim=True)
    y = 128 * U * one_c * w.abs() + 4 * U * b.abs()
    gate = 16 * U * (1 + zz)
    big = one_c * w.abs() + b.abs()
    return dict(y=(y + gate * big) * zs + 1e-37, dz=None if z is None else (y + gate * big) * (dy * sg).abs() * (1 + zz) + 1e-37,
                dx=(400 * U * one_c + gate.amax(-1, keepdim=True) if z is not None else 400 * U * one_c) * dmax * s + 1e-37,
                dw=256 * U * (dd * one_c).sum(0) + (gate * dd * one_c).sum(0) + 1e-37,
                db=256 * U * dd.sum(0) + (gate * dd).sum(0) + 1e-37)


def near(got, ref, bound, t, label):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), label
    off = ((got - ref).abs() - half(t) * ref.abs() * (1 + 1e-6)) / bound
    record(float(off.max()), label)
    assert (off <= 1).all(), (label, float(off.max()))


SIZES = [3, 60, 100, 127, 129, 200, 256, 257, 300, 511, 999, 1000, 1024, 1999, 2000, 2048, 4095, 4097, 5000, 8191, 8192]


@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)])
def test_large_means(n, gated, xt, yt):
    d = make(n, xt, yt, gated)
    y, dx, dz, dw, db = run_both(d, False, xt, yt)
    lim = limits(d)
    z = None if d["z"] is None else d["z"].double()
    near(y, plain64.norm(d["x"].double(), d["w"].double(), d["b"].double(), z, False, EPS), lim["y"], yt, "y")
    rdx, rdz, rdw, rdb = plain64.norm_grads(d["x"], d["w"], d["b"], d["z"], d["dy"], False, EPS)
    if n >= 60:   # (a row of few values can have a dx far below the terms it is the sum of)
        assert (lim["dx"] <= rdx.abs().amax(-1, keepdim=True) / 500).all()
    near(dx, rdx, lim["dx"], xt, "dx")
    if gated:
        near(dz, rdz, lim["dz"], yt, "dz")
    near(dw, rdw, lim["dw"], F32, "dw")
    near(db, rdb, lim["db"], F32, "db")


@pytest.mark.parametrize("n", [127, 300, 1000, 1999, 2000, 5000, 8191])
@pytest.mark.parametrize("value", [100.0, 1000.0, 0.1, -77.7, 3e4])
def test_rows_of_one_value_come_out_as_zeros(n, value):
    # x - m = 0: nothing but the mean's own error can show, which 1 / sqrt(eps) = 1000 brings out. The first mean is
    # off by d <= 30 u |value|; all values less it are the same d, whose mean is off by 27 u of it. (The variance is then
    # off by 27 u d^2, and s by 14 u d^2 / eps of itself.)
    x = torch.full((5, n), value, device="cuda")
    y = torch.full_like(x, float("nan"))
    gdn.gdn_norm_fwd(x, None, None, None, y, eps=EPS, rms=False)
    assert float(y.abs().max()) <= 27 * U * 30 * U * abs(value) * 1000 + U
    # the gradients: dx = (dy - mean(dy)) / sqrt(eps), dw = 0
    dy = torch.randn(5, n, generator=torch.Generator().manual_seed(n)).cuda()
    dx, dw, db = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    gdn.gdn_norm_bwd(x, None, None, None, dy, dx, None, dw, db, gdn.alloc_norm_bwd_workspace(5, n), eps=EPS, rms=False)
    want = 1000 * (dy.double() - dy.double().mean(-1, keepdim=True))
    off_s = 14 * U * (30 * U * value) ** 2 / EPS
    assert float((dx.double() - want).abs().max()) <= (64 * U + off_s) * 1000 * float(dy.abs().max())
    assert float(dw.abs().max()) <= 5 * float(dy.abs().max()) * (27 * U * 30 * U * abs(value) * 1000 + U)


@pytest.mark.parametrize("n", [128, 1999, 8192])
def test_eps_of_zero_and_infinite_values(n):
    x = torch.randn(6, n, generator=torch.Generator().manual_seed(n)) + 50.0
    x[1, 3], x[4, n - 1] = float("inf"), float("nan")
    c, y = x.cuda(), torch.empty(6, n, device="cuda")
    gdn.gdn_norm_fwd(c, None, None, None, y, eps=0.0, rms=False)
    y = y.double().cpu()
    good = [0, 2, 3, 5]
    ref = plain64.norm(x[good].double(), None, None, None, False, 0.0)
    assert torch.isnan(y[[1, 4]]).all()
    assert float((y[good] - ref).abs().max()) <= 128 * U * (1 + float(ref.abs().max()) + 30 * U * 60)


@pytest.mark.parametrize("n", [8, 40, 64, 100, 127, 128, 250, 256, 300, 511, 512, 1999])
@pytest.mark.parametrize("t", [F32, BF])
def test_rows_do_not_depend_on_their_neighbours(n, t):
    # rows with ordinary means come out bit for bit as they do where no row has a large one
    gen = torch.Generator().manual_seed(n)
    x = (torch.randn(64, n, generator=gen) + 0.7).to(t)
    dy = torch.randn(64, n, generator=gen).to(t).cuda()
    mixed = x.clone()
    big = torch.randperm(64, generator=gen)[:20]
    mixed[big] = (mixed[big].float() * 0.1 + 50.0).to(t)
    rest = [i for i in range(64) if i not in set(big.tolist())]
    out = []
    for a in (x.cuda(), mixed.cuda()):
        y, dx = torch.empty_like(a), torch.empty_like(a)
        gdn.gdn_norm_fwd(a, None, None, None, y, eps=EPS, rms=False)
        gdn.gdn_norm_bwd(a, None, None, None, dy, dx, None, None, None, gdn.alloc_norm_bwd_workspace(64, n), eps=EPS,
                         rms=False)
        out.append((y[rest], dx[rest]))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
