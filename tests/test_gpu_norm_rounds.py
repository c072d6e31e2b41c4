"""Rows of pairs (lengths that are no multiple of four) in numbers that take a group of threads through several
rounds of the grid and its ring of stages more than once: the stages' reuse, the rule that a group's rows
start alike, the copies of the weights. Against the plain 64-bit form (on the GPU, in float64), with the
tolerances of test_gpu_norm: its chains of additions for dw and db, at most 400, hold here too (a thread's rows, at
most 34, then 32 groups, 5 blocks and 5 exchanges)."""
import pytest
import torch

import plain64
from context_scan_gb300 import gdn
from test_gpu_norm import BF, EPS, F32, U, _lib, half  # noqa: F401
from gpu_util import record

pytestmark = pytest.mark.gpu

# (length, threads of a row): every group from a part of a warp to a whole block
WIDTHS = [(62, 8), (125, 16), (250, 32), (511, 32), (999, 64), (1999, 128), (4095, 256), (4097, 512)]


def enough(n, g):
    """Rows for eight rounds of the largest grid that an SM's 2048 threads allow (a ring is at most seven
    stages deep), and some: an odd number, so that the last round is not full."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 8 * sms * (2048 // g) + 37


def near(got, ref, bound, t, label):
    assert torch.isfinite(got).all(), label
    off = ((got.double() - ref).abs() - half(t) * ref.abs() * (1 + 1e-6)) / bound
    record(float(off.max()), label)
    assert float(off.max()) <= 1, (label, float(off.max()))


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("n,g", WIDTHS)
def test_several_rounds(n, g, xt, yt, gated, rms):
    rows = enough(n, g)
    gen = torch.Generator(device="cuda").manual_seed(n)

    def normal(*shape, t=F32, mean=0.0, sd=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(sd).add_(mean).to(t)

    x, dy, w, b = normal(rows, n, t=xt, mean=0.3), normal(rows, n, t=yt), normal(n, mean=1.0, sd=0.3), normal(n, sd=0.3)
    z = normal(rows, n, t=yt, sd=2.0) if gated else None
    y = torch.full((rows, n), float("nan"), dtype=yt, device="cuda")
    dx, dz = torch.full_like(x, float("nan")), torch.full_like(z, float("nan")) if gated else None
    dw, db = torch.full_like(w, float("nan")), torch.full_like(b, float("nan"))
    gdn.gdn_norm_fwd(x, w, b, z, y, eps=EPS, rms=rms)
    gdn.gdn_norm_bwd(x, w, b, z, dy, dx, dz, dw, db, gdn.alloc_norm_bwd_workspace(rows, n), eps=EPS, rms=rms)
    x64, w64, b64, dy64 = x.double(), w.double(), b.double(), dy.double()
    z64 = None if z is None else z.double()
    sg = 1.0 if z is None else torch.sigmoid(z64)
    zs = 1.0 if z is None else (z64 * sg).abs()
    zz = 1.0 if z is None else 1 + z64.abs()
    xm = x64 if rms else x64 - x64.mean(-1, keepdim=True)
    s = 1 / torch.sqrt(xm.square().mean(-1, keepdim=True) + EPS)
    top = (x64.abs().amax(-1, keepdim=True) * s).clamp(min=1.0)
    y0, dd = top * w64.abs() + b64.abs(), dy64.abs() * zs
    near(y, plain64.norm(x64, w64, b64, z64, rms, EPS), 128 * U * y0 * zs + 1e-37, yt, "y")
    rdx, rdz, rdw, rdb = plain64.norm_grads(x, w, b, z, dy, rms, EPS)
    near(dx, rdx, 256 * U * (1 + top * top) * (dd * w64.abs()).amax(-1, keepdim=True) * s, xt, "dx")
    if gated:
        near(dz, rdz, 128 * U * y0 * (dy64 * sg).abs() * zz + 1e-37, yt, "dz")
    near(dw, rdw, 400 * U * (dd * top).sum(0), F32, "dw")
    near(db, rdb, 400 * U * dd.sum(0), F32, "db")


@pytest.mark.parametrize("n,g", WIDTHS)
def test_rows_do_not_depend_on_the_round(n, g):
    # the same few rows over and over: each comes out as it does in the first round
    rows, k = enough(n, g), 6
    few = torch.randn(k, n, generator=torch.Generator().manual_seed(n)).to(BF).cuda()
    x = few.repeat(rows // k + 1, 1)[:rows].contiguous()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_norm_fwd(x, None, None, None, y, eps=EPS, rms=False)
    gdn.gdn_norm_bwd(x, None, None, None, x, dx, None, None, None, gdn.alloc_norm_bwd_workspace(rows, n), eps=EPS,
                     rms=False)
    for t in (y, dx):
        assert torch.equal(t, t[:k].repeat(rows // k + 1, 1)[:rows])
