"""The gate z sigmoid(z) and its gradient over the whole range where it is a number of fp32, through rows
that the normalisation leaves at +-1.

Tolerance, derived (u = 2^-24): x is +-1 (and one 0), so the sums are exact, s = 1 / sqrt(mean + eps) to 2 u
of rounding and rsqrt's 4 u, and xh adds one: 7 u. sigmoid(z) = 1 / (1 + 2^(-z log2(e))): the product is rounded, u of itself,
and so is the constant, 0.23 u; both count |z| log2(e) ln(2) = |z| times in the exponential, which itself is good to 2 units of the
last place, 4 u; the sum adds u, the reciprocal 2 u, the two products with z and xh 2 u: 16 u + 1.25 |z| u of the value.
dz = xh sigmoid(z) (1 + z (1 - sigmoid(z))) adds the last factor, off by at most (9 + 1.25 |z|) u (1 + |z|) of the terms it
is the sum of, where sigmoid(z) is less than 1 / 2, and otherwise by (9 + 1.25 |z|) u |z| (1 - sigmoid(z)), which is less:
(32 + 2.5 |z|) u xh sigmoid(z) (1 + |z|). Values under the smallest normal number may be zero."""
import pytest
import torch

from context_scan_gb300 import gdn
from test_gpu_norm import EPS, U, _lib  # noqa: F401

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126


@pytest.mark.parametrize("n", [128, 131, 2000, 4096])
@pytest.mark.parametrize("rms", [True, False])
def test_every_size_of_gate(n, rms):
    gen = torch.Generator().manual_seed(n)
    rows = 200
    x = torch.ones(rows, n)
    x[:, 1::2] = -1.0
    if n % 2 and not rms:
        x[:, -1] = 0.0                         # (the mean is zero)
    z = torch.linspace(-87.0, 87.0, rows * n).view(n, rows).t().contiguous()
    z[0, :4] = torch.tensor([-300.0, 300.0, 0.0, -88.5])
    y, dx, dz = (torch.full((rows, n), float("nan"), device="cuda") for _ in range(3))
    xc, zc, one = x.cuda(), z.cuda(), torch.ones(rows, n, device="cuda")
    gdn.gdn_norm_fwd(xc, None, None, zc, y, eps=EPS, rms=rms)
    gdn.gdn_norm_bwd(xc, None, None, zc, one, dx, dz, None, None, gdn.alloc_norm_bwd_workspace(rows, n), eps=EPS,
                     rms=rms)
    z, x = z.double(), x.double()
    xh = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    sg = torch.sigmoid(z)
    y, dz = y.double().cpu(), dz.double().cpu()
    assert torch.isfinite(dx).all()
    ref = xh * z * sg
    off = ((y - ref).abs() - TINY * (1 + z.abs())) / ref.abs().clamp(min=1e-300)
    off = off / (16 + 1.25 * z.abs())
    assert float(off.max()) <= U, float(off.max() / U)
    ref, size = xh * sg * (1 + z * (1 - sg)), (xh * sg).abs() * (1 + z.abs())
    off = ((dz - ref).abs() - TINY * (1 + z.abs())) / size.clamp(min=1e-300)
    off = off / (32 + 2.5 * z.abs())
    assert float(off.max()) <= U, float(off.max() / U)
