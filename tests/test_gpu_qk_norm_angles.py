"""The rotation's angles at any position and frequency, against n freq modulo a turn in whole numbers: freq is a fraction, 1 / 2 pi
has 600 binary digits (Machin's formula), so that what is left of a turn is exact.

Tolerance: that of the forward (24 steps of 2^-24 of the pair's values, the angle's rounding to fp32 among them); nothing is
added for far positions or large frequencies."""
import math
from fractions import Fraction

import pytest
import torch

import plain64_linear as plain
from context_scan_gb300 import gdn
from gpu_util import record
from test_gpu_qk_norm import F32, STEP, call, make, pairs

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, -1, 2**31 - 1, -2**31, 10**9 + 7, 123456789, 2**24 + 1, -(10**6), 131071, 2**30 + 12345, -2**31 + 1]
DIGITS = 600


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def inverse_turn():
    def arctan_inverse(x):
        term = (1 << DIGITS + 40) // x
        total, n, sign = term, 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total
    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return Fraction((1 << 2 * DIGITS + 40) // (2 * pi), 1 << DIGITS)


def angles(freq, positions):
    """[positions, pairs] in float64, within half a turn of 0."""
    inv, out = inverse_turn(), []
    for n in positions:
        turns = [n * Fraction(float(f)) * inv for f in freq]
        out.append([2 * math.pi * float(t - round(t)) for t in turns])
    return torch.tensor(out, dtype=torch.float64)


FREQ = {
    "usual": [10000.0 ** (-2 * i / 256) for i in range(128)],
    "one": [(-1.0) ** i * (1 + 2.0 ** -23 * (37 * i % 8388607)) for i in range(128)],
    "large": [1.7 ** i for i in range(128)],
    "small": [(-1.0) ** (i // 3) * 1.99 ** -i for i in range(128)],
    "every_exponent": [1.2345 * 2.0 ** (2 * i - 128) for i in range(128)],
    "ends": [0.0, -0.0, 2.0 ** -149, -2.0 ** -149, 2.0 ** -126, 1.5 * 2.0 ** -127, 3.4e38, -3.4e38] + [1.999 * 2.0 ** (i - 63) for i in range(120)],
}


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("name", sorted(FREQ))
def test_angles(name, il):
    d = make(1, len(POSITIONS), 2, 1, 256, 256, x=F32, y=F32)
    d["freq"] = torch.tensor(FREQ[name], dtype=torch.float64).float().cuda()
    d["pos"] = torch.tensor([POSITIONS], dtype=torch.int32).cuda()
    t = angles(d["freq"].cpu(), POSITIONS)[None, :, None, :]
    for got, x, w in zip(call(d, il), (d["q"], d["k"]), (d["wq"], d["wk"])):
        u = plain.qk_norm(x.double().cpu(), w.double().cpu(), None, None, il, 1e-6)
        a, b = (u[..., 0::2], u[..., 1::2]) if il else (u[..., :128], u[..., 128:])
        ya, yb = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
        ref = torch.stack([ya, yb], -1).flatten(-2) if il else torch.cat([ya, yb], -1)
        tol = 24 * STEP * pairs(u, 256, il)
        off = (got.double().cpu() - ref).abs()
        record(float((off / tol).max()), "y")
        assert (off <= tol).all(), float((off / tol).max())
