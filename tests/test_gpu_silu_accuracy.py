"""eq_silu_mul's fp32 arithmetic, read through the scales of an 8-bit output of
one column: scale = |y| / L, two roundings away from the kernel's y.

Tolerance: the exponential's argument is corrected by its residual, so relative errors
do not grow with |g| but for ln 2's own rounding (2 ulp at |g| = 87). In units of 2^-23:
up to two hardware exponentials and a reciprocal 1 each, the residual 2, 1 + e, its
correction, up to four products and the two roundings of the scale 1/2 each: 9, and
second-order terms far below one: 10 * 2^-23."""
import pytest
import torch

from conftest import gpu_available
from gpu_util import log
from rans_decode_amd import eq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

ULPS = 10 * 2.0 ** -23


@pytest.mark.parametrize("low,high", [(-1.0, 1.0), (-20.0, 20.0), (-60.0, -20.0), (-91.0, -60.0), (60.0, 120.0)])
def test_relative_error_does_not_grow(low, high):
    log(f"case silu accuracy {low} {high}")
    n = 200000
    g = low + (high - low) * torch.rand(n, 1, generator=torch.Generator().manual_seed(1))
    lift = 2.0 ** 100 if low < -20 else 1.0  # keeps |y| well above the floor of a row's maximum
    u = (0.5 + torch.rand(n, 1, generator=torch.Generator().manual_seed(2))) * lift
    out, scale = torch.empty(n, 1, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    eq.eq_silu_mul(g.cuda(), u.cuda(), out, out_scale=scale)
    torch.cuda.synchronize()
    y = (g.double() / (1 + torch.exp(-g.double())) * u.double()).flatten()
    off = ((scale.cpu().double() * 127 - y.abs()).abs() / y.abs())[y.abs() > 2.0 ** -90]
    log(f"largest {float(off.max()) * 2 ** 23:.2f} * 2^-23, root of mean square {float(off.square().mean().sqrt()) * 2 ** 23:.3f}")
    assert off.numel() > n // 2 and float(off.max()) <= ULPS


def test_ends_of_the_range():
    """Zeros, infinities and NaN as g / (1 + exp(-g)) has them in fp32's range."""
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([0.0, -0.0, inf, -inf, nan, 3.4e38, -3.4e38, -500.0, -104.0, 1.0, 1.0], device="cuda")
    u = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 0.5, 1e38, 1e38, 1.0, inf, nan], device="cuda")
    o = torch.empty(11, dtype=torch.bfloat16, device="cuda")
    eq.eq_silu_mul(g, u, o)
    torch.cuda.synchronize()
    got = o.float().cpu()
    assert float(got[0]) == 0 and float(got[1]) == 0 and got[2] == inf
    assert torch.isnan(got[3]) and torch.isnan(got[4])
    assert torch.equal(got[5], torch.tensor(1.7e38).to(torch.bfloat16).float())
    assert float(got[6]) == 0 and float(got[7]) == 0 and abs(float(got[8])) < 1e-40
    assert got[9] == inf and torch.isnan(got[10])
