"""eq_add_rmsnorm over the whole range of finite rows: where squares overflow or
vanish in fp32, and where s * weight does before the row's factor is applied.

Tolerances as in test_gpu_rownorm (E = 2^-16 for sums over a row; the output is of
ordinary size, whatever the row's)."""
import pytest
import torch

from conftest import gpu_available
from gpu_util import log
from rans_decode_amd import eq
from test_gpu_rownorm import BF16, E, E4M3, F32, I8, check_out, outputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def run(tokens, cols, size, xt, rt, out, eps=0.0, in_place=False, weight_size=1.0, wt=F32):
    """Rows of about `size`, every third of ordinary size."""
    what = f"norm range {tokens}x{cols} size {size:g} eps {eps:g} {xt} {rt} -> {out}"
    log("case " + what)
    g = torch.Generator().manual_seed(cols)
    sizes = torch.tensor([1.0 if t % 3 == 1 else size for t in range(tokens)], dtype=torch.float64)[:, None]
    x = ((torch.rand(tokens, cols, generator=g).double() * 2 - 1) * sizes).to(xt)
    r = ((torch.rand(tokens, cols, generator=g).double() * 2 - 1) * sizes * 0.5).to(rt) if rt else None
    w = ((1 + 0.3 * torch.randn(cols, generator=g)) * weight_size).to(wt) if wt else None
    s = (x.float() + r.float()).to(rt) if rt else x
    assert torch.isfinite(s.float()).all()
    o, scale, _ = outputs(tokens, cols, out)
    rd = r.cuda() if rt else None
    ro = None if in_place or not rt else torch.empty_like(rd)
    eq.eq_add_rmsnorm(x.cuda(), w.cuda() if wt else None, eps, o, out_scale=scale, residual=rd, residual_out=ro)
    torch.cuda.synchronize()
    if rt:
        assert torch.equal((rd if in_place else ro).cpu(), s), what
    s = s.double()
    eps = float(torch.tensor(eps, dtype=torch.float32))
    y = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps) * (w.double() if wt else 1.0)
    check_out(y, E, o, scale, what)


@pytest.mark.parametrize("cols", [1, 100, 4096, 20000, 33000])
@pytest.mark.parametrize("out", [BF16, I8, E4M3])
def test_squares_out_of_range(cols, out):
    for size in (1e18, 1e20, 1e30, 2e38):
        run(4, cols, size, F32, None, out, eps=1e-5)
        run(4, cols, size, BF16, BF16, out, eps=1e-5, in_place=cols % 2 == 0)
        run(3, cols, size, BF16, F32, out, eps=1e-5)
    for size in (1e-18, 1e-20, 1e-25, 1e-36):
        run(4, cols, size, F32, None, out)
        run(4, cols, size, BF16, BF16, out, in_place=cols % 2 == 0)
        run(3, cols, size, F32, F32, out, eps=size * size)  # eps of the squares' own size, where fp32 holds it


@pytest.mark.parametrize("out", [BF16, I8, E4M3])
def test_many_rows_out_of_range(out):
    run(1100, 1000, 1e25, BF16, None, out, eps=1e-5)
    run(1030, 17001, 1e30, BF16, BF16, out, eps=1e-5)


@pytest.mark.parametrize("out", [BF16, I8, E4M3])
def test_products_with_the_weight_out_of_range(out):
    """s * weight overflows, s / rms * weight does not."""
    for cols in (100, 4096, 33000):
        run(4, cols, 3e38, F32, None, out, eps=1e-5)
        run(4, cols, 1e15, F32, None, out, eps=1e-5, weight_size=1e25)
        run(4, cols, 1e10, BF16, BF16, out, eps=1e-5, weight_size=1e30, wt=BF16)


@pytest.mark.parametrize("out", [BF16, I8, E4M3])
def test_huge_weights(out):
    """s * weight overflows where s itself is of ordinary size, and where s is small and eps 0."""
    for cols in (7, 100, 4096, 20000, 33000):
        run(4, cols, 100.0, F32, None, out, eps=1e-5, weight_size=5e37)
        run(4, cols, 30.0, BF16, BF16, out, eps=1e-5, weight_size=5e37, wt=BF16)
        run(5, cols, 1e-14, F32, None, out, weight_size=1e30)
        run(4, cols, 1e-20, BF16, F32, out, weight_size=5e37)
        run(4, cols, 1e19, F32, F32, out, eps=1e-5, weight_size=5e37, in_place=True)
