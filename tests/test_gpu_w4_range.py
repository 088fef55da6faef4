"""eq_w4_matvec with bf16 activations that are infinite or near the end of
their range, where sums of codes taken as 16 + u (INT4) or taken before their scale
overflow although the output does not.

Exact comparison, as in test_gpu_w4: whole activations times one power of two,
scales that are powers of two, so that every partial sum of W x is exact in
fp32; an output that is an infinity or a NaN by the definition (0 times an
infinity, infinities of both signs) is that infinity or a NaN."""
import pytest
import torch

from conftest import gpu_available
from gpu_util import log
from rans_decode_amd import eq
from test_gpu_w4 import BF16, F32, KINDS, Weights, make_x

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

KINDS16 = [k for k in KINDS if k[2] == BF16]
# tokens, rows, cols: by number of tokens and of rows every way of sharing out the work; ragged ends of each side
SHAPES = [(1, 40, 300), (3, 4117, 130), (4, 33, 1000), (7, 4133, 264), (8, 16, 128), (16, 50, 777), (16, 10260, 200),
          (20, 300, 600), (31, 10300, 129), (40, 19, 640), (64, 4120, 300), (9, 41000, 520), (20, 41000, 130),
          (64, 30001, 1100), (70, 25, 90)]


def scaled_down(w, by):
    """The same weights with scales (powers of two) times 2^-by."""
    w.scales = (w.scales.float() * 2.0 ** -by).to(BF16)
    w.w = w.w * 2.0 ** -by
    return w


def product(w, x, yt):
    y = torch.empty(x.shape[0], w.rows, dtype=yt, device="cuda")
    eq.eq_w4_matvec(eq.W4Block([w.device()]), [x], [y])
    torch.cuda.synchronize()
    return y.cpu()


def same(got, want):
    """Equal where a number or an infinity, NaN where NaN."""
    nan = torch.isnan(want)
    return torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("kind,zeros,xt", KINDS16)
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_large_finite_activations_exact(kind, zeros, xt, tokens, rows, cols):
    """|x| up to 2^127: sums of whole codes overflow, the outputs stay below 2^118."""
    for group in (32, 64, 128):
        log(f"case w4 large x {kind} {zeros} {tokens} x {rows} x {cols} group {group}")
        w = scaled_down(Weights(31, rows, cols, kind, zeros, group, True), 24)
        x, _, x64 = make_x(32, tokens, cols, xt, True)
        big = torch.arange(tokens) % 3 != 1  # tokens of ordinary size among them
        factor = torch.where(big, 2.0 ** 125, 1.0)[:, None]
        x.mul_(factor.cuda().to(BF16))
        assert torch.isfinite(x).all()
        want = (x64 * factor.double()) @ w.w.t()
        for yt in (F32, BF16):
            assert same(product(w, x, yt), want.to(yt)), yt


@pytest.mark.parametrize("kind,zeros,xt", KINDS16)
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_infinite_activations(kind, zeros, xt, tokens, rows, cols):
    """One infinity in some tokens, of one sign or both in others: y as defined, other tokens exact."""
    log(f"case w4 infinite x {kind} {zeros} {tokens} x {rows} x {cols}")
    w = Weights(41, rows, cols, kind, zeros, 64, True)
    x, _, x64 = make_x(42, tokens, cols, xt, True)
    x, x64 = x.clone(), x64.clone()
    for t in range(tokens):
        at = {0: [(cols // 2, 1.0)], 1: [], 2: [(cols - 1, -1.0)], 3: [(0, 1.0), (cols - 1, -1.0)]}[t % 4]
        for c, sign in at:
            x[t, c] = x64[t, c] = sign * float("inf")
    # by the definition: the finite part, and the products with infinities (0 times one is a NaN)
    want = x64.nan_to_num(posinf=0.0, neginf=0.0) @ w.w.t()
    for t in range(tokens):
        for c in torch.isinf(x64[t]).nonzero().flatten().tolist():
            want[t] += x64[t, c] * w.w[:, c]
    for yt in (F32, BF16):
        assert same(product(w, x, yt), want.to(yt)), yt
