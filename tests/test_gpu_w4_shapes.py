"""eq_w4_matvec: tensors of very different sizes in one call.

The kernel is chosen for the call's tensors together; a tensor of a few rows
(a router or a gate) beside large ones must not change theirs: y of the large
tensor is bit for bit what it is alone."""
import pytest
import torch

from conftest import gpu_available
from gpu_util import log
from rans_decode_amd import eq
from test_gpu_w4 import F32, KINDS, Weights, check, make_x

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
@pytest.mark.parametrize("tokens,rows,cols", [(4, 41000, 600), (9, 41000, 1100), (16, 11000, 600), (20, 41000, 1100), (64, 41000, 600),
                                              (64, 18000, 1100), (24, 11000, 300)])
def test_small_tensors_beside_a_large_one(kind, zeros, xt, tokens, rows, cols):
    log(f"case w4 small beside large {kind} {zeros} {xt} {tokens} x {rows} x {cols}")
    ws = [Weights(51 + i, r, cols, kind, zeros, 128, exact) for i, (r, exact) in
          enumerate([(rows, False), (5, True), (16, True), (33, True), (49, True)])]
    packed = [w.device() for w in ws]
    x, scale, x64 = make_x(61, tokens, cols, xt, False)
    xs, _, xs64 = make_x(62, tokens, cols, xt, True)
    ones = torch.ones(tokens, device="cuda") if scale is not None else None

    def run(which):
        ys = [torch.full((tokens, ws[i].rows), 77.0, dtype=F32, device="cuda") for i in which]
        eq.eq_w4_matvec(eq.W4Block([packed[i] for i in which]), [x if i == 0 else xs for i in which], ys,
                        [scale if i == 0 else ones for i in which] if scale is not None else None)
        torch.cuda.synchronize()
        return ys

    alone = run([0])[0]
    check(alone, ws[0], x64, False, "alone")
    plain = xs.cpu().float().double()
    for which in ([0, 1], [2, 0], [0, 1, 2, 3, 4], [3, 4, 0]):
        for i, y in zip(which, run(which)):
            if i == 0:
                assert torch.equal(y, alone), which
            else:
                check(y, ws[i], plain, True, f"tensor of {ws[i].rows} rows beside {rows}")
