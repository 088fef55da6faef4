"""The operators together, as examples/w4_mlp.py runs them: entropy-coded
projection, residual + norm, 4-bit MLP with int8 activations, norm.

Tolerance: int8 activations are off by half a step at most, 1/254 of a token's
largest value, and by 1 / (127 sqrt(12)) of it in the mean square; with the largest of a few thousand near-normal values at about 4 sigma (and
heavier tails after silu * up, up to about 15), the norm's input to each
product is off by about 4 / (127 * sqrt(12)) = 0.9% and the down product's by
up to 3.4%; random signs carry both into the MLP's output at that size, and
the residual (twice the MLP's output or more in norm) dilutes them: 5% bounds
the output, bf16's 0.4% included."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT, gpu_available
from gpu_util import log
from rans_decode_amd import eq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def example():
    spec = importlib.util.spec_from_file_location("w4_mlp", os.path.join(ROOT, "examples", "w4_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("hidden,inner,group", [(1024, 2816, 128), (512, 1000, 32)])
def test_step_matches_64_bits(hidden, inner, group):
    log(f"case half block {hidden} {inner} {group}")
    off, off_residual = example().main(["--hidden", str(hidden), "--inner", str(inner), "--group", str(group)])
    assert off < 0.05 and off_residual < 0.05


def test_step_in_a_graph():
    """The whole step captured once and replayed, each replay against the eager step."""
    log("case half block in a graph")
    m = example()
    block = m.Block(512, 1024, 64)
    attention = torch.randn(512, device="cuda").to(torch.bfloat16)
    start = torch.randn(512, device="cuda")
    residual = start.clone()
    block.step(attention, residual)  # warm
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        block.step(attention, residual)
    for i in range(4):
        new = torch.randn(512, device="cuda").to(torch.bfloat16)
        attention.copy_(new)
        residual.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        out, res = block.out.clone(), residual.clone()
        residual.copy_(start)
        want = block.step(attention, residual)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(res, residual), i


def test_norm_output_feeds_the_products():
    """int8 and E4M3 matrices of the norm go straight into the products: exact against their values."""
    log("case norm to product")
    g = torch.Generator().manual_seed(5)
    for xt, dtype in ((torch.int8, eq.EQ_DTYPE_INT4), (torch.float8_e4m3fn, eq.EQ_DTYPE_E2M1)):
        tokens, cols, rows = 5, 300, 40
        x = torch.randn(tokens, cols, generator=g).cuda()
        a, s = torch.empty(tokens, cols, dtype=xt, device="cuda"), torch.empty(tokens, device="cuda")
        eq.eq_add_rmsnorm(x, None, 1e-5, a, out_scale=s)
        codes = torch.randint(0, 256, (rows, cols // 2), generator=g).to(torch.uint8)
        w = eq.W4Tensor(codes.cuda(), torch.ones(rows, 5, dtype=torch.bfloat16, device="cuda"), dtype=dtype, group=64)
        y = torch.empty(tokens, rows, device="cuda")
        eq.eq_w4_matvec(eq.W4Block([w]), [a], [y], [s])
        torch.cuda.synchronize()
        q = torch.stack([codes & 15, codes >> 4], dim=2).flatten(1).to(torch.int64)
        v = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6] if xt != torch.int8 else [*range(8), *range(-8, 0)]
        w64 = torch.tensor(v, dtype=torch.float64)[q]
        x64 = a.cpu().float().double() * s.cpu().double()[:, None]
        # 48 = the largest |16 + u| + |24| an INT4 product adds up, per unit of |x|
        bound = (cols + 16) * 2.0 ** -24 * x64.abs().sum(dim=1, keepdim=True) * 48
        assert bool(((y.cpu().double() - x64 @ w64.t()).abs() <= bound).all())
