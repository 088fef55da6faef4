"""Every kernel that eq_w4_matvec chooses among, each case with the kernel it is
there for: by tokens that share a matrix instruction (TP), token tiles (NT) and
rows of tiles a wave (R), and the one that shares activations ("wide"). The
kernel's name is read from a profile of the call, so that a change of the rule
which moves a case to another kernel shows here.

Exact comparison as in test_gpu_w4. Accuracy on full-precision values, by the
2-norm of y - W x over that of W x. With rounding errors of random signs, 2^-24 /
sqrt(3) of the value rounded each: INT4 x bf16 sums groups of codes 16 + u and of
16 + zero, 5.5 times the size of W x for uniform codes, in up to 8 roundings
each: sqrt(16) 5.5 2^-24 / sqrt(3) = 7.6e-7; joining up to 896 groups of a long row
adds sqrt(896 / 2) 2^-24 / sqrt(3) = 7.3e-7 and x's scale less than 1e-7: below
1.5e-6. (Sums held in fewer than 32 bits were 1e-5 off.)"""
import re

import pytest
import torch
from torch.profiler import ProfilerActivity, profile

from conftest import gpu_available
from gpu_util import log
from rans_decode_amd import eq
from test_gpu_w4 import BF16, E2M1, E4M3, I8, KINDS

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

# tokens, rows, cols, (TP, NT, R) or ("wide", NT, R); rows and columns end inside tiles and groups
CASES = [(1, 300, 2100, (4, 1, 1)), (3, 3000, 2100, (4, 1, 1)), (2, 4200, 2100, (4, 1, 2)), (4, 12000, 2100, (4, 1, 2)),
         (6, 300, 2100, (8, 1, 1)), (5, 4200, 2100, (8, 1, 2)), (8, 9000, 2100, (8, 1, 2)),
         (9, 300, 2100, (16, 1, 1)), (16, 4200, 2100, (16, 1, 2)), (13, 10250, 2100, (16, 1, 4)),
         (160, 2050, 2100, (16, 2, 1)), (31, 8300, 2100, (16, 2, 2)), (24, 10250, 2100, (16, 2, 4)),
         (300, 2050, 2100, (16, 4, 1)), (64, 8300, 2100, (16, 4, 2)), (37, 16001, 2100, (16, 4, 2)),
         (16, 41000, 700, ("wide", 1, 2)), (20, 25000, 1100, ("wide", 2, 1)), (32, 41000, 700, ("wide", 2, 2)),
         (64, 17000, 1100, ("wide", 4, 1)), (50, 41000, 700, ("wide", 4, 2)), (130, 41000, 300, ("wide", 4, 2))]


class Weights:
    """Random 4-bit weights on the GPU: packed, and W in 64 bits."""

    def __init__(self, seed, rows, cols, kind, zeros, group, exact):
        g = torch.Generator(device="cuda").manual_seed(seed)
        groups = -(-cols // group)
        codes = torch.randint(0, 16, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)
        padded = torch.nn.functional.pad(codes, (0, cols % 2), value=15)
        if exact:
            scales = (2.0 ** torch.randint(-3, 2, (rows, groups), generator=g, device="cuda")).to(BF16)
        else:
            scales = (0.002 + 0.006 * torch.rand(rows, groups, generator=g, device="cuda")).to(BF16)
        z = torch.randint(0, 16, (rows, groups), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
        self.block = eq.W4Block([eq.W4Tensor((padded[:, 0::2] + 16 * padded[:, 1::2]).contiguous(), scales, z, group=group, cols=cols,
                                             dtype=eq.EQ_DTYPE_E2M1 if kind == "e2m1" else eq.EQ_DTYPE_INT4)])
        at = torch.arange(cols, device="cuda") // group
        if kind == "e2m1":
            q = E2M1.cuda()[codes.int()]
        elif zeros:
            q = codes.double() - z.double()[:, at]
        else:
            q = torch.where(codes > 7, codes.double() - 16, codes.double())
        self.w = q.mul_(scales.double()[:, at])


def activations(seed, tokens, cols, xt, exact):
    g = torch.Generator(device="cuda").manual_seed(seed)
    scale = None
    if exact:
        v = torch.randint(-4, 5, (tokens, cols), generator=g, device="cuda").float()
        if xt != BF16:
            scale = 2.0 ** torch.randint(-2, 3, (tokens,), generator=g, device="cuda").float()
    else:
        v = torch.randn(tokens, cols, generator=g, device="cuda")
        if xt != BF16:
            v, scale = v * 30, 0.01 + 0.02 * torch.rand(tokens, generator=g, device="cuda")
            v = v.round().clamp(-127, 127) if xt == I8 else v.clamp(-448, 448)
    x = v.to(xt)
    x64 = x.float().double()
    return x, scale, x64 if scale is None else x64 * scale.double()[:, None]


def product(weights, x, scale, rows):
    """y, and the kernel that computed it as (TP, NT, R) or ("wide", NT, R); None where the profile names none."""
    y = torch.full((x.shape[0], rows), 77.0, device="cuda")
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        eq.eq_w4_matvec(weights.block, [x], [y], None if scale is None else [scale])
        torch.cuda.synchronize()
    ran = [m.groups() for m in (re.search(r"k_w4(_wide)?<([^>]*)>", e.name) for e in p.events()) if m]
    if not ran:
        return y, None
    args = [int(v) for v in re.findall(r"(\d+)u?(?:,|$)", ran[0][1].replace("false", "0").replace("true", "1"))]
    return y, ("wide", *args[4:6]) if ran[0][0] else tuple(args[4:7])


def expected(shape, xt, group):
    """8-bit activations in groups of 64 or 128 come 64 columns at a time: no four pieces a tile."""
    return (8, *shape[1:]) if shape[0] == 4 and xt in (I8, E4M3) and group != 32 else shape


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_kernel_exact(kind, zeros, xt, group):
    for i, (tokens, rows, cols, shape) in enumerate(CASES):
        log(f"case w4 kernel {shape} {kind} zeros={zeros} {xt} group {group}: {tokens} x {rows} x {cols}")
        w = Weights(100 + i, rows, cols, kind, zeros, group, True)
        x, scale, x64 = activations(200 + i, tokens, cols, xt, True)
        y, ran = product(w, x, scale, rows)
        want = x64 @ w.w.t()
        assert torch.equal(y.double(), want), f"{int((y != want).sum())} of {y.numel()} differ"
        assert ran is None or ran == expected(shape, xt, group)


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
@pytest.mark.parametrize("group", [32, 128])
def test_every_kernel_keeps_32_bits(kind, zeros, xt, group):
    cases = [(t, r, 8192 + 52, s) for t, r, _, s in CASES] + [(1, 300, 28672, (4, 1, 1)), (16, 4200, 28672, (16, 1, 2)),
                                                              (64, 8300, 28672, (16, 4, 2)), (64, 17000, 28672, ("wide", 4, 1))]
    for i, (tokens, rows, cols, shape) in enumerate(cases):
        log(f"case w4 accuracy {shape} {kind} zeros={zeros} {xt} group {group}: {tokens} x {rows} x {cols}")
        w = Weights(300 + i, rows, cols, kind, zeros, group, False)
        x, scale, x64 = activations(400 + i, tokens, cols, xt, False)
        y, ran = product(w, x, scale, rows)
        want = x64 @ w.w.t()
        off = float((y.double() - want).norm() / want.norm())
        log(f"{off:.2e}")
        assert off < 1.5e-6
        assert ran is None or ran == expected(shape, xt, group)


def test_most_tokens_of_a_call_exact():
    """64 * 65535 tokens: as many passes as a grid's second dimension has."""
    log("case w4 most tokens")
    tokens = 64 * 65535
    w = Weights(7, 1, 8, "int4", False, 32, True)
    x, scale, x64 = activations(8, tokens, 8, BF16, True)
    y = torch.empty(tokens, 1, device="cuda")
    eq.eq_w4_matvec(w.block, [x], [y])
    torch.cuda.synchronize()
    assert torch.equal(y.double(), x64 @ w.w.t())
