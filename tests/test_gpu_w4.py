"""eq_w4_pack and eq_w4_matvec against the definition in 64 bits.

Two kinds of comparison. Exact: small whole activations, scales that are
powers of two: every product and every partial sum is a multiple of the
smallest scale times 1/2 and stays far below 2^24 of them, so fp32 sums are
exact in any order and y has one right value. Bounded: any values; with codes
read as 16 + u (INT4) the terms of one output add up in absolute value to
A = sum |scale| |x| (|16 + u| + |16 + zero|) (E2M1: sum |scale| |x| |q|), at
most cols + 16 roundings lie on any term's way into y, so
|y - exact| <= (cols + 16) 2^-24 A; a bf16 y lies between the roundings of
the lowest and the highest such value."""
import numpy as np
import pytest
import torch

from conftest import gpu_available
from gpu_util import log
from rans_decode_amd import eq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

F32, BF16, I8, E4M3 = torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
KINDS = [("int4", False, BF16), ("int4", True, BF16), ("int4", False, I8), ("int4", True, I8),
         ("e2m1", False, BF16), ("e2m1", False, E4M3)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Weights:
    """Random 4-bit weights on the CPU: row-major bytes, scales, zeros, and W in 64 bits."""

    def __init__(self, seed, rows, cols, kind, zeros, group, exact):
        g = gen(seed)
        self.rows, self.cols, self.group, self.kind = rows, cols, group, kind
        groups = -(-cols // group)
        self.codes = torch.randint(0, 16, (rows, cols), generator=g)
        padded = torch.nn.functional.pad(self.codes, (0, cols % 2), value=15)  # the spare half byte holds anything
        self.bytes = (padded[:, 0::2] + 16 * padded[:, 1::2]).to(torch.uint8).contiguous()
        if exact:
            self.scales = (2.0 ** torch.randint(-3, 2, (rows, groups), generator=g)).to(BF16)
        else:
            self.scales = (0.01 * torch.randn(rows, groups, generator=g)).to(BF16)
        self.zeros = torch.randint(0, 16, (rows, groups), generator=g).to(torch.uint8) if zeros else None
        at = torch.arange(cols) // group
        s = self.scales.double()[:, at]
        if kind == "e2m1":
            q = E2M1[self.codes]
            size = q.abs()
        elif zeros:
            z = self.zeros.double()[:, at]
            q = self.codes.double() - z
            size = (16 + self.codes.double()) + (16 + z)
        else:
            q = torch.where(self.codes > 7, self.codes - 16, self.codes).double()
            size = (24 + q) + 24
        self.w, self.size = q * s, size * s.abs()

    def device(self):
        return eq.W4Tensor(self.bytes.cuda(), self.scales.cuda(), self.zeros.cuda() if self.zeros is not None else None,
                           dtype=eq.EQ_DTYPE_INT4 if self.kind == "int4" else eq.EQ_DTYPE_E2M1, group=self.group,
                           cols=self.cols)


def make_x(seed, tokens, cols, xt, exact, stride=None):
    g = gen(seed)
    scale = None
    if exact:
        v = torch.randint(-4, 5, (tokens, cols), generator=g).double()
        if xt in (I8, E4M3):
            scale = 2.0 ** torch.randint(-2, 3, (tokens,), generator=g).float()
    elif xt == I8:
        v, scale = torch.randint(-128, 128, (tokens, cols), generator=g).double(), torch.rand(tokens, generator=g) * 0.02
    elif xt == E4M3:
        v = (torch.randn(tokens, cols, generator=g) * 60).clamp(-448, 448).to(E4M3).double()
        scale = torch.rand(tokens, generator=g) * 0.02
    else:
        v = torch.randn(tokens, cols, generator=g).to(BF16).double()
    buf = torch.full((tokens, stride or cols), 100 if xt == I8 else float("nan"), dtype=torch.float32).to(xt)
    buf[:, :cols] = v.to(xt)
    return buf.cuda()[:, :cols], scale.cuda() if scale is not None else None, v * (scale.double()[:, None] if scale is not None else 1)


def check(y, w, x64, exact, what):
    want = x64 @ w.w.t()
    got = y.cpu().double()
    if exact and y.dtype == F32:
        assert torch.equal(got, want), f"{what}: {int((got != want).sum())} of {got.numel()} differ"
        return
    bound = (w.cols + 16) * 2.0 ** -24 * (x64.abs() @ w.size.t())
    low, high = want - bound, want + bound
    if y.dtype == BF16:
        low, high = low.to(BF16).double(), high.to(BF16).double()
    assert bool(((low <= got) & (got <= high)).all()), f"{what}: off by {float((got - want).abs().max()):g}"


def run(seed, tokens, rows_list, cols, kind, zeros, xt, group, yt=F32, exact=True, strides=False):
    what = f"w4 {tokens} x {rows_list} x {cols} {kind} zeros={zeros} {xt} group {group} -> {yt}"
    log("case " + what)
    ws = [Weights(seed + i, r, cols, kind, zeros, group, exact) for i, r in enumerate(rows_list)]
    x, scale, x64 = make_x(seed + 50, tokens, cols, xt, exact, cols + 5 if strides else None)
    bufs = [torch.full((tokens, r + (3 if strides else 0)), 77.0, dtype=yt, device="cuda") for r in rows_list]
    ys = [b[:, :r] for b, r in zip(bufs, rows_list)]
    block = eq.W4Block([w.device() for w in ws])
    n = len(ws)
    eq.eq_w4_matvec(block, [x] * n, ys, [scale] * n if scale is not None else None)
    torch.cuda.synchronize()
    for w, y, b in zip(ws, ys, bufs):
        check(y, w, x64, exact, what)
        assert bool((b[:, w.rows:] == 77.0).all()), what


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_sizes_exact(kind, zeros, xt, group):
    """Sides around the 16 x 128 tile, the group, the byte; whole and ragged numbers of tokens."""
    for i, (tokens, rows, cols) in enumerate([(1, 1, 1), (1, 16, 128), (2, 17, 129), (3, 5, 31), (1, 100, 33), (16, 33, 64),
                                              (17, 16, 255), (5, 48, 1000), (32, 7, 511), (33, 31, 384), (1, 64, 4096),
                                              (64, 20, 1025), (65, 18, 130), (129, 3, 200)]):
        run(100 * i + group, tokens, [rows], cols, kind, zeros, xt, group)


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_values_bounded(kind, zeros, xt, group):
    for i, (tokens, rows, cols) in enumerate([(1, 70, 300), (4, 33, 128), (16, 50, 777), (40, 19, 640), (64, 100, 200)]):
        for yt in (F32, BF16):
            run(7000 + 10 * i + group, tokens, [rows], cols, kind, zeros, xt, group, yt=yt, exact=False, strides=True)


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
def test_larger_shapes_exact(kind, zeros, xt):
    """Several tensors in one call, as a block has them, and a long row."""
    run(1, 1, [1024, 128, 128], 1024, kind, zeros, xt, 128)
    run(2, 4, [520, 1000], 2048, kind, zeros, xt, 64)
    run(3, 16, [64], 28672, kind, zeros, xt, 128)
    run(4, 48, [300], 4100, kind, zeros, xt, 32, strides=True)
    run(5, 64, [2048], 512, kind, zeros, xt, 128)


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_many_rows_exact(kind, zeros, xt, group):
    """Enough rows that a workgroup's waves share the activations: chunks of 512 columns, none to several of them, whole and ragged."""
    for i, (tokens, cols) in enumerate([(9, 100), (16, 512), (17, 640), (32, 1111), (33, 1024), (64, 1700), (80, 513)]):
        run(9000 + 20 * i + group, tokens, [25000, 40], cols, kind, zeros, xt, group, strides=i % 2 == 0, yt=F32 if i else BF16)
    run(9500 + group, 48, [30001], 256, kind, zeros, xt, group, exact=False)


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_very_many_rows_exact(kind, zeros, xt, group):
    """The same with two rows of tiles a wave; the last workgroup's waves partly and wholly past the end."""
    for i, (tokens, cols) in enumerate([(9, 100), (16, 600), (20, 512), (64, 1025)]):
        run(9700 + 20 * i + group, tokens, [41000, 33], cols, kind, zeros, xt, group)


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
def test_rows_per_wave_exact(kind, zeros, xt):
    """Row counts where a wave takes 1, 2 or 4 rows of tiles, with rows of tiles left over, and columns split among 1 to 8 waves."""
    for i, (tokens, rows, cols) in enumerate([(1, 4100, 300), (3, 4100, 2100), (4, 4117, 130), (7, 4133, 1100), (16, 4133, 600),
                                              (12, 10260, 1300), (24, 10300, 390), (30, 4150, 2050), (50, 4120, 520)]):
        run(9900 + i, tokens, [rows], cols, kind, zeros, xt, (32, 64, 128)[i % 3])
    run(9950, 10, [10241, 64], 260, kind, zeros, xt, 64)


@pytest.mark.parametrize("kind,zeros,xt", KINDS)
def test_single_columns(kind, zeros, xt):
    """x with one 1 per token picks single weights: the layout, column by column."""
    cols, rows, group = 200, 21, 64
    w = Weights(9, rows, cols, kind, zeros, group, True)
    block = eq.W4Block([w.device()])
    eye = torch.eye(cols)
    scale = torch.ones(cols, device="cuda") if xt in (I8, E4M3) else None
    y = torch.empty(cols, rows, device="cuda")
    log(f"case w4 single columns {kind} {zeros} {xt}")
    eq.eq_w4_matvec(block, [eye.to(xt).cuda()], [y], [scale] if scale is not None else None)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().double(), w.w.t())


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 bytes of codes, x and y rows more than 2^32 bytes apart."""
    rows, cols, group = 140000, 65536, 128
    log("case w4 large offsets")
    g = torch.Generator(device="cuda").manual_seed(11)
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    for at in range(0, rows, 20000):
        codes[at:at + 20000].random_(0, 256, generator=g)
    scales = (2.0 ** torch.randint(-3, 2, (rows, cols // group), generator=g, device="cuda")).to(BF16)
    block = eq.W4Block([eq.W4Tensor(codes, scales, group=group)])
    assert block.tensors[0].codes.numel() > 1 << 32
    sample = torch.cat([torch.arange(40), torch.randint(0, rows, (200,), generator=gen(1)), torch.arange(rows - 40, rows)]).cuda()
    c = codes[sample]
    q = torch.stack([c & 15, c >> 4], dim=2).flatten(1).to(torch.int16)
    w = torch.where(q > 7, q - 16, q).double() * scales[sample].double().repeat_interleave(group, dim=1)
    del codes
    for tokens in (1, 3):  # 3 rows of x and y in buffers of about 13 GB
        step = (1 << 31) + 64
        x = torch.empty((tokens - 1) * step + cols, dtype=BF16, device="cuda")
        y = torch.empty((tokens - 1) * (step // 2) + rows, dtype=F32, device="cuda")
        xv, yv = x.as_strided((tokens, cols), (step, 1)), y.as_strided((tokens, rows), (step // 2, 1))
        xv.copy_(torch.randint(-2, 3, (tokens, cols), generator=g, device="cuda"))
        eq.eq_w4_matvec(block, [xv], [yv])
        torch.cuda.synchronize()
        assert torch.equal(yv[:, sample].double(), xv.double() @ w.t())
        del x, y, xv, yv
    torch.cuda.empty_cache()


def test_very_many_tokens_exact():
    """Passes along a grid's second dimension, near its limit, for a matrix of one workgroup."""
    for tokens, rows, cols in ((1100000, 16, 8), (4 * 65535 + 3, 5, 130)):
        run(31, tokens, [rows], cols, "int4", False, BF16, 32)


def test_kinds_mixed_in_one_call():
    """Tensors of several kinds and widths, more than fit one launch."""
    log("case w4 mixed kinds")
    ws, xs, scales, x64s, ys = [], [], [], [], []
    for i in range(40):
        kind, zeros, xt = KINDS[i % len(KINDS)]
        w = Weights(300 + i, 10 + 7 * i, 40 + 31 * i, kind, zeros, (32, 64, 128)[i % 3], True)
        x, s, x64 = make_x(600 + i, 6, w.cols, xt, True)
        ws.append(w), xs.append(x), scales.append(s), x64s.append(x64)
        ys.append(torch.empty(6, w.rows, dtype=F32 if i % 4 else BF16, device="cuda"))
    eq.eq_w4_matvec(eq.W4Block([w.device() for w in ws]), xs, ys, scales)
    torch.cuda.synchronize()
    for i, (w, x64, y) in enumerate(zip(ws, x64s, ys)):
        check(y, w, x64, y.dtype == F32, f"mixed {i}")


def test_bad_values_stay_with_their_token_and_row():
    """NaN and infinities in one token's x or one row's scales reach that token or row alone."""
    for kind, zeros, xt in KINDS:
        for group in (32, 128):
            log(f"case w4 bad values {kind} {zeros} {xt} {group}")
            w = Weights(21, 40, 300, kind, zeros, group, True)
            x, scale, x64 = make_x(22, 5, 300, xt, True)
            want = x64 @ w.w.t()
            if xt == I8:
                scale[3] = float("nan")
            else:
                x[3, 299] = float("nan")
            w.scales[7, 0] = float("inf")
            y = torch.empty(5, 40, device="cuda")
            eq.eq_w4_matvec(eq.W4Block([w.device()]), [x], [y], [scale] if scale is not None else None)
            torch.cuda.synchronize()
            y = y.cpu().double()
            assert torch.isnan(y[3]).all()
            rest = [0, 1, 2, 4]
            cols = [r for r in range(40) if r != 7]
            assert torch.equal(y[rest][:, cols], want[rest][:, cols])
            assert not torch.isfinite(y[rest, 7]).any()


def test_no_tokens_no_tensors_and_other_streams():
    log("case w4 nothing to do")
    w = Weights(1, 33, 150, "int4", False, 64, True)
    block = eq.W4Block([w.device()])
    eq.eq_w4_matvec(eq.W4Block([]), [], [])
    eq.eq_w4_matvec(block, [torch.empty(0, 150, dtype=BF16, device="cuda")], [torch.empty(0, 33, device="cuda")])
    log("case w4 another stream")
    x, _, x64 = make_x(2, 9, 150, BF16, True)
    y = torch.empty(9, 33, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eq.eq_w4_matvec(block, [x], [y], stream=side)
    torch.cuda.synchronize()
    check(y, w, x64, True, "another stream")


def test_one_token_in_one_dimension_and_repeats():
    log("case w4 one dimension, repeated")
    w = Weights(3, 1000, 2000, "int4", False, 128, False)
    block = eq.W4Block([w.device()])
    x, _, x64 = make_x(4, 1, 2000, BF16, False)
    first = None
    for _ in range(5):
        y = torch.empty(1000, device="cuda")
        eq.eq_w4_matvec(block, [x[0]], [y])
        torch.cuda.synchronize()
        check(y[None], w, x64, False, "one dimension")
        first = y if first is None else first
        assert torch.equal(first, y)


def test_pack_layout():
    """The tiled arrays, entry by entry, from the layout's description."""
    for kind, zeros, group, rows, cols in (("int4", True, 32, 19, 300), ("e2m1", False, 128, 32, 129), ("int4", False, 64, 3, 5)):
        log(f"case w4 layout {kind} {group}")
        w = Weights(5, rows, cols, kind, zeros, group, True)
        t = w.device()
        k_tiles, per = -(-cols // 128), 128 // group
        words = t.codes.cpu().numpy().view(np.uint32).reshape(-(-rows // 16), k_tiles, 4, 16, 4)
        place = [0, 2, 4, 6, 1, 3, 5, 7] if kind == "int4" else list(range(8))
        scales = t.scales.cpu().view(torch.int16).numpy().reshape(-(-rows // 16), k_tiles, 16, per)
        src = w.scales.view(torch.int16).numpy()
        zs = t.zeros.cpu().numpy().reshape(scales.shape) if zeros else None
        for r in range(16 * -(-rows // 16)):
            for c in range(128 * k_tiles):
                if group == 32:
                    quarter, j = c % 32 // 8, c % 128 // 32
                else:
                    quarter, j = c % 64 // 16, c % 128 // 64 * 2 + c % 16 // 8
                word = int(words[r // 16, c // 128, quarter, r % 16, j])
                got = word >> 4 * place.index(c % 8) & 15
                assert got == (int(w.codes[r, c]) if r < rows and c < cols else 0)
            for g in range(k_tiles * per):
                there = r < rows and g < src.shape[1]
                assert scales[r // 16, g // per, r % 16, g % per] == (src[r, g] if there else 0)
                if zeros:
                    assert zs[r // 16, g // per, r % 16, g % per] == (int(w.zeros[r, g]) if there else 0)


def test_wrapper_refusals():
    w = Weights(1, 32, 128, "int4", False, 64, True)
    t = w.device()
    block = eq.W4Block([t])
    x = torch.zeros(2, 128, dtype=BF16, device="cuda")
    y = torch.zeros(2, 32, device="cuda")
    s = torch.ones(2, device="cuda")
    codes, scales = w.bytes.cuda(), w.scales.cuda()
    for call in (lambda: eq.eq_w4_matvec(block, [x, x], [y]),
                 lambda: eq.eq_w4_matvec(block, [x[:, :127]], [y]),
                 lambda: eq.eq_w4_matvec(block, [x], [y[:1]]),
                 lambda: eq.eq_w4_matvec(block, [x], [y], [s]),
                 lambda: eq.eq_w4_matvec(block, [x.to(I8)], [y]),
                 lambda: eq.eq_w4_matvec(block, [x.cpu()], [y]),
                 lambda: eq.W4Tensor(codes, scales[:, :1].contiguous(), group=64),
                 lambda: eq.W4Tensor(codes, scales.float(), group=64),
                 lambda: eq.W4Tensor(codes, scales, group=64, cols=126),
                 lambda: eq.W4Tensor(codes.to(I8), scales, group=64),
                 lambda: eq.W4Tensor(codes, scales, scales, group=64)):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: eq.eq_w4_matvec(block, [x.to(E4M3)], [y], [s]), eq.EQ_EUNSUPPORTED),
                         (lambda: eq.eq_w4_matvec(block, [x.float()], [y]), eq.EQ_EINVAL),
                         (lambda: eq.eq_w4_matvec(block, [x], [y.to(I8)], None), None),
                         (lambda: eq.W4Tensor(codes, scales, group=48), eq.EQ_EINVAL),
                         (lambda: eq.W4Tensor(codes, scales, dtype=eq.EQ_DTYPE_BF16, group=64), eq.EQ_EINVAL),
                         (lambda: eq.W4Tensor(codes, scales, torch.zeros_like(scales, dtype=torch.uint8),
                                              dtype=eq.EQ_DTYPE_E2M1, group=64), eq.EQ_EINVAL)):
        with pytest.raises((eq.EqError, ValueError)) as e:
            call()
        assert status is None or e.value.status == status
