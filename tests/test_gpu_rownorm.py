"""eq_add_rmsnorm and eq_silu_mul against their formulas in 64 bits.

Tolerances. fp32 evaluation: a thread adds at most cols / 1024 + 32 squares in
a row and the tree adds fewer than 32 partial sums, so for the widths here the
mean is within 2^-16.5 of its value, its root within 2^-17.5, and four more
roundings and a 1-ulp reciprocal root keep y within E = 2^-16 (relative). A bf16
output lies between the roundings of y's lowest and highest such value; on
top of the error of y int8 rounds by half a step of the scale and E4M3 by
2^-4 (half a step of 3 bits) or 2^-10 steps of the scale near zero.
silu: exp(-g) is off by at most (|g| + 4) 2^-23, a reciprocal and two products
by 4 * 2^-23 more. The stored sum is one fp32 addition rounded once: exact.
"""
import numpy as np
import pytest
import torch

from conftest import gpu_available
from gpu_util import log
from rans_decode_amd import eq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

F32, BF16, I8, E4M3 = torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn
LARGEST = {I8: 127.0, E4M3: 448.0}
E = 2.0 ** -16
# cols around the chunk of 8, a wave's 512, the workgroup sizes and the limit of rows in registers (32768)
COLS = [1, 2, 7, 8, 9, 63, 511, 512, 513, 1000, 4096, 5003, 8192, 8193, 11008, 28672, 32768, 32769, 40003]


def rows_of(seed, tokens, cols, dtype, stride=None):
    """[tokens, cols] values of hidden-state size in rows of `stride` elements (the gaps hold NaN)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, cols, generator=g)
    x[:, torch.randint(cols, (1 + cols // 1000,), generator=g)] *= 30
    if tokens > 2:
        x[tokens // 2] = 0
    stride = stride or cols
    buf = torch.full((max(tokens, 1), stride), float("nan"), dtype=dtype)
    buf[:tokens, :cols] = x.to(dtype)
    return buf.cuda()[:tokens, :cols]


def outputs(tokens, cols, out, stride=None):
    buf = torch.empty(max(tokens, 1), stride or cols, dtype=out, device="cuda")
    buf.view(torch.uint8).fill_(0x55)
    scale = torch.full((tokens,), float("nan"), device="cuda") if out in LARGEST else None
    return buf[:tokens, :cols], scale, buf


def between_roundings(got, y, off):
    """Whether every got is a bf16 rounding of a value within `off` of y (rounding is monotone)."""
    low, high = (torch.from_numpy(v).to(BF16).double().numpy() for v in (y - off, y + off))
    return bool(((low <= got) & (got <= high)).all())


def check_out(y, rel, out, scale, what):
    """out (and scale) against the 64-bit y, `rel` off at most before the last rounding."""
    got = out.cpu().to(torch.float32).double().numpy()
    y = y.numpy()
    rel = rel.numpy() if isinstance(rel, torch.Tensor) else rel
    if scale is None:
        assert between_roundings(got, y, 2 * rel * np.abs(y) + 2.0 ** -120), what
        return
    L = LARGEST[out.dtype]
    amax = np.maximum(np.abs(y).max(axis=1), 2.0 ** -96)
    worst = np.max(rel) if np.size(rel) else 0
    s = scale.cpu().double().numpy()
    assert (np.abs(s - amax / L) <= (2 * worst + 2.0 ** -22) * amax / L).all(), what
    assert np.isfinite(got).all() and (np.abs(got) <= L).all(), what
    step = (2 * worst + 2.0 ** -20) * amax[:, None]  # what the row's scale and values may be off
    half = 0.5 * s[:, None] if out.dtype == I8 else np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s[:, None])
    assert (np.abs(got * s[:, None] - y) <= half * (1 + 2.0 ** -10) + step).all(), what
    live = np.abs(y).max(axis=1) > 2.0 ** -96
    assert (np.abs(got).max(axis=1)[live] == L).all(), f"{what}: the largest value takes the largest code"


def run_norm(tokens, cols, xt, rt, out, wt=BF16, strides=False, in_place=False, seed=0, eps=1e-5):
    st = cols + 3 if strides else None
    x = rows_of(seed, tokens, cols, xt, st)
    res = rows_of(seed + 1, tokens, cols, rt, cols + 5 if strides else None) if rt else None
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed + 2))).to(wt).cuda() if wt else None
    o, scale, buf = outputs(tokens, cols, out, cols + 11 if strides else None)
    s32 = x.cpu().float() + (res.cpu().float() if rt else 0)
    s = s32.to(rt) if rt else s32
    res_out = None
    if rt and not in_place:
        res_out = outputs(tokens, cols, rt, cols + 1 if strides else None)[0]
    eq.eq_add_rmsnorm(x, w, eps, o, out_scale=scale, residual=res, residual_out=res_out)
    torch.cuda.synchronize()
    what = f"norm {tokens}x{cols} {xt} {rt} -> {out}"
    if rt:
        got = (res if in_place else res_out).cpu()
        assert torch.equal(got.view(torch.int16 if rt == BF16 else torch.int32),
                           s.view(torch.int16 if rt == BF16 else torch.int32)), what
    s = s.double()
    y = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps) * (w.cpu().double() if wt else 1.0)
    check_out(y, E, o, scale, what)
    if strides:  # the gaps between rows are left alone
        gap = buf.view(torch.uint8).cpu()[:, cols * o.element_size():]
        assert (gap == 0x55).all(), what


@pytest.mark.parametrize("cols", COLS)
def test_norm_widths(cols):
    log(f"case norm width {cols}")
    for out in (BF16, I8, E4M3):
        run_norm(3, cols, BF16, BF16, out, seed=cols)
        run_norm(1, cols, F32, None, out, seed=cols + 1)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("rt", [None, F32, BF16])
@pytest.mark.parametrize("out", [BF16, I8, E4M3])
def test_norm_types_strides_and_places(xt, rt, out):
    log(f"case norm types {xt} {rt} {out}")
    for tokens, cols in ((1, 4096), (5, 1003), (2, 33000), (17, 72)):
        run_norm(tokens, cols, xt, rt, out, wt=F32, strides=True, seed=tokens)
        run_norm(tokens, cols, xt, rt, out, wt=None, in_place=rt is not None, seed=tokens + 7)


def test_norm_many_tokens():
    """More rows than one grid dimension takes."""
    tokens, cols = (1 << 20) + 5, 8
    log("case norm many tokens")
    x = torch.randn(tokens, cols, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    o = torch.empty(tokens, cols, dtype=BF16, device="cuda")
    eq.eq_add_rmsnorm(x, None, 0.0, o)
    y = x.double() / torch.sqrt((x.double() ** 2).mean(dim=1, keepdim=True))
    assert between_roundings(o.cpu().double().numpy(), y.cpu().numpy(), 2 * E * np.abs(y.cpu().numpy()))


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes apart, inputs and outputs, both kernels."""
    log("case rows far apart")
    tokens, cols, step = 3, 1003, (1 << 31) + 6
    def far(dtype):
        return torch.empty((tokens - 1) * step + cols, dtype=dtype, device="cuda").as_strided((tokens, cols), (step, 1))
    near = rows_of(4, tokens, cols, BF16)
    x, r, ro, o, o8 = far(BF16), far(BF16), far(BF16), far(BF16), far(I8)
    x.copy_(near)
    r.copy_(near)
    scale, want_scale = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    want, want_r, want8 = torch.empty_like(near), torch.empty_like(near), torch.empty(tokens, cols, dtype=I8, device="cuda")
    eq.eq_add_rmsnorm(near, None, 1e-5, want, residual=near, residual_out=want_r)
    eq.eq_add_rmsnorm(x, None, 1e-5, o, residual=r, residual_out=ro)
    eq.eq_silu_mul(near, near, want8, out_scale=want_scale)
    eq.eq_silu_mul(x, r, o8, out_scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(ro, want_r) and torch.equal(o8, want8) and torch.equal(scale, want_scale)
    del x, r, ro, o, o8
    torch.cuda.empty_cache()


def test_norm_rows_of_zeros_and_tiny_values():
    log("case norm zeros")
    for scale_of, cols in ((0.0, 100), (2.0 ** -110, 100), (2.0 ** -140, 64)):
        x = torch.ones(4, cols, device="cuda") * scale_of
        for out in (BF16, I8, E4M3):
            o, s, _ = outputs(4, cols, out)
            eq.eq_add_rmsnorm(x, None, 1e-6, o, out_scale=s)
            torch.cuda.synchronize()
            assert torch.isfinite(o.float()).all()
            if s is not None:
                assert torch.isfinite(s).all() and (s > 0).all()
                if scale_of < 2.0 ** -130:
                    assert (o.float() == 0).all()  # below the floor's half step


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_values_stay_in_their_row(bad):
    log(f"case bad values {bad}")
    for cols in (100, 4096, 33000):
        x = rows_of(1, 5, cols, F32)
        x[2] = 1.0
        clean = x.clone()
        x[3, cols // 2] = bad
        for out in (BF16, I8, E4M3):
            pairs = []
            for src in (clean, x):
                o, s, _ = outputs(5, cols, out)
                eq.eq_add_rmsnorm(src, None, 1e-5, o, out_scale=s)
                h, hs, _ = outputs(5, cols, out)
                eq.eq_silu_mul(src, src, h, out_scale=hs)
                torch.cuda.synchronize()
                pairs.append((o.float(), s, h.float(), hs))
            keep = [0, 1, 2, 4]
            for a, b in zip(*pairs):
                assert a is None or torch.equal(a[keep], b[keep])
            o, s, h, hs = pairs[1]
            if out == BF16:
                assert torch.isnan(o[3, cols // 2]) and not torch.isfinite(h[3, cols // 2])
            else:
                assert not torch.isfinite(s[3]) and not torch.isfinite(hs[3])


def run_silu(tokens, cols, xt, out, strides=False, seed=0, spread=3.0):
    x = rows_of(seed, tokens, 2 * cols, xt, 2 * cols + 3) if strides else None
    gate = x[:, :cols] if strides else rows_of(seed, tokens, cols, xt)
    up = x[:, cols:] if strides else rows_of(seed + 1, tokens, cols, xt)
    if not strides:
        gate.mul_(spread)
    o, scale, buf = outputs(tokens, cols, out, cols + 5 if strides else None)
    eq.eq_silu_mul(gate, up, o, out_scale=scale)
    torch.cuda.synchronize()
    g, u = gate.cpu().double(), up.cpu().double()
    rel = (g.abs() + 8) * 2.0 ** -23
    check_out(g / (1 + torch.exp(-g)) * u, rel, o, scale, f"silu {tokens}x{cols} {xt} -> {out}")
    if strides:
        assert (buf.view(torch.uint8).cpu()[:, cols * o.element_size():] == 0x55).all()


@pytest.mark.parametrize("cols", COLS)
def test_silu_widths(cols):
    log(f"case silu width {cols}")
    for out in (BF16, I8, E4M3):
        run_silu(3, cols, BF16, out, seed=cols)
        run_silu(1, cols, F32, out, seed=cols + 1)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("out", [BF16, I8, E4M3])
def test_silu_halves_of_one_buffer(xt, out):
    log(f"case silu halves {xt} {out}")
    for tokens, cols in ((1, 4096), (5, 1003), (2, 33000), (17, 72)):
        run_silu(tokens, cols, xt, out, strides=True, seed=tokens)


def test_silu_far_values():
    """Gates where exp(-g) overflows or vanishes."""
    log("case silu far values")
    g = torch.tensor([-1e30, -200.0, -100.0, -88.0, -20.0, -0.0, 0.0, 20.0, 88.0, 100.0, 1e30], device="cuda")
    o = torch.empty(11, dtype=BF16, device="cuda")
    eq.eq_silu_mul(g, torch.ones_like(g), o)
    torch.cuda.synchronize()
    got = o.float().cpu().numpy().astype(np.float64)
    v = g.cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        want = v / (1 + np.exp(-v))
    assert between_roundings(got, want, (np.minimum(np.abs(v), 128) + 8) * 2.0 ** -22 * np.abs(want) + 1e-34)


def test_no_tokens_and_other_streams():
    log("case no tokens")
    e = torch.empty(0, 64, device="cuda")
    eq.eq_add_rmsnorm(e, None, 1e-5, torch.empty(0, 64, dtype=BF16, device="cuda"))
    eq.eq_silu_mul(e, e, torch.empty(0, 64, dtype=BF16, device="cuda"))
    log("case another stream")
    x = rows_of(5, 64, 2048, BF16)
    want = torch.empty(64, 2048, dtype=BF16, device="cuda")
    eq.eq_add_rmsnorm(x, None, 1e-5, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    eq.eq_add_rmsnorm(x, None, 1e-5, got, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.stream(side):
        again = torch.zeros_like(want)
        eq.eq_add_rmsnorm(x, None, 1e-5, again)
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(want, again)


def test_results_do_not_change_between_runs():
    log("case repeat")
    x = rows_of(6, 9, 28672, F32)
    first = None
    for _ in range(5):
        o, s, _ = outputs(9, 28672, I8)
        eq.eq_add_rmsnorm(x, None, 1e-5, o, out_scale=s)
        torch.cuda.synchronize()
        got = (o.cpu(), s.cpu())
        first = first or got
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


def test_wrapper_refusals():
    x = torch.zeros(4, 64, device="cuda")
    o = torch.zeros(4, 64, dtype=I8, device="cuda")
    b = torch.zeros(4, 64, dtype=BF16, device="cuda")
    s = torch.zeros(4, device="cuda")
    for call in (lambda: eq.eq_add_rmsnorm(x, None, 1e-5, o),                              # no scales
                 lambda: eq.eq_add_rmsnorm(x, None, 1e-5, o, out_scale=s[:3]),
                 lambda: eq.eq_add_rmsnorm(x, None, 1e-5, b, out_scale=s),                 # scales of a bf16 output
                 lambda: eq.eq_add_rmsnorm(x, s, 1e-5, b),                                 # weight of another width
                 lambda: eq.eq_add_rmsnorm(x, None, 1e-5, b[:3]),
                 lambda: eq.eq_add_rmsnorm(x.t(), None, 1e-5, torch.zeros(64, 4, dtype=BF16, device="cuda")),
                 lambda: eq.eq_add_rmsnorm(x, None, 1e-5, b, residual_out=b),
                 lambda: eq.eq_add_rmsnorm(x.double(), None, 1e-5, b),
                 lambda: eq.eq_add_rmsnorm(x.cpu(), None, 1e-5, b),
                 lambda: eq.eq_silu_mul(x, x[:, :63], b),
                 lambda: eq.eq_silu_mul(x, x.cpu(), b)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: eq.eq_add_rmsnorm(x, None, -1.0, b),
                 lambda: eq.eq_add_rmsnorm(x, None, float("nan"), b),
                 lambda: eq.eq_add_rmsnorm(x, None, 1e-5, x),                              # fp32 output
                 lambda: eq.eq_silu_mul(x, b, b),                                          # types differ
                 lambda: eq.eq_add_rmsnorm(x[:, :0], None, 1e-5, b[:, :0]),
                 lambda: eq.eq_add_rmsnorm(x[:1].expand(4, 64), None, 1e-5, b)):           # rows on top of each other
        with pytest.raises(eq.EqError) as e:
            call()
        assert e.value.status == eq.EQ_EINVAL
