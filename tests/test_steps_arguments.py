"""Argument checks of eq_add_rmsnorm, eq_silu_mul, eq_w4_pack and eq_w4_matvec:
each refusal is made on the host before any HIP call, so it runs without a
GPU. Pointers are plain numbers that nothing reads."""
import ctypes

import pytest

from rans_decode_amd import eq

L = eq._lib
P = 1 << 20  # a 16-byte aligned address
BF16, F32, I8, E4M3, INT4, E2M1 = (eq.EQ_DTYPE_BF16, eq.EQ_DTYPE_F32, eq.EQ_DTYPE_INT8, eq.EQ_DTYPE_E4M3,
                                   eq.EQ_DTYPE_INT4, eq.EQ_DTYPE_E2M1)


def m(dtype, stride=64, d=P, scale=0, reserved=0):
    return eq._pack_matrix(d, stride, scale, dtype, reserved)


def norm(x=m(BF16), r=None, ro=None, w=P, wt=BF16, eps=1e-5, tokens=4, cols=64, out=m(BF16)):
    return L.eq_add_rmsnorm(x, r, ro, w, wt, eps, tokens, cols, out, None)


def silu(g=m(F32), u=m(F32), tokens=4, cols=64, out=m(BF16)):
    return L.eq_silu_mul(g, u, tokens, cols, out, None)


BAD_MATRICES = [None, m(BF16, d=0), m(BF16, stride=63), m(BF16, stride=1 << 41), m(BF16, d=P + 1), m(F32, d=P + 2),
                m(BF16, reserved=1), m(0), m(7), m(INT4), m(E2M1)]


def test_norm_refusals():
    for bad in BAD_MATRICES:
        assert norm(x=bad) == eq.EQ_EINVAL
        assert norm(out=bad) == eq.EQ_EINVAL
        if bad is not None:
            assert norm(r=bad, ro=bad) == eq.EQ_EINVAL
    assert norm(x=m(I8, scale=P)) == eq.EQ_EINVAL           # 8-bit input
    assert norm(out=m(F32)) == eq.EQ_EINVAL
    for t in (I8, E4M3):
        assert norm(out=m(t)) == eq.EQ_EINVAL               # no scales
        assert norm(out=m(t, scale=P + 2)) == eq.EQ_EINVAL
    assert norm(r=m(BF16)) == eq.EQ_EINVAL                  # one of the two
    assert norm(ro=m(BF16)) == eq.EQ_EINVAL
    assert norm(r=m(BF16), ro=m(F32)) == eq.EQ_EINVAL
    assert norm(r=m(I8, scale=P), ro=m(I8, scale=P)) == eq.EQ_EINVAL
    assert norm(wt=I8) == eq.EQ_EINVAL
    assert norm(w=P + 1) == eq.EQ_EINVAL
    assert norm(w=P + 2, wt=F32) == eq.EQ_EINVAL
    for eps in (-1e-9, float("nan"), float("-inf")):
        assert norm(eps=eps) == eq.EQ_EINVAL
    for cols in (0, 1 << 31):
        assert norm(x=m(BF16, 1 << 32), out=m(BF16, 1 << 32), cols=cols) == eq.EQ_EINVAL
    assert norm(tokens=1 << 31) == eq.EQ_EINVAL
    assert norm(tokens=0) == eq.EQ_OK
    assert norm(tokens=0, x=m(BF16, d=0), out=m(BF16, d=0)) == eq.EQ_OK


def test_silu_refusals():
    for bad in BAD_MATRICES:
        assert silu(g=bad) == eq.EQ_EINVAL
        assert silu(u=bad) == eq.EQ_EINVAL
        assert silu(out=bad) == eq.EQ_EINVAL
    assert silu(u=m(BF16)) == eq.EQ_EINVAL                  # gate and up of different types
    assert silu(out=m(E4M3)) == eq.EQ_EINVAL
    assert silu(out=m(F32)) == eq.EQ_EINVAL
    assert silu(cols=0) == eq.EQ_EINVAL
    assert silu(tokens=1 << 31) == eq.EQ_EINVAL
    assert silu(tokens=0) == eq.EQ_OK


def w4(dtype=INT4, group=64, rows=32, cols=128, codes=P, scales=P, zeros=None):
    return eq.eq_w4_tensor(dtype, group, rows, cols, codes, scales, zeros)


BAD_TENSORS = [dict(dtype=I8), dict(dtype=0), dict(group=0), dict(group=16), dict(group=96), dict(group=256), dict(rows=0),
               dict(cols=0), dict(rows=1 << 31), dict(cols=1 << 31), dict(codes=0), dict(scales=0), dict(codes=P + 8),
               dict(scales=P + 4), dict(zeros=P + 2), dict(dtype=E2M1, zeros=P)]


def matvec(tensors, xs, ys, tokens=2):
    arr = (eq.eq_w4_tensor * len(tensors))(*tensors)
    return L.eq_w4_matvec(arr, len(tensors), b"".join(xs), b"".join(ys), tokens, None)


@pytest.mark.parametrize("bad", BAD_TENSORS)
def test_w4_tensors_refused(bad):
    assert L.eq_w4_pack(ctypes.byref(w4(**bad)), P, P, P if bad.get("zeros") else None, None) == eq.EQ_EINVAL
    x, y = m(BF16, 1 << 32), m(F32, 1 << 32)
    assert matvec([w4(**bad)], [x], [y]) == eq.EQ_EINVAL
    assert matvec([w4(), w4(**bad)], [x, x], [y, y]) == eq.EQ_EINVAL  # nothing of the first is enqueued either


def test_w4_pack_refusals():
    t = w4()
    assert L.eq_w4_pack(None, P, P, None, None) == eq.EQ_EINVAL
    assert L.eq_w4_pack(ctypes.byref(t), None, P, None, None) == eq.EQ_EINVAL
    assert L.eq_w4_pack(ctypes.byref(t), P, None, None, None) == eq.EQ_EINVAL
    assert L.eq_w4_pack(ctypes.byref(t), P, P + 1, None, None) == eq.EQ_EINVAL
    assert L.eq_w4_pack(ctypes.byref(t), P, P, P, None) == eq.EQ_EINVAL         # zeros without a place for them
    assert L.eq_w4_pack(ctypes.byref(w4(zeros=P)), P, P, None, None) == eq.EQ_EINVAL
    huge = w4(rows=1 << 20, cols=1 << 20)                                        # more tiles than one launch takes
    assert L.eq_w4_pack(ctypes.byref(huge), P, P, None, None) == eq.EQ_EINVAL


def test_w4_matvec_refusals():
    x, y, t = m(BF16, 128), m(F32, 32), w4()
    assert L.eq_w4_matvec(None, 1, x, y, 2, None) == eq.EQ_EINVAL
    assert L.eq_w4_matvec(ctypes.byref(t), 1, None, y, 2, None) == eq.EQ_EINVAL
    assert L.eq_w4_matvec(ctypes.byref(t), 1, x, None, 2, None) == eq.EQ_EINVAL
    for bad in (m(BF16, 127), m(BF16, 128, d=0), m(BF16, 128, d=P + 1), m(BF16, 128, reserved=1), m(F32, 128),
                m(I8, 128), m(I8, 128, scale=P + 2), m(BF16, 1 << 41)):
        assert matvec([t], [bad], [y]) == eq.EQ_EINVAL
    for bad in (m(F32, 31), m(F32, 32, d=0), m(F32, 32, d=P + 2), m(BF16, 32, d=P + 1), m(I8, 32, scale=P), m(F32, 1 << 41)):
        assert matvec([t], [x], [bad]) == eq.EQ_EINVAL
    assert matvec([t], [m(E4M3, 128, scale=P)], [y]) == eq.EQ_EUNSUPPORTED
    assert matvec([w4(dtype=E2M1)], [m(I8, 128, scale=P)], [y]) == eq.EQ_EUNSUPPORTED
    assert matvec([t], [x], [y], tokens=64 * 65535 + 1) == eq.EQ_EINVAL
    assert matvec([w4(rows=8388593)], [x], [m(F32, 1 << 32)]) == eq.EQ_EINVAL
    assert matvec([w4(rows=8388592)], [x], [m(F32, 1 << 32)], tokens=0) == eq.EQ_OK
    assert matvec([t], [m(BF16, 128, d=0)], [m(F32, 32, d=0)], tokens=0) == eq.EQ_OK
    assert L.eq_w4_matvec(None, 0, None, None, 2, None) == eq.EQ_OK


def test_w4_sizes():
    assert L.eq_w4_codes_bytes(1, 1) == 1024
    assert L.eq_w4_codes_bytes(17, 129) == 4 * 1024
    assert L.eq_w4_codes_bytes(28672, 8192) == 28672 * 8192 // 2
    assert L.eq_w4_groups(17, 129, 32) == 4 * 16 * 4
    assert L.eq_w4_groups(28672, 8192, 128) == 28672 * 64
    for rows, cols, group in ((0, 1, 32), (1, 0, 32), (1 << 31, 1, 32), (1, 1, 33)):
        assert L.eq_w4_groups(rows, cols, group) == 0
    assert L.eq_w4_codes_bytes(0, 5) == 0 and L.eq_w4_codes_bytes(5, 0) == 0


def test_structures_match_the_header():
    assert ctypes.sizeof(eq.eq_w4_tensor) == 48
    assert len(m(BF16)) == 32
