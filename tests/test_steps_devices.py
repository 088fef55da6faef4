"""The steps around the products on a GPU that is not the current one: a
call launches with its tensors' GPU current (the default stream's handle is 0 on
every GPU and means the current one's), and refuses tensors of several
GPUs. Checked without a GPU: tensors are stand-ins with a device number, and
the library is a recorder of the calls and of the device that was current."""
import contextlib

import pytest
import torch

from rans_decode_amd import eq

BF16, F32, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8


class Tensor:
    """What the binding asks of a tensor."""

    def __init__(self, *shape, dtype=F32, gpu=1):
        self.shape, self.dtype, self.gpu = torch.Size(shape), dtype, gpu
        self.is_cuda, self.device = gpu >= 0, torch.device("cuda", gpu) if gpu >= 0 else torch.device("cpu")

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return 1 << 20

    def is_contiguous(self):
        return True


class Stream:
    def __init__(self, gpu):
        self.device, self.cuda_stream = torch.device("cuda", gpu), 70 + gpu


@pytest.fixture
def gpus(monkeypatch):
    """Two pretended GPUs, 0 current; the calls made: (name, current GPU, stream handle)."""
    now, calls = [0], []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], torch.device(index).index if not isinstance(index, int) else index
        try:
            yield
        finally:
            now[0] = before

    class Library:
        def __getattr__(self, name):
            if name in ("eq_w4_groups", "eq_w4_codes_bytes"):
                return getattr(real, name)
            return lambda *args: calls.append((name, now[0], args[-1])) or eq.EQ_OK

    real = eq._lib
    monkeypatch.setattr(eq, "_lib", Library())
    monkeypatch.setattr(eq, "_raw_stream", lambda: lambda index: 40 + index)
    monkeypatch.setattr(eq, "_current_gpu", lambda: lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Tensor(64, dtype=k["dtype"], gpu=k["device"].index)
                        if getattr(k.get("device"), "type", "") == "cuda" else empty(*a, **k))
    yield calls
    assert now[0] == 0  # the caller's device is back


empty = torch.empty


def tensor4(gpu):
    return eq.W4Tensor(Tensor(32, 64, dtype=U8, gpu=gpu), Tensor(32, 2, dtype=BF16, gpu=gpu),
                       Tensor(32, 2, dtype=U8, gpu=gpu), group=64)


@pytest.mark.parametrize("gpu", [0, 1])
def test_launched_on_the_tensors_gpu(gpus, gpu):
    def t(*shape, dtype=F32):
        return Tensor(*shape, dtype=dtype, gpu=gpu)
    eq.eq_add_rmsnorm(t(4, 64), t(64, dtype=BF16), 1e-5, t(4, 64, dtype=I8), out_scale=t(4), residual=t(4, 64))
    eq.eq_silu_mul(t(4, 64), t(4, 64), t(4, 64, dtype=BF16))
    block = eq.W4Block([tensor4(gpu), tensor4(gpu)])
    eq.eq_w4_matvec(block, [t(4, 128, dtype=I8)] * 2, [t(4, 32)] * 2, [t(4)] * 2)
    assert gpus == [(name, gpu, 40 + gpu) for name in ("eq_add_rmsnorm", "eq_silu_mul", "eq_w4_pack", "eq_w4_pack", "eq_w4_matvec")]
    del gpus[:]
    eq.eq_silu_mul(t(4, 64), t(4, 64), t(4, 64, dtype=BF16), stream=Stream(gpu))
    eq.eq_silu_mul(t(4, 64), t(4, 64), t(4, 64, dtype=BF16), stream=12345)  # a handle: the caller's word
    assert gpus == [("eq_silu_mul", gpu, 70 + gpu), ("eq_silu_mul", gpu, 12345)]


@pytest.mark.parametrize("here,other", [(0, 1), (1, 0), (1, -1)])
def test_tensors_of_several_gpus_refused(gpus, here, other):
    def t(*shape, dtype=F32, gpu=here):
        return Tensor(*shape, dtype=dtype, gpu=gpu)
    norm = dict(x=t(4, 64), weight=t(64, dtype=BF16), eps=1e-5, out=t(4, 64, dtype=I8), out_scale=t(4), residual=t(4, 64),
                residual_out=t(4, 64))
    for name in ("x", "weight", "out", "out_scale", "residual", "residual_out"):
        moved = dict(norm)
        moved[name] = Tensor(*norm[name].shape, dtype=norm[name].dtype, gpu=other)
        with pytest.raises(ValueError):
            eq.eq_add_rmsnorm(**moved)
    silu = dict(gate=t(4, 64), up=t(4, 64), out=t(4, 64, dtype=I8), out_scale=t(4))
    for name in silu:
        moved = dict(silu)
        moved[name] = Tensor(*silu[name].shape, dtype=silu[name].dtype, gpu=other)
        with pytest.raises(ValueError):
            eq.eq_silu_mul(**moved)
    block = eq.W4Block([tensor4(here), tensor4(here)])
    del gpus[:]
    for at in range(2):  # one tensor's x, y or scales elsewhere
        for which in range(3):
            xs, ys, scales = [t(4, 128, dtype=I8)] * 2, [t(4, 32)] * 2, [t(4)] * 2
            lists = [xs, ys, scales]
            lists[which][at] = Tensor(*lists[which][at].shape, dtype=lists[which][at].dtype, gpu=other)
            with pytest.raises(ValueError):
                eq.eq_w4_matvec(block, xs, ys, scales)
    if other >= 0:  # the weights elsewhere, or a stream of another GPU
        for tensors in ([tensor4(here), tensor4(other)], [tensor4(other), tensor4(here)]):
            del gpus[:]
            with pytest.raises(ValueError):
                eq.eq_w4_matvec(eq.W4Block(tensors), [t(4, 128, dtype=I8)] * 2, [t(4, 32)] * 2, [t(4)] * 2)
        with pytest.raises(ValueError):
            eq.eq_silu_mul(t(4, 64), t(4, 64), t(4, 64, dtype=BF16), stream=Stream(other))
    assert not gpus
