"""One token through the second half of a transformer block, as a serving loop
runs it: the entropy-coded output projection, the residual's addition and
norm, a 4-bit MLP with int8 activations, and the norm that feeds the next
block's entropy-coded projections.

    python examples/w4_mlp.py [--hidden 1024] [--inner 2816] [--group 128] [--steps 50]

    attention output (bf16)
      -> eq_decode_gemv_bf16    o projection, weights entropy-coded      fp32
      -> eq_add_rmsnorm         residual += o; norm                      int8 + scale
      -> eq_w4_matvec           gate and up in one call, INT4 weights    fp32
      -> eq_silu_mul            silu(gate) * up                          int8 + scale
      -> eq_w4_matvec           down                                     fp32
      -> eq_add_rmsnorm         residual += down; norm                   bf16

Weights are random. The result is compared with the same steps in 64 bits on
the same quantised weights; what differs is the rounding of the activations. With
--steps N the step is also captured in a HIP graph and timed over N replays.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rans_decode_amd import eq  # noqa: E402

EPS = 1e-5


def quantize_int4(w: torch.Tensor, group: int):
    """Signed 4-bit codes (two a byte, the lower half first) and one bf16 scale
    per `group` columns: scale = max|w| / 7, code = round(w / scale)."""
    rows, cols = w.shape
    groups = -(-cols // group)
    padded = torch.nn.functional.pad(w, (0, groups * group - cols)).view(rows, groups, group)
    scales = (padded.abs().amax(dim=2) / 7).clamp_min(2.0 ** -100).to(torch.bfloat16)
    q = torch.round(padded / scales.float()[:, :, None]).clamp(-8, 7).to(torch.int16).view(rows, -1)[:, :cols + cols % 2] & 15
    return (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8).contiguous(), scales


def dequantize_int4(codes: torch.Tensor, scales: torch.Tensor, cols: int, group: int) -> torch.Tensor:
    q = torch.stack([codes & 15, codes >> 4], dim=2).flatten(1)[:, :cols].to(torch.int16)
    q = torch.where(q > 7, q - 16, q).double()
    return q * scales.double()[:, torch.arange(cols, device=codes.device) // group]


class Block:
    """The weights of one half block, laid out once."""

    def __init__(self, hidden: int, inner: int, group: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.hidden, self.inner, self.group = hidden, inner, group
        # output projection: low-entropy int8 codes with a scale per row, entropy-coded in whole-row chunks
        codes = torch.randn(hidden, hidden, generator=g).mul_(1.5).round_().clamp_(-127, 127).to(torch.int8).numpy().view(np.uint8)
        scales = np.full(hidden, 0.5 / hidden ** 0.5, np.float32)
        rows_per_chunk = max(1, 16384 // hidden)
        blob = eq.encode_host(eq.build_tables(codes.ravel()), eq.EQ_DTYPE_INT8, hidden, hidden, codes.ravel(), scales,
                              chunk_symbols=rows_per_chunk * hidden)
        self.o = eq.Block([eq.DeviceContainer(blob)])
        self.o64 = (torch.from_numpy(codes.view(np.int8)).float() * torch.from_numpy(scales)[:, None]).to(torch.bfloat16).double().cuda()
        # gate, up, down: 4 bits
        self.mlp64, packed = [], []
        for rows, cols in ((inner, hidden), (inner, hidden), (hidden, inner)):
            c, s = quantize_int4((torch.randn(rows, cols, generator=g) / cols ** 0.5).cuda(), group)
            self.mlp64.append(dequantize_int4(c, s, cols, group))
            packed.append(eq.W4Tensor(c, s, group=group, cols=cols))
        self.gate_up, self.down = eq.W4Block(packed[:2]), eq.W4Block(packed[2:])
        self.norm1, self.norm2 = ((1 + 0.1 * torch.randn(hidden, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
        # buffers of one step
        new = lambda n, t: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
        self.y, self.a, self.a_scale = new(hidden, torch.float32), new(hidden, torch.int8), new(1, torch.float32)
        self.g, self.u = new(inner, torch.float32), new(inner, torch.float32)
        self.h, self.h_scale = new(inner, torch.int8), new(1, torch.float32)
        self.out = new(hidden, torch.bfloat16)

    def step(self, attention: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        """attention: bf16 [hidden]; residual: fp32 [hidden], updated in place.
        Returns the next block's input (bf16 [hidden], this object's buffer)."""
        eq.eq_decode_gemv_bf16(self.o, [attention], [self.y])
        eq.eq_add_rmsnorm(self.y, self.norm1, EPS, self.a, out_scale=self.a_scale, residual=residual)
        eq.eq_w4_matvec(self.gate_up, [self.a, self.a], [self.g, self.u], [self.a_scale, self.a_scale])
        eq.eq_silu_mul(self.g, self.u, self.h, out_scale=self.h_scale)
        eq.eq_w4_matvec(self.down, [self.h], [self.y], [self.h_scale])
        eq.eq_add_rmsnorm(self.y, self.norm2, EPS, self.out, residual=residual)
        return self.out

    def step64(self, attention: torch.Tensor, residual: torch.Tensor):
        """The same in 64 bits, without rounding activations; returns (output, residual)."""
        def norm(x, w):
            return x / torch.sqrt((x * x).mean() + EPS) * w.double()
        r = residual.double() + self.o64 @ attention.double()
        a = norm(r, self.norm1)
        g, u = self.mlp64[0] @ a, self.mlp64[1] @ a
        r = r + self.mlp64[2] @ (g * torch.sigmoid(g) * u)
        return norm(r, self.norm2), r


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=2816)
    ap.add_argument("--group", type=int, default=128, choices=(32, 64, 128))
    ap.add_argument("--steps", type=int, default=0, help="time this many graph replays of the step")
    args = ap.parse_args(argv)
    block = Block(args.hidden, args.inner, args.group)
    attention = torch.randn(args.hidden, device="cuda").to(torch.bfloat16)
    residual = torch.randn(args.hidden, device="cuda")
    want, want_residual = block.step64(attention, residual)
    got = block.step(attention, residual)
    torch.cuda.synchronize()
    off = float((got.double() - want).norm() / want.norm())
    off_residual = float((residual.double() - want_residual).norm() / want_residual.norm())
    print(f"hidden {args.hidden}, inner {args.inner}, group {args.group}: output {off:.2e}, residual {off_residual:.2e} "
          "from the same step in 64 bits (2-norm)")
    if args.steps > 0:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block.step(attention, residual)
        graph.replay()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(args.steps):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"{begin.elapsed_time(end) * 1e3 / args.steps:.1f} us per step (6 kernels, one graph)")
    return off, off_residual


if __name__ == "__main__":
    main()
