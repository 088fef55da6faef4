"""eq_add_rmsnorm and eq_silu_mul: every number of chunks a thread holds (NV: 1 to
4, and 0 for rows computed twice), for few rows and for many. The kernel's name is
read from a profile of the call, so that a change of the rule which moves a case to
another kernel shows here. Comparisons as in test_gpu_rownorm."""
import re

import pytest
import torch
from torch.profiler import ProfilerActivity, profile

from conftest import gpu_available
from gpu_util import log
from test_gpu_rownorm import BF16, E4M3, F32, I8, run_norm, run_silu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

# tokens, cols, NV
CASES = [(2, 8192, 1), (2, 8197, 2), (3, 16384, 2), (3, 16385, 3), (2, 20003, 3), (2, 24576, 3), (2, 24583, 4), (1, 32768, 4),
         (2, 32775, 0), (1030, 77, 1), (1024, 1027, 3), (1100, 5003, 3), (1025, 11008, 3), (1024, 6144, 3), (1030, 2050, 3),
         (1026, 700, 2), (1024, 24579, 4)]


def kernel_of(call):
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [int(m.group(1)) for m in (re.search(r"k_row<[^>]*, (\d+)>", e.name) for e in p.events()) if m]


@pytest.mark.parametrize("tokens,cols,nv", CASES)
def test_every_kernel(tokens, cols, nv):
    for out in (BF16, I8, E4M3):
        log(f"case row kernel {tokens} x {cols} -> {out}")
        ran = kernel_of(lambda: run_norm(tokens, cols, BF16, BF16, out, seed=cols))
        ran += kernel_of(lambda: run_norm(tokens, cols, F32, None, out, wt=F32, strides=True, seed=cols + 1))
        ran += kernel_of(lambda: run_silu(tokens, cols, BF16, out, seed=cols + 2))
        assert set(ran) <= {nv}, ran  # a profile may lack a launch
