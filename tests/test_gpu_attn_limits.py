"""The attention kernels at the ends of what include/gdn_attn.h supports: the largest and
the smallest scale.  Tolerances are those of test_gpu_attn.py."""
import numpy as np
import pytest
import torch

from .gpu_util import banner
from .test_gpu_attn import IO, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("op", ["prefill", "step"])
def test_the_largest_and_the_smallest_scale(gpu, io, op):
    """Queries of 0 see every key alike under any scale; and under the smallest one so does every query."""
    new = [1, 1] if op == "step" else [40, 3]
    for scale in (2.0 ** 127, 2.0 ** -149):
        banner("scale", io, op, scale)
        c = Case(new, [300, 5], 4, 2, 64, 16, io, scale=scale)
        c.scale = float(np.float32(scale))
        if scale > 1:
            c.qw.zero_()
        c.run_and_check(op)
        assert torch.isfinite(c.run(op)[:c.used]).all()
