"""The state space kernels on the paths that served sizes take, and their
edges: the same oracle and bounds as test_gpu_ssm.py, without an allowance."""
import numpy as np
import pytest
import torch

from .gpu_util import banner
from .test_gpu_ssm import DT, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("N", [32, 64, 128, 256])
def test_the_output_type_changes_the_last_rounding_only(gpu, io, N):
    # the same operands enter the products whatever y's type.  y of fp32 is the
    # last sum v rounded to fp32, so v lies between that value's two neighbours;
    # y of 16 bits is v rounded once (fp16: by the multiply-add that forms it) or
    # y of fp32 rounded again.  Rounding is monotone: either way it is not below
    # the lower neighbour's rounding nor above the upper one's.
    L = Layer([700, 65, 1], H=4, P=64, G=2, N=N, io=io, seed=21)
    banner("y of", io, "and of fp32, N", N)
    y, S = L.run_scan()
    y32, S32 = L.run_scan("f32")
    assert torch.equal(S, S32)
    lo, hi = (torch.nextafter(y32, torch.full_like(y32, v)).to(DT[io]) for v in (-np.inf, np.inf))
    wrong = int(((y < lo) | (y > hi) | (y != y)).sum())
    assert not wrong, f"{wrong} of {y.numel()} outputs rounded from something else"
