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


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_that_is_not_finite_leaves_the_tokens_before_it(gpu, io, N, bad):
    # one bad value of x, B, C or dt at places all over a chunk, in the first
    # segment and in a later one: outputs before it, of other sequences and (x, dt)
    # of other channels or heads are bit for bit those of the clean inputs
    H, P = 4, 64
    L = Layer([130, 600, 77], H=H, P=P, G=2, N=N, io=io, seed=22)
    L.A_log.fill_(-3.0)  # decays that keep the value in the state to the end
    clean_x, clean_dt = L.xbc.clone(), L.dt.clone()
    for out in sorted({io, "f32"}):
        L.xbc.copy_(clean_x), L.dt.copy_(clean_dt)
        y0, S0 = L.run_scan(out)
        banner("not finite", io, out, N, bad)
        for t in (0, 1, 17, 31, 32, 47, 63, 64, 300, 511, 575, 599):
            at, end = 130 + t, 730
            for what, col in (("x", 2 * P + 37), ("B", H * P + 5), ("C", H * P + 2 * N + N + 9), ("dt", 3)):
                L.xbc.copy_(clean_x), L.dt.copy_(clean_dt)
                (L.dt if what == "dt" else L.xbc)[at, col] = bad
                y, S = L.run_scan(out)
                same = y == y0
                assert same[:at].all() and same[end:].all(), (what, t)
                assert torch.equal(S[0], S0[0]) and torch.equal(S[2], S0[2])
                if what == "x":
                    same[at:end, 2, 37] = True
                    assert not torch.isfinite(y[at, 2, 37]) and not torch.isfinite(S[1, 2, 37]).any()
                elif what == "dt":
                    same[at:end, 3] = True
                    assert not torch.isfinite(y[at, 3]).any()
                elif what == "B":
                    same[at:end, :2] = True
                    assert not torch.isfinite(y[at, :2]).any()
                else:
                    same[at, 2:] = True
                    assert not torch.isfinite(y[at, 2:]).any()
                assert same.all(), (what, t)


def test_fp16_scan_of_a_state_far_above_its_inputs(gpu):
    # states of 2^100 that hardly decay, then inputs that are the smallest of fp16:
    # everything stays inside fp32's range, so does the scan
    for lens in ([200, 3], [700]):
        L = Layer(lens, H=2, G=1, io="f16", seed=23)
        L.state *= 2.0 ** 100
        L.A_log.fill_(-12.0)
        L.xbc[:, :2 * 64] *= 2.0 ** -22
        banner("gdn_ssm_scan of large states", lens)
        y, S = L.run_scan("f32")
        L.check_scan(y, S, "f32")


def test_fp16_scan_of_steps_far_above_one(gpu):
    # steps of 1e19 with decays of e^-1.35 a token: what the last 64 tokens of a
    # segment of 128 leave in its state is 2^124 times what the first ones do
    L = Layer([900, 40], H=2, P=64, G=1, io="f16", seed=24)
    L.dt_bias.fill_(1e19)
    L.A_log.fill_(-43.45)
    L.xbc[:, :2 * 64 + 128] *= 1e4
    assert L.xbc.isfinite().all()
    banner("gdn_ssm_scan of large steps")
    y, S = L.run_scan("f32")
    L.check_scan(y, S, "f32")
