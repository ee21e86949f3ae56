"""The state space kernels on the paths that served sizes take, and their
edges, against the oracle's bounds on an fp32 evaluation plus half a step of the
stored type, with no allowance for 16-bit y."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_pre_amd import ssm
from oracle import ssm_oracle as orc

from .gpu_util import banner
from .test_gpu_ssm import DT, Guard, Layer, check, f64

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


def held(L, y, S, out):
    """y and S inside the bounds of an fp32 evaluation, y rounded once."""
    dt, lam = L.steps()
    ry, ey, rS, eS = orc.scan(L.cu, f64(L.xbc), dt, lam, f64(L.D), f64(L.state), *L.dims())
    check("state", S, rS, orc.rounded(rS, eS, "f32"))
    check("y", y[:L.used], ry[:L.used], orc.rounded(ry, ey, out)[:L.used])


def _slow(L):
    """Every other head decays by a few thousandths of a log a token: nothing fades."""
    L.A_log[::2] = float(np.log(0.02))
    return L


# Segments of a 512th of tokens x heads x row tiles: 384 tokens and more, so that
# the walk over a segment from its end takes its decays in several batches of
# 256; heads in another order for each segment; up to 7 segments, and more.
LONG = [
    # lens, H, P, G, N
    ([1500, 1317, 200], 64, 32, 8, 32),
    ([3001], 64, 16, 4, 32),
    ([4700], 64, 16, 2, 32),
    ([1500, 1317, 200], 64, 16, 8, 128),
    ([1100, 900], 32, 80, 4, 32),
    ([2200, 300], 16, 256, 2, 32),
    ([1700, 411], 48, 64, 3, 64),
]


@pytest.mark.parametrize("io,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("lens,H,P,G,N", LONG, ids=[f"{max(c[0])}-H{c[1]}P{c[2]}N{c[4]}" for c in LONG])
def test_scan_of_long_segments_and_many_heads(gpu, io, out, lens, H, P, G, N):
    L = _slow(Layer(lens, H=H, P=P, G=G, N=N, io=io, seed=25, tail=2))
    banner("gdn_ssm_scan", io, out, lens, H, P, G, N)
    y, S = L.run_scan(out)
    held(L, y, S, out)
    S2 = L.state.clone()  # state updated in place: bit for bit the same
    y2, _ = L.run_scan(out, state=S2, state_out=S2)
    assert torch.equal(y[:L.used], y2[:L.used]) and torch.equal(S, S2)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_scan_of_long_segments_with_the_largest_state(gpu, io):
    L = _slow(Layer([1300, 813], H=64, P=16, G=8, N=256, io=io, seed=29))
    banner("gdn_ssm_scan", io, "N 256")
    y, S = L.run_scan("f32")
    held(L, y, S, "f32")


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,H,P,G,N", [
    ([70, 1, 0, 130, 33], 24, 64, 3, 64), ([65, 64], 16, 128, 4, 32), ([90, 31], 8, 144, 8, 32),
])
def test_scan_of_many_heads_in_one_piece(gpu, io, lens, H, P, G, N):
    L = _slow(Layer(lens, H=H, P=P, G=G, N=N, io=io, seed=26))
    banner("gdn_ssm_scan", io, lens, H, P, G, N)
    y, S = L.run_scan()
    held(L, y, S, io)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("P", [48, 80, 256])
def test_scan_of_short_segments_and_odd_heads(gpu, io, P):
    L = _slow(Layer([700, 300, 129], H=2, P=P, G=2, N=64, io=io, seed=27))
    banner("gdn_ssm_scan", io, P)
    y, S = L.run_scan()
    held(L, y, S, io)
    S2 = L.state.clone()
    y2, _ = L.run_scan(state=S2, state_out=S2)
    assert torch.equal(y, y2) and torch.equal(S, S2)


# tiles of 64 rows: from 2048 tiles of 32 on, with heads of more than 32 channels
@pytest.mark.parametrize("io,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("n,H,P,G,N,K", [
    (16, 64, 64, 8, 32, 4), (22, 32, 80, 4, 64, 3), (33, 32, 48, 1, 32, 2), (64, 8, 144, 8, 128, 4), (8, 32, 256, 2, 256, 4),
])
def test_step_of_a_served_batch(gpu, io, out, n, H, P, G, N, K):
    assert n * H * -(-P // 32) >= 2048
    L = Layer([1] * n, H=H, P=P, G=G, N=N, K=K, io=io, seed=28)
    y, S, h = Guard((n, H, P), DT[out]), Guard(tuple(L.state.shape), torch.float32), Guard(tuple(L.hist.shape), DT[io])
    banner("gdn_ssm_step", io, out, n, H, P, G, N, K)

    def run(hist, hist_out, state, state_out, yy):
        ssm.gdn_ssm_step(L.shape(out), L.raw, L.conv_w, L.conv_b, L.dt, L.A_log, L.dt_bias, L.D, hist, hist_out, state, state_out, yy)

    run(L.hist, h.t, L.state, S.t, y.t)
    torch.cuda.synchronize()
    assert y.intact() and S.intact() and h.intact()
    c, ce, new = orc.conv(L.cu, f64(L.raw), f64(L.conv_w), f64(L.conv_b), f64(L.hist))
    dt, lam = L.steps()
    ry, ey, rS, eS = orc.scan(L.cu, c, dt, lam, f64(L.D), f64(L.state), H, P, G, N, xbc_err=ce)
    check("state", S.t, rS, orc.rounded(rS, eS, "f32"))
    check("y", y.t, ry, orc.rounded(ry, ey, out))
    assert np.array_equal(f64(h.t), new)
    hist, state, y2 = L.hist.clone(), L.state.clone(), torch.empty_like(y.t)
    run(hist, hist, state, state, y2)  # everything in place: the same bits
    assert torch.equal(y2, y.t) and torch.equal(state, S.t) and torch.equal(hist, h.t)
