"""The state space kernels against the fp64 oracle (oracle/ssm_oracle.py).

Tolerances are the oracle's own bounds on an fp32 evaluation plus half a step
of the stored type.  For 16-bit y the scan may form its products from operands
held in two 8-bit-significand parts (each off by at most 2^-18 of its value,
two of them in a term): 2^-16 of the sum of absolute terms is added there.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_pre_amd import ssm
from oracle import ssm_oracle as orc

from .gpu_util import banner

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FILL = 0x5A


class Guard:
    """A device tensor between bands of a known byte; `.t` goes to the kernel."""

    PAD = 8192

    def __init__(self, size, dtype, init=None):
        n = int(np.prod(size)) * dtype.itemsize
        self.n = n
        self.buf = torch.full((n + 2 * self.PAD,), FILL, dtype=torch.uint8, device="cuda")
        self.t = self.buf[self.PAD:self.PAD + n].view(dtype).view(size)
        if init is not None:
            self.t.copy_(init)

    def intact(self):
        return bool((self.buf[:self.PAD] == FILL).all() and (self.buf[self.PAD + self.n:] == FILL).all())

    def untouched(self, rows):
        return bool((rows.contiguous().view(torch.uint8) == FILL).all())


def f64(t):
    return t.detach().double().cpu().numpy()


def check(what, got, ref, tol):
    got = f64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - tol
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else ()
    assert not over.size or over[at] <= 0, f"{what} at {at}: {got[at]} for {ref[at]}, tolerance {tol[at]:.3g}"


class Layer:
    """One layer's inputs on the GPU, and the same values for the oracle."""

    def __init__(self, lens, H=4, P=64, G=2, N=128, K=4, io="bf16", seed=0, tail=0, pad=0, state=True):
        rng = np.random.default_rng([7, seed, H, P, N])
        self.H, self.P, self.G, self.N, self.K, self.io = H, P, G, N, K, io
        self.C, self.lens = H * P + 2 * G * N, list(lens)
        self.cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int64)
        self.n, self.used = len(self.lens), int(self.cu[-1])
        self.T = self.used + tail
        up = lambda a, dt=DT[io]: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(dt)  # noqa: E731
        f32 = torch.float32
        width = self.C + H + pad
        width += -width % 8
        self.proj = up(rng.normal(size=(self.T, width)))
        self.raw, self.dt = self.proj[:, :self.C], self.proj[:, self.C:self.C + H]
        x = rng.normal(size=(self.T, self.C))
        self.xbc = up(x / (1 + np.exp(-x)))
        self.conv_w, self.conv_b = up(rng.normal(size=(self.C, K)) * 0.4), up(rng.normal(size=self.C) * 0.2)
        self.hist = up(rng.normal(size=(self.n, K - 1, self.C)))
        self.A_log = up(np.log(rng.uniform(1, 16, H)), f32)
        dt0 = np.exp(rng.uniform(np.log(1e-3), np.log(0.1), H))
        self.dt_bias = up(dt0 + np.log(-np.expm1(-dt0)), f32)
        self.D = up(rng.normal(1, 0.2, H), f32)
        self.state = up(rng.normal(size=(self.n, H, P, N)) * (0.1 if state else 0), f32)
        self.cu_t = torch.from_numpy(self.cu.astype(np.int32)).cuda()

    def shape(self, out=None, strided=True, **kw):
        return ssm.make_ssm_shape(self.H, self.P, self.G, self.N, kw.pop("n_seq", self.n), kw.pop("T", self.T),
                                  kw.pop("max_T", max(self.lens, default=0)), io=self.io, out=out or self.io,
                                  conv_width=self.K, xbc_stride=self.proj.stride(0) if strided else 0,
                                  dt_stride=self.proj.stride(0) if strided else 0, **kw)

    def dims(self):
        return self.H, self.P, self.G, self.N

    def steps(self, **kw):
        return orc.step_size(f64(self.dt), f64(self.dt_bias), f64(self.A_log), **kw)

    def run_scan(self, out=None, state_out=None, y=None, D=True, state=True, shape_kw=None, ws=None, **kw):
        s = self.shape(out, **(shape_kw or {}))
        y = torch.empty(self.T, self.H, self.P, dtype=DT[out or self.io], device="cuda") if y is None else y
        if state_out is None:
            state_out = torch.empty_like(self.state)
        if ws is None:
            ws = torch.empty(max(256, ssm.gdn_ssm_scan_workspace_bytes(s)), dtype=torch.uint8, device="cuda")
        ssm.gdn_ssm_scan(s, self.cu_t, self.xbc, self.dt, self.A_log, self.dt_bias, self.D if D else None,
                         (self.state if state is True else state) if state is not False else None, state_out, y, ws, **kw)
        return y, state_out

    def check_scan(self, y, S, out=None, D=True, state=True, **clamp):
        out = out or self.io
        dt, lam = self.steps(**clamp)
        Dv = f64(self.D) if D else np.zeros(self.H)
        S0 = f64(self.state) if state else np.zeros_like(f64(self.state))
        args = (self.cu, f64(self.xbc), dt, lam, Dv, S0, *self.dims())
        ry, ey, rS, eS = orc.scan(*args)
        if out != "f32":
            ey = ey + 2.0 ** -16 * orc.scan_magnitude(*args)
        check("state", S, rS, orc.rounded(rS, eS, "f32"))
        check("y", y[:self.used], ry[:self.used], orc.rounded(ry, ey, out)[:self.used])


# ----------------------------------------------------------------- the conv
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K,lens,H,G,N", [
    (4, [37], 6, 2, 64), (3, [1, 0, 2, 3, 31, 32, 33, 0, 64], 4, 1, 32), (2, [1], 1, 1, 32),
    (4, [0, 300, 5], 17, 1, 128), (2, [7, 8, 9, 129], 3, 3, 64),
])
def test_conv(gpu, io, K, lens, H, G, N):
    L = Layer(lens, H=H, G=G, N=N, K=K, io=io, tail=5)
    out, hist = Guard((L.T, L.C), DT[io]), Guard(tuple(L.hist.shape), DT[io])
    banner("gdn_ssm_conv", io, K, lens)
    ssm.gdn_ssm_conv(L.shape(), L.cu_t, L.raw, L.conv_w, L.conv_b, L.hist, hist.t, out.t)
    torch.cuda.synchronize()
    assert out.intact() and hist.intact() and out.untouched(out.t[L.used:])
    ref, err, new = orc.conv(L.cu, f64(L.raw), f64(L.conv_w), f64(L.conv_b), f64(L.hist))
    check("out", out.t[:L.used], ref[:L.used], orc.rounded(ref, err, io)[:L.used])
    assert np.array_equal(f64(hist.t), new)
    # in place, no bias; then no history at all: the same as zeros
    again = L.hist.clone()
    ssm.gdn_ssm_conv(L.shape(), L.cu_t, L.raw, L.conv_w, None, again, again, out.t)
    ref, err, _ = orc.conv(L.cu, f64(L.raw), f64(L.conv_w), np.zeros(L.C), f64(L.hist))
    check("out", out.t[:L.used], ref[:L.used], orc.rounded(ref, err, io)[:L.used])
    assert torch.equal(again, hist.t)
    ssm.gdn_ssm_conv(L.shape(), L.cu_t, L.raw, L.conv_w, None, None, None, out.t)
    zeros = torch.zeros_like(L.hist)
    two = torch.empty_like(out.t)
    ssm.gdn_ssm_conv(L.shape(), L.cu_t, L.raw, L.conv_w, None, zeros, zeros, two)
    assert torch.equal(out.t[:L.used], two[:L.used])


# ----------------------------------------------------------------- the scan
SCAN = [
    # lens, H, P, G, N
    ([1], 1, 16, 1, 32), ([2, 0, 15, 16, 17], 4, 64, 2, 128), ([63, 64, 65], 2, 64, 1, 64),
    ([31, 32, 33, 1], 3, 48, 3, 128), ([127, 128, 129, 0], 2, 32, 1, 256), ([300], 6, 64, 2, 64),
    ([0, 0], 2, 64, 1, 128), ([200, 1, 70], 2, 128, 1, 128), ([90], 1, 80, 1, 64), ([65, 130], 2, 256, 2, 32),
    ([700, 40], 4, 64, 1, 128),
]


@pytest.mark.parametrize("io,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("lens,H,P,G,N", SCAN, ids=[f"{max(c[0])}-H{c[1]}P{c[2]}N{c[4]}" for c in SCAN])
def test_scan(gpu, io, out, lens, H, P, G, N):
    L = Layer(lens, H=H, P=P, G=G, N=N, io=io, tail=3)
    y, S = Guard((L.T, H, P), DT[out]), Guard(tuple(L.state.shape), torch.float32)
    banner("gdn_ssm_scan", io, out, lens, H, P, G, N)
    L.run_scan(out, S.t, y.t, shape_kw=dict(strided=True))
    torch.cuda.synchronize()
    assert y.intact() and S.intact() and y.untouched(y.t[L.used:])
    L.check_scan(y.t, S.t, out)


# sequences of 1 to 9 segments of 128 tokens (2 heads), and of one of 256; the
# last segment from 1 token to a whole one
@pytest.mark.parametrize("io,N", [("f32", 32), ("f16", 128), ("bf16", 128), ("bf16", 256)])
@pytest.mark.parametrize("lens", [[256], [257], [255, 256, 1], [512, 129, 0, 128], [7 * 128], [7 * 128 + 1],
                                  [8 * 128], [9 * 128, 130, 384, 1]], ids=str)
def test_scan_of_few_and_many_segments(gpu, io, N, lens):
    L = Layer(lens, H=2, P=64, G=1, N=N, io=io, seed=11)
    y, S = L.run_scan()
    L.check_scan(y, S)
    S2 = L.state.clone()  # state updated in place: bit for bit the same
    y2, _ = L.run_scan(state=S2, state_out=S2)
    assert torch.equal(y, y2) and torch.equal(S, S2)


def test_scan_without_a_state_to_keep(gpu):
    for lens in ([300, 40], [1200, 5], [37]):
        L = Layer(lens, H=2, P=48, G=1, N=64, io="bf16", seed=12)
        s = L.shape()
        y, _ = L.run_scan()
        y2 = torch.empty_like(y)
        ws = torch.empty(max(256, ssm.gdn_ssm_scan_workspace_bytes(s)), dtype=torch.uint8, device="cuda")
        ssm.gdn_ssm_scan(s, L.cu_t, L.xbc, L.dt, L.A_log, L.dt_bias, L.D, L.state, None, y2, ws)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_sequence(gpu, io, bad):
    # 2 heads of 32, the bad token 700 of the second sequence of 1000
    L = Layer([130, 1000, 77], H=2, P=32, G=1, N=64, io=io, seed=13)
    y0, S0 = L.run_scan()
    at, n = 130 + 700, L.cu
    clean = L.xbc.clone()
    L.xbc[at, 32 + 5] = bad  # channel 5 of head 1
    y, S = L.run_scan()
    y0c, yc = y0.clone(), y.clone()
    y0c[at - 63:n[2], 1, 5], yc[at - 63:n[2], 1, 5] = 0, 0
    S0c, Sc = S0.clone(), S.clone()
    S0c[1, 1, 5], Sc[1, 1, 5] = 0, 0
    assert torch.equal(y0c, yc) and torch.equal(S0c, Sc)
    assert not torch.isfinite(y[at, 1, 5]) and not torch.isfinite(S[1, 1, 5]).any()
    L.xbc.copy_(clean)
    L.xbc[at, 2 * 32 + 7] = bad  # B's value 7
    y, S = L.run_scan()
    for lo, hi in ((0, at - 63), (n[2], n[3])):
        assert torch.equal(y0[lo:hi], y[lo:hi])
    assert torch.equal(S0[0], S[0]) and torch.equal(S0[2], S[2])
    assert not torch.isfinite(y[at]).any()


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_scan_options(gpu, io):
    L = Layer([100, 5], io=io)
    banner("gdn_ssm_scan without D and state", io)
    y, S = L.run_scan(D=False, state=False)
    L.check_scan(y, S, D=False, state=False)
    banner("in place, clamped steps", io)
    S = L.state.clone()
    y, _ = L.run_scan(state=S, state_out=S, shape_kw=dict(dt_min=0.01, dt_max=0.25))
    L.check_scan(y, S, dt_min=float(np.float32(0.01)), dt_max=0.25)
    # the outputs do not depend on whether the state is kept, or where
    y2, S2 = L.run_scan(shape_kw=dict(dt_min=0.01, dt_max=0.25))
    assert torch.equal(y, y2) and torch.equal(S, S2)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_scan_with_extreme_steps(gpu, io):
    # raw steps of -inf leave the state (decay 1, nothing written); huge ones
    # clear it (decay 0); ordinary ones stand right after them
    L = Layer([150, 70], H=2, G=1, io=io)
    L.dt[::7] = float("-inf")
    L.dt[3::11] = 60.0
    L.dt[64] = 3000.0
    L.A_log[0] = 6.0
    banner("gdn_ssm_scan extreme steps", io)
    y, S = L.run_scan("f32")
    L.check_scan(y, S, "f32")
    L.dt[:] = float("-inf")
    y, S = L.run_scan("f32")
    assert torch.equal(S, L.state)


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-4, 300.0])
def test_scan_of_small_and_large_inputs(gpu, io, scale):
    L = Layer([130], H=2, G=1, io=io)
    L.xbc[:, :L.H * L.P] *= scale
    L.state *= scale
    L.state[:, 1] *= 1e-3  # a head whose state is far below its inputs
    banner("gdn_ssm_scan scaled", io, scale)
    y, S = L.run_scan("f32")
    L.check_scan(y, S, "f32")


def test_scan_reads_nothing_of_other_rows(gpu):
    # NaN and infinity in the neighbours of a sequence and behind the last one
    for io in ("f32", "f16", "bf16"):
        L = Layer([40, 70, 17], H=2, G=1, io=io, tail=60)
        y0, S0 = L.run_scan()
        L.xbc[:40] = float("nan")
        L.dt[:40] = float("inf")
        L.xbc[110:] = float("inf")
        L.dt[110:] = float("nan")
        banner("gdn_ssm_scan neighbours", io)
        y, S = L.run_scan()
        assert torch.equal(y[40:110], y0[40:110]) and torch.equal(S[1], S0[1])


def test_scan_of_a_long_sequence(gpu):
    # many segments of one sequence, few heads; then pieces of it in turn
    for io, out in (("bf16", "f32"), ("f32", "f32")):
        L = Layer([5000, 130], H=2, P=64, G=1, N=64, io=io)
        banner("gdn_ssm_scan long", io)
        y, S = L.run_scan(out)
        L.check_scan(y, S, out)
        L2 = Layer([5000, 130], H=2, P=64, G=1, N=64, io=io)
        state = L2.state[:1].clone()
        ys = []
        for a, b in ((0, 1), (1, 38), (38, 1062), (1062, 5000)):
            part = Layer([b - a], H=2, P=64, G=1, N=64, io=io)
            part.A_log, part.dt_bias, part.D = L2.A_log, L2.dt_bias, L2.D
            part.xbc, part.proj = L2.xbc[a:b], L2.proj[a:b]
            part.dt, part.state = L2.dt[a:b], state
            yp, state = part.run_scan(out)
            ys.append(yp)
        L.check_scan(torch.cat(ys + [y[5000:]]), torch.cat([state, S[1:]]), out)


def test_scan_of_an_empty_batch_copies_the_state(gpu):
    L = Layer([0, 0, 0], H=2, G=1)
    S = torch.empty_like(L.state)
    banner("gdn_ssm_scan, conv: no tokens")
    ssm.gdn_ssm_scan(L.shape(T=0, max_T=0), L.cu_t, None, None, L.A_log, L.dt_bias, None, L.state, S, None)
    h = torch.empty_like(L.hist)
    ssm.gdn_ssm_conv(L.shape(T=0, max_T=0), L.cu_t, None, L.conv_w, None, L.hist, h, None)
    assert torch.equal(S, L.state) and torch.equal(h, L.hist)


def test_many_sequences(gpu):
    # more sequences than a launch grid's second dimension takes in one piece
    n = 40000
    L = Layer([1] * n, H=1, P=16, G=1, N=32, K=2, io="f16")
    banner("gdn_ssm_conv, scan, step: 40000 sequences")
    out, hist = torch.empty(n, L.C, dtype=torch.float16, device="cuda"), torch.empty_like(L.hist)
    ssm.gdn_ssm_conv(L.shape(), L.cu_t, L.raw, L.conv_w, L.conv_b, L.hist, hist, out)
    y, S = L.run_scan("f32")
    sy, sS, sh = torch.empty(n, 1, 16, device="cuda"), torch.empty_like(L.state), torch.empty_like(hist)
    ssm.gdn_ssm_step(L.shape("f32"), L.raw, L.conv_w, L.conv_b, L.dt, L.A_log, L.dt_bias, L.D, L.hist, sh, L.state, sS, sy)
    torch.cuda.synchronize()
    assert torch.equal(sh, hist)
    at = np.r_[0:3, 32766:32771, n - 3:n]  # around the grid's seam, and the ends
    part = Layer([1] * len(at), H=1, P=16, G=1, N=32, K=2, io="f16")
    pick = torch.from_numpy(at).cuda()
    for k in ("proj", "xbc", "hist", "state"):
        setattr(part, k, getattr(L, k)[pick].contiguous())
    part.raw, part.dt = part.proj[:, :L.C], part.proj[:, L.C:L.C + 1]
    for k in ("conv_w", "conv_b", "A_log", "dt_bias", "D"):
        setattr(part, k, getattr(L, k))
    part.check_scan(y[pick], S[pick], "f32")
    c, ce, new = orc.conv(part.cu, f64(part.raw), f64(L.conv_w), f64(L.conv_b), f64(part.hist))
    check("out", out[pick], c, orc.rounded(c, ce, "f16"))
    assert np.array_equal(f64(hist[pick]), new)
    dt, lam = part.steps()
    ry, ey, rS, eS = orc.scan(part.cu, c, dt, lam, f64(L.D), f64(part.state), 1, 16, 1, 32, xbc_err=ce)
    check("step y", sy[pick], ry, orc.rounded(ry, ey, "f32"))
    check("step state", sS[pick], rS, orc.rounded(rS, eS, "f32"))


def test_rows_past_32_bits(gpu):
    # the last sequence lies behind 2^31 elements of xbc and y: the same bits as
    # a call on its rows alone
    H, P, G, N, tail = 64, 64, 1, 128, 70
    C = H * P + 2 * G * N
    T = (1 << 31) // (H * P) + 200
    small = Layer([tail], H=H, P=P, G=G, N=N)
    xbc = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    dt = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    xbc[-tail:], dt[-tail:] = small.xbc, small.dt
    y = torch.empty(T, H * P, dtype=torch.bfloat16, device="cuda")
    state = torch.cat([torch.zeros_like(small.state), small.state])
    S = torch.empty_like(state)
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    s = ssm.make_ssm_shape(H, P, G, N, 2, T, T - tail)
    ws = torch.empty(ssm.gdn_ssm_scan_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    banner("gdn_ssm_scan, conv past 2^31 elements", T)
    ssm.gdn_ssm_scan(s, cu, xbc, dt, small.A_log, small.dt_bias, small.D, state, S, y, ws)
    ys, Ss = small.run_scan()
    assert torch.equal(y[-tail:].view(tail, H, P), ys) and torch.equal(S[1:], Ss)
    assert not y[:1000].any() and not y[T // 2:T // 2 + 1000].any() and not S[0].any()
    # the conv of the same rows, its output over y's old place
    hist = torch.zeros(2, 3, C, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(xbc)
    ssm.gdn_ssm_conv(s, cu, xbc, small.conv_w, None, hist, hist, out)
    one = torch.empty(tail, C, dtype=torch.bfloat16, device="cuda")
    ssm.gdn_ssm_conv(small.shape(strided=False), small.cu_t, small.xbc, small.conv_w, None, None, None, one)
    assert torch.equal(out[-tail:], one) and torch.equal(hist[1], small.xbc[-3:]) and not out[:1000].any()


def test_bounds_outside_the_rows_are_taken_as_their_ends(gpu):
    # cu_seqlens below 0, past total_T, and falling: no access leaves the
    # buffers, and a call whose max_T is too small is right all the same
    L = Layer([30, 90], H=2, P=64, G=1, N=64, io="bf16")
    y, S = Guard((L.T, 2, 64), torch.bfloat16), Guard(tuple(L.state.shape), torch.float32)
    out, hist = Guard((L.T, L.C), torch.bfloat16), Guard(tuple(L.hist.shape), torch.bfloat16)
    for cu in ([-7, 30, 1 << 30], [40, 10, 120], [0, 120, 60]):
        L.cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        banner("cu_seqlens", cu)
        L.run_scan(state_out=S.t, y=y.t)
        ssm.gdn_ssm_conv(L.shape(), L.cu_t, L.raw, L.conv_w, None, L.hist, hist.t, out.t)
        torch.cuda.synchronize()
        assert y.intact() and S.intact() and out.intact() and hist.intact()
        if cu[1] == 30:
            L.check_scan(y.t, S.t)
    L = Layer([700], H=2, P=64, G=1, N=64, io="bf16")
    banner("max_T too small")
    y, S = L.run_scan(shape_kw=dict(max_T=1))
    L.check_scan(y, S)


# ----------------------------------------------------------------- the step
@pytest.mark.parametrize("io,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n,H,P,G,N,K", [
    (1, 6, 64, 2, 128, 4), (5, 2, 16, 1, 32, 2), (3, 4, 80, 4, 64, 3), (2, 2, 256, 1, 256, 4), (33, 8, 48, 2, 128, 4),
])
def test_step(gpu, io, out, n, H, P, G, N, K):
    L = Layer([1] * n, H=H, P=P, G=G, N=N, K=K, io=io)
    y, S = Guard((n, H, P), DT[out]), Guard(tuple(L.state.shape), torch.float32)
    h = Guard(tuple(L.hist.shape), DT[io])
    banner("gdn_ssm_step", io, out, n, H, P, G, N, K)

    def run(hist, hist_out, state, state_out, yy, D=L.D, b=L.conv_b):
        ssm.gdn_ssm_step(L.shape(out), L.raw, L.conv_w, b, L.dt, L.A_log, L.dt_bias, D, hist, hist_out, state, state_out, yy)

    run(L.hist, h.t, L.state, S.t, y.t)
    torch.cuda.synchronize()
    assert y.intact() and S.intact() and h.intact()
    c, ce, new = orc.conv(L.cu, f64(L.raw), f64(L.conv_w), f64(L.conv_b), f64(L.hist))
    dt, lam = L.steps()
    ry, ey, rS, eS = orc.scan(L.cu, c, dt, lam, f64(L.D), f64(L.state), H, P, G, N, xbc_err=ce)
    check("state", S.t, rS, orc.rounded(rS, eS, "f32"))
    check("y", y.t, ry, orc.rounded(ry, ey, out))
    assert np.array_equal(f64(h.t), new)
    # everything in place: the same bits
    hist, state, y2 = L.hist.clone(), L.state.clone(), torch.empty_like(y.t)
    run(hist, hist, state, state, y2)
    assert torch.equal(y2, y.t) and torch.equal(state, S.t) and torch.equal(hist, h.t)
    # nothing given, nothing kept: as with zeros
    run(None, None, None, None, y2, D=None, b=None)
    run(torch.zeros_like(hist), None, torch.zeros_like(state), None, y.t, D=torch.zeros_like(L.D), b=torch.zeros_like(L.conv_b))
    assert torch.equal(y2, y.t)


# ----------------------------------------------------------------- the norm
@pytest.mark.parametrize("x,io", [("f32", "f32"), ("f16", "f16"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,size,groups", [
    (1, 8, 1), (3, 64, 5), (7, 72, 3), (300, 128, 2), (2, 256, 1), (5, 512, 8), (3, 1024, 3), (2, 1000, 1), (1, 2048, 1),
    (2, 4096, 2), (1, 8192, 1), (1, 16384, 2),
])
def test_group_norm(gpu, x, io, rows, size, groups):
    rng = np.random.default_rng([8, rows, size])
    ch = size * groups
    xs, zs = ch + 8, ch + 16
    xt = torch.from_numpy(rng.normal(0.2, 0.5, (rows, xs))).to("cuda").to(DT[x])
    zt = torch.from_numpy(rng.normal(size=(rows, zs))).to("cuda").to(DT[io])
    w = torch.from_numpy(rng.normal(1, 0.2, ch)).to("cuda").to(DT[io])
    b = torch.from_numpy(rng.normal(size=ch)).to("cuda").to(DT[io])
    for centre in (False, True):
        for last in (False, True):
            for z_, w_, b_ in ((zt, w, b), (zt, w, None), (None, None, b)):
                s = ssm.make_norm_shape(rows, ch, groups, x=x, io=io, eps=1e-5, centre=centre, gate_last=last,
                                        x_stride=xs, z_stride=zs)
                y = Guard((rows, ch), DT[io])
                banner("gdn_group_norm", x, io, rows, size, groups, centre, last, z_ is None)
                ssm.gdn_group_norm(s, xt, z_, w_, b_, y.t)
                torch.cuda.synchronize()
                assert y.intact()
                np_ = lambda t: None if t is None else f64(t)  # noqa: E731
                ref, err = orc.group_norm(f64(xt)[:, :ch], None if z_ is None else f64(zt)[:, :ch], np_(w_), np_(b_), groups,
                                          float(np.float32(1e-5)), centre, last)
                check("y", y.t, ref, orc.rounded(ref, err, io))


def test_group_norm_of_zeros_and_of_a_large_mean(gpu):
    # an all-zero group gives the bias; a mean of 1000 with a spread of 1
    # keeps fp32 accuracy (the squares are those of the differences)
    rng = np.random.default_rng(9)
    x = torch.from_numpy(np.stack([np.zeros(512), 1000 + rng.normal(size=512)])).float().cuda()
    y = torch.empty_like(x)
    banner("gdn_group_norm zeros, large mean")
    ssm.gdn_group_norm(ssm.make_norm_shape(2, 512, 1, io="f32", centre=True), x, None, None, None, y)
    ref, err = orc.group_norm(f64(x), None, None, None, 1, float(np.float32(1e-5)), True, False)
    check("y", y, ref, orc.rounded(ref, err, "f32"))
    assert not y[0].any()


# ------------------------------------------------------------- used together
def _layer(L, bufs, out="f32", stream=None):
    """conv -> scan -> norm of one layer, as a model runs them."""
    ssm.gdn_ssm_conv(L.shape(out), L.cu_t, L.raw, L.conv_w, L.conv_b, L.hist, bufs["hist"], bufs["xbc"], stream=stream)
    s = L.shape(out)
    ssm.gdn_ssm_scan(s, L.cu_t, bufs["xbc"], L.dt, L.A_log, L.dt_bias, L.D, L.state, bufs["state"], bufs["y"], bufs["ws"], stream=stream)
    ssm.gdn_group_norm(bufs["norm"], bufs["y"], bufs["z"], bufs["w"], None, bufs["o"], stream=stream)


def _bufs(L, out="f32"):
    io, ch = DT[L.io], L.H * L.P
    g = torch.Generator(device="cuda").manual_seed(3)
    return dict(hist=torch.empty_like(L.hist), xbc=torch.empty(L.T, L.C, dtype=io, device="cuda"),
                state=torch.empty_like(L.state), y=torch.empty(L.T, ch, dtype=DT[out], device="cuda"),
                ws=torch.empty(max(256, ssm.gdn_ssm_scan_workspace_bytes(L.shape(out))), dtype=torch.uint8, device="cuda"),
                norm=ssm.make_norm_shape(L.T, ch, L.G, x=out, io=L.io), z=torch.randn(L.T, ch, generator=g, device="cuda").to(io),
                w=torch.randn(ch, generator=g, device="cuda").to(io), o=torch.empty(L.T, ch, dtype=io, device="cuda"))


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_layer_of_the_operators(gpu, io):
    L = Layer([70, 1, 0, 200], H=4, P=64, G=2, N=128, io=io)
    b = _bufs(L)
    banner("conv, scan, norm", io)
    _layer(L, b)
    torch.cuda.synchronize()
    c, ce, new = orc.conv(L.cu, f64(L.raw), f64(L.conv_w), f64(L.conv_b), f64(L.hist))
    check("xbc", b["xbc"], c, orc.rounded(c, ce, io))
    L.xbc = b["xbc"]  # each stage is held to its own inputs
    L.check_scan(b["y"].view(L.T, L.H, L.P), b["state"], "f32")
    ref, err = orc.group_norm(f64(b["y"]), f64(b["z"]), f64(b["w"]), None, L.G, float(np.float32(1e-5)), False, False)
    check("o", b["o"], ref, orc.rounded(ref, err, io))
    assert np.array_equal(f64(b["hist"]), new)


def test_steps_continue_a_prompt(gpu):
    # a prompt of 29 tokens, then 8 steps: as one prompt of 37 (fp32, so that
    # conv's rounding between the operators is within the bounds)
    L = Layer([37], H=3, P=64, G=1, N=64, io="f32")
    P29 = Layer([29], H=3, P=64, G=1, N=64, io="f32")
    for k in ("conv_w", "conv_b", "hist", "A_log", "dt_bias", "D", "state"):
        setattr(P29, k, getattr(L, k))
    P29.proj, P29.raw, P29.dt = L.proj[:29], L.raw[:29], L.dt[:29]
    b = _bufs(P29)
    banner("prompt, then steps")
    _layer(P29, b)
    ys = [b["y"].view(29, 3, 64)]
    hist, state = b["hist"], b["state"]
    s = L.shape(T=1, max_T=1)
    for t in range(29, 37):
        y, h2 = torch.empty(1, 3, 64, device="cuda"), torch.empty_like(hist)
        ssm.gdn_ssm_step(s, L.raw[t:t + 1], L.conv_w, L.conv_b, L.dt[t:t + 1], L.A_log, L.dt_bias, L.D, hist, h2, state, state, y)
        hist = h2
        ys.append(y)
    c, ce, new = orc.conv(L.cu, f64(L.raw), f64(L.conv_w), f64(L.conv_b), f64(L.hist))
    ce = orc.rounded(c, ce, "f32")
    dt, lam = L.steps()
    ry, ey, rS, eS = orc.scan(L.cu, c, dt, lam, f64(L.D), f64(L.state), 3, 64, 1, 64, xbc_err=ce)
    check("y", torch.cat(ys), ry, orc.rounded(ry, ey, "f32"))
    check("state", state, rS, orc.rounded(rS, eS, "f32"))
    assert np.array_equal(f64(hist), new)


def test_captured_layer_and_step_replay_as_eager(gpu):
    # a prompt's layer and a decode step in one graph, replayed with new inputs
    # copied in and eager work between the replays
    L = Layer([300, 65], H=4, P=64, G=1, N=128, io="bf16")
    S1 = Layer([1, 1], H=4, P=64, G=1, N=128, io="bf16", seed=5)
    b, e = _bufs(L, "bf16"), _bufs(L, "bf16")
    y1, y2 = (torch.empty(2, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    h1, h2 = torch.empty_like(L.hist), torch.empty_like(L.hist)

    def run(bufs, y, h):
        _layer(L, bufs, "bf16")
        ssm.gdn_ssm_step(S1.shape(), S1.raw, L.conv_w, L.conv_b, S1.dt, L.A_log, L.dt_bias, L.D, bufs["hist"], h,
                         bufs["state"], bufs["state"], y)

    banner("captured layer and step")
    run(b, y1, h1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, y1, h1)
    for k in range(4):
        L.proj.copy_(Layer([300, 65], H=4, P=64, G=1, N=128, io="bf16", seed=10 + k).proj)
        b["ws"].fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        run(e, y2, h2)
        torch.cuda.synchronize()
        for name in ("hist", "xbc", "state", "y", "o"):
            assert torch.equal(b[name], e[name]), (k, name)
        assert torch.equal(y1, y2) and torch.equal(h1, h2)


def test_two_calls_at_once_on_two_streams(gpu):
    a, b = (Layer([900, 300], H=4, P=64, G=1, N=128, io="bf16", seed=s) for s in (1, 2))
    ba, bb, ra, rb = _bufs(a), _bufs(b), _bufs(a), _bufs(b)
    _layer(a, ra)
    _layer(b, rb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    banner("two streams")
    for _ in range(5):
        _layer(a, ba, stream=s1)
        _layer(b, bb, stream=s2)
    torch.cuda.synchronize()
    for got, ref in ((ba, ra), (bb, rb)):
        for name in ("hist", "xbc", "state", "y", "o"):
            assert torch.equal(got[name], ref[name]), name
