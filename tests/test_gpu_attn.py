"""The attention kernels against the fp64 oracle (oracle/attn_oracle.py).

Tolerances are the oracle's bounds on an fp32 evaluation, half a step of the stored type,
and for 16-bit io what include/gdn_attn.h says of the weights as operands: in a prompt they
are rounded to io (half a step of each; fp16's smallest step is 2^-24, so at least 2^-25 of the largest),
in a step they keep 16 bits at least (2^-16 of each, and of fp16's again 2^-25 of the largest).
"""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_pre_amd import attn
from oracle import attn_oracle as orc

from .gpu_util import banner
from .test_gpu_ssm import DT, Guard, check, f64

pytestmark = pytest.mark.gpu

WEIGHTS = {"prefill": {"f32": (0.0, 0.0), "f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 0.0)},
           "step": {"f32": (0.0, 0.0), "f16": (2.0 ** -16, 2.0 ** -25), "bf16": (2.0 ** -16, 0.0)}}


class Case:
    """One layer's rows, cache and page table on the GPU; `stale`: what rows without a token hold."""

    def __init__(self, new, past, H=4, KV=2, D=64, page=16, io="bf16", seed=0, window=0, gate=True, tail=0, pad=16,
                 scale=None, q_std=2.0, stale=None, interleaved_cache=True):
        rng = np.random.default_rng([11, seed, H, KV, D, page])
        self.H, self.KV, self.D, self.page, self.io, self.window = H, KV, D, page, io, window
        self.new = np.array(new)
        self.kv = np.maximum(self.new + np.array(past), 0)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int64)
        self.n, self.used = len(new), int(self.cu[-1])
        self.T = self.used + tail
        self.scale = float(np.float32(D ** -0.5 if scale is None else scale))
        up = lambda a, dt=DT[io]: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(dt)  # noqa: E731
        self.up = up
        held = -(-self.kv // page)
        self.n_pages = int(held.sum()) + 3
        order = rng.permutation(self.n_pages)
        self.table = np.full((self.n, max(1, int(held.max()))), 1 << 30, dtype=np.int64)  # no page: far outside
        at = 0
        for i, c in enumerate(held):
            self.table[i, :c] = order[at:at + c]
            at += c
        pages = rng.normal(size=(self.n_pages, 2, KV, page, D))
        if stale is not None:
            live = np.zeros((self.n_pages, page), bool)
            for i in range(self.n):
                j = np.arange(self.kv[i])
                live[self.table[i, j // page], j % page] = True
            pages = np.where(live[:, None, None, :, None], pages, stale)
        self.pages = Guard(pages.shape, DT[io], up(pages))
        self.k, self.v = self.pages.t[:, 0], self.pages.t[:, 1]
        width = H * D
        self.qw, self.gw = up(rng.normal(size=(self.T, width + pad)) * q_std), up(rng.normal(size=(self.T, width + 2 * pad)) * 2)
        self.q, self.gate = self.qw[:, :width], self.gw[:, :width] if gate else None
        self.cu_t = torch.from_numpy(self.cu.astype(np.int32)).cuda()
        self.kv_t = torch.from_numpy(self.kv.astype(np.int32)).cuda()
        self.table_t = torch.from_numpy(self.table.astype(np.int32)).cuda()

    def shape(self, **kw):
        d = dict(n_seq=self.n, total_T=self.T, max_T=int(self.new.max()), max_kv=int(self.kv.max()), n_pages=self.n_pages,
                 table_pages=self.table.shape[1], page_size=self.page, io=self.io, scale=self.scale, window=self.window,
                 page_stride=self.pages.t.stride(0), q_stride=self.qw.stride(0), gate_stride=self.gw.stride(0))
        return attn.make_attn_shape(self.H, self.KV, self.D, **{**d, **kw})

    def run(self, op, out=None, ws=None, **kw):
        s = self.shape(**kw)
        size = attn.gdn_attn_step_workspace_bytes if op == "step" else attn.gdn_attn_prefill_workspace_bytes
        ws = torch.empty(max(256, size(s)), dtype=torch.uint8, device="cuda") if ws is None else ws
        out = torch.empty(self.T, self.H, self.D, dtype=DT[self.io], device="cuda") if out is None else out
        if op == "step":
            attn.gdn_attn_step(s, self.kv_t, self.table_t, self.q, self.k, self.v, self.gate, out, ws)
        else:
            attn.gdn_attn_prefill(s, self.cu_t, self.kv_t, self.table_t, self.q, self.k, self.v, self.gate, out, ws)
        return out

    def reference(self, op):
        gate = None if self.gate is None else f64(self.gate).reshape(self.T, self.H, self.D)
        step, least = WEIGHTS[op][self.io]
        ref, err = orc.attention(self.cu, self.kv, self.table, f64(self.q).reshape(self.T, self.H, self.D), f64(self.k), f64(self.v),
                                 self.page, self.scale, self.window, gate, step, least)
        return ref[:self.used], orc.rounded(ref, err, self.io)[:self.used]

    def check(self, op, out):
        ref, tol = self.reference(op)
        check("out", out[:self.used], ref, tol)

    def run_and_check(self, op):
        out = Guard((self.T, self.H, self.D), DT[self.io])
        was = self.pages.t.clone().view(torch.uint8)
        self.run(op, out.t)
        torch.cuda.synchronize()
        assert out.intact() and out.untouched(out.t[self.used:])
        assert torch.equal(was, self.pages.t.view(torch.uint8))
        self.check(op, out.t)
        return out.t


IO = ["f32", "f16", "bf16"]


# --------------------------------------------------------------------- append
APPEND = [
    # new, past, H, KV, D, page, rope, pairs, norm
    ([1], [0], 1, 1, 64, 16, 64, False, False), ([1], [700], 16, 2, 256, 64, 64, False, True),
    ([37], [0], 6, 2, 64, 16, 32, True, False), ([5, 0, 1, 90], [3, 9, 100, 0], 4, 4, 128, 16, 128, True, True),
    ([30, 2], [0, 1], 3, 1, 96, 32, 48, False, True), ([17, 16, 15], [15, 16, 17], 8, 2, 192, 16, 192, True, False),
    ([300], [1], 2, 1, 256, 1024, 0, False, True), ([3], [40], 2, 2, 96, 16, 16, True, True),
    ([2000], [5], 2, 1, 64, 128, 48, False, True), ([9000, 300], [0, 0], 1, 1, 64, 64, 64, False, False),
]


def append_inputs(c, rope, norm, rng):
    width = (c.H + 2 * c.KV) * c.D
    proj = c.up(rng.normal(size=(c.T, width + 16)) * 1.5)
    cols = np.cumsum([0, c.H * c.D, c.KV * c.D, c.KV * c.D])
    q, k, v = (proj[:, a:b] for a, b in zip(cols, cols[1:]))
    w = [c.up(rng.normal(1, 0.2, c.D)) if norm else None for _ in range(2)]
    freq = c.up(1e4 ** (-np.arange(rope // 2) / max(1, rope // 2)), torch.float32)
    return proj, q, k, v, w, freq


def check_append(c, rope, pairs, norm, seed, positions=None, rope_scale=1.0, **over):
    rng = np.random.default_rng([12, seed])
    proj, q, k, v, w, freq = append_inputs(c, rope, norm, rng)
    q_out = Guard((c.T, c.H * c.D), DT[c.io])
    was = c.pages.t.clone()
    st = proj.stride(0)
    s = c.shape(rope_dim=rope, interleaved=pairs, rope_scale=rope_scale, eps=1e-5, q_stride=st, k_stride=st, v_stride=st, **over)
    pt = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    attn.gdn_attn_append(s, c.cu_t, c.kv_t, c.table_t, pt, q, k, v, freq if rope else None, *w, q_out.t, c.k, c.v)
    torch.cuda.synchronize()
    assert q_out.intact() and c.pages.intact() and q_out.untouched(q_out.t[c.used:])
    seq, p = orc.positions(c.cu, c.kv)
    P = p if positions is None else np.array(positions)[:c.used]
    heads = lambda t, n: f64(t)[:c.used].reshape(c.used, n, c.D)  # noqa: E731
    f = f64(freq)[:rope // 2]
    kw = dict(eps=float(np.float32(1e-5)), scale=float(np.float32(rope_scale)))
    ref, err = orc.rotated(heads(q, c.H), P, f, pairs, None if w[0] is None else f64(w[0]), **kw)
    check("q_out", q_out.t[:c.used], ref, orc.rounded(ref, err, c.io))
    ref, err = orc.rotated(heads(k, c.KV), P, f, pairs, None if w[1] is None else f64(w[1]), **kw)
    put = (p >= 0) & (p < s.max_kv)
    page, row = torch.from_numpy(c.table[seq[put], p[put] // c.page]).cuda(), torch.from_numpy(p[put] % c.page).cuda()
    check("k", c.k[page, :, row], ref[put], orc.rounded(ref, err, c.io)[put])
    assert torch.equal(c.v[page, :, row].reshape(-1), v[:c.used].reshape(c.used, c.KV, c.D)[torch.from_numpy(put).cuda()].reshape(-1))
    # nothing else changes
    was[page, 0, :, row], was[page, 1, :, row] = c.k[page, :, row], c.v[page, :, row]
    assert torch.equal(was.view(torch.uint8), c.pages.t.view(torch.uint8))
    return q_out.t


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("new,past,H,KV,D,page,rope,pairs,norm", APPEND, ids=[f"{c[0]}-D{c[4]}r{c[6]}" for c in APPEND])
def test_append(gpu, io, new, past, H, KV, D, page, rope, pairs, norm):
    banner("gdn_attn_append", io, new, past, H, KV, D, page, rope)
    check_append(Case(new, past, H, KV, D, page, io, tail=3), rope, pairs, norm, 1)


@pytest.mark.parametrize("io", IO)
def test_append_at_far_and_given_positions(gpu, io):
    c = Case([4, 3], [0, 20], 2, 1, 64, 16, io, tail=1)
    far = [0, 1 << 20, (1 << 30) - 1, 7, -5, 131071, 999983, 0]
    banner("gdn_attn_append far positions", io)
    check_append(c, 64, False, True, 2, positions=far, rope_scale=1.2)
    check_append(c, 64, True, False, 3, positions=far)


def test_append_leaves_out_what_has_no_place(gpu):
    # more new tokens than the cache holds: the first three stand below 0; the last two not below max_kv
    c = Case([20, 2], [-3, 4], 2, 1, 64, 16, "bf16")
    banner("gdn_attn_append negative positions")
    check_append(c, 32, False, True, 4)
    c = Case([16], [20], 2, 1, 64, 16, "f32")
    c.table_t[0, 1] = -1  # a page of none: positions 16..31
    was = c.pages.t.clone()
    rng = np.random.default_rng(5)
    proj, q, k, v, w, freq = append_inputs(c, 32, True, rng)
    st = proj.stride(0)
    s = c.shape(rope_dim=32, q_stride=st, k_stride=st, v_stride=st)
    q_out = torch.empty(c.T, c.H * c.D, device="cuda")
    attn.gdn_attn_append(s, c.cu_t, c.kv_t, c.table_t, None, q, k, v, freq, *w, q_out, c.k, c.v)
    torch.cuda.synchronize()
    rows = torch.zeros(c.n_pages, 16, dtype=torch.bool, device="cuda")
    rows[int(c.table[0, 2]), :4] = True  # positions 32 to 35
    assert torch.equal(was.transpose(1, 3)[~rows], c.pages.t.transpose(1, 3)[~rows])
    assert torch.equal(c.v[int(c.table[0, 2]), 0, :4], v[12:16])


# ------------------------------------------------------------------- attention
PREFILL = [
    # new, past, H, KV, D, page
    ([1], [0], 1, 1, 64, 16), ([37], [0], 6, 2, 64, 16), ([1, 0, 2, 31, 32, 33], [0, 5, 63, 1, 0, 31], 4, 2, 128, 16),
    ([64, 65, 63], [0, 0, 64], 8, 8, 96, 16), ([130, 5], [70, 500], 16, 2, 256, 64), ([40], [25], 5, 1, 192, 32),
    ([300], [0], 2, 1, 128, 1024), ([3, 2], [0, 90], 128, 1, 64, 16), ([17], [1000], 12, 4, 64, 16), ([2], [2000], 3, 3, 128, 16),
]


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("new,past,H,KV,D,page", PREFILL, ids=[f"{c[0]}-D{c[4]}" for c in PREFILL])
def test_prefill(gpu, io, new, past, H, KV, D, page):
    banner("gdn_attn_prefill", io, new, past, H, KV, D, page)
    Case(new, past, H, KV, D, page, io, tail=2).run_and_check("prefill")


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 5000])
def test_prefill_window(gpu, io, window):
    banner("gdn_attn_prefill window", io, window)
    Case([150, 3, 1], [0, 400, 99], 6, 2, 64, 16, io, window=window).run_and_check("prefill")
    Case([70], [40], 2, 1, 256, 16, io, window=window, gate=False).run_and_check("prefill")


STEP = [
    # kv lengths, H, KV, D, page
    ([1], 1, 1, 64, 16), ([1, 2, 15, 16, 17, 31, 32, 33], 16, 2, 128, 16), ([127, 128, 129, 0, 255, 256, 257], 8, 1, 256, 64),
    ([700], 16, 2, 256, 64), ([3000, 1, 0, 511], 8, 8, 64, 16), ([100, 1000], 128, 1, 96, 32), ([65, 300], 34, 2, 192, 16),
    ([9000], 32, 8, 128, 16), (list(range(0, 200, 7)), 6, 3, 64, 16),
]


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("kv,H,KV,D,page", STEP, ids=[f"{max(c[0])}-H{c[1]}D{c[3]}" for c in STEP])
def test_step(gpu, io, kv, H, KV, D, page):
    banner("gdn_attn_step", io, kv, H, KV, D, page)
    Case([1] * len(kv), [n - 1 for n in kv], H, KV, D, page, io).run_and_check("step")


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("window", [1, 2, 31, 129, 1000])
def test_step_window(gpu, io, window):
    banner("gdn_attn_step window", io, window)
    Case([1] * 5, [-1, 0, 30, 700, 3000], 6, 2, 128, 16, io, window=window).run_and_check("step")


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("op", ["prefill", "step"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_hidden_values_do_not_matter(gpu, io, op, bad):
    new = [1, 1, 1] if op == "step" else [50, 1, 90]
    past = [0, 70, 300]
    banner("stale rows", io, op, bad)
    Case(new, past, 4, 2, 128, 16, io, stale=bad).run_and_check(op)
    Case(new, past, 4, 2, 64, 16, io, stale=bad, window=20).run_and_check(op)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 40])
def test_prefill_values_that_are_not_finite_stay_with_those_that_see_them(gpu, io, bad, window):
    c = Case([200], [30], 4, 2, 64, 16, io, window=window, gate=False)
    y0 = c.run("prefill")
    at = 100  # a key: seen by the queries from position 100 on, and for `window` of them
    page, row = int(c.table[0, at // 16]), at % 16
    sees = np.zeros(200, bool)
    sees[at - 30:at - 30 + window if window else 200] = True
    sees = torch.from_numpy(sees).cuda()
    clean = c.pages.t.clone()
    c.v[page, 1, row, 5] = bad
    y = c.run("prefill")
    assert torch.equal(y[~sees], y0[~sees]) and torch.equal(y[:, :2], y0[:, :2])
    assert not torch.isfinite(y[sees][:, 2:, 5]).any()
    assert torch.equal(y[:, :, :5], y0[:, :, :5]) and torch.equal(y[:, :, 6:], y0[:, :, 6:])
    c.pages.t.copy_(clean)
    c.k[page, 1, row, 5] = float("nan")
    y = c.run("prefill")
    assert torch.equal(y[~sees], y0[~sees]) and torch.equal(y[:, :2], y0[:, :2]) and torch.isnan(y[sees][:, 2:]).all()
    c.pages.t.copy_(clean)
    c.qw[77, 64 * 3 + 1] = float("nan")
    y = c.run("prefill")
    rest = torch.ones(200, 4, dtype=torch.bool, device="cuda")
    rest[77, 3] = False
    assert torch.equal(y[rest], y0[rest]) and torch.isnan(y[77, 3]).all()


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("op", ["prefill", "step"])
def test_large_and_small_scores(gpu, io, op):
    new = [1, 1] if op == "step" else [70, 3]
    for q_std, scale in ((30.0, None), (2.0, 1e-3), (2.0, 3.0)):
        banner("scores", io, op, q_std, scale)
        Case(new, [300, 500], 4, 2, 64, 16, io, q_std=q_std, scale=scale).run_and_check(op)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("rising", [False, True])
def test_prefill_where_the_largest_score_comes_late_or_early(gpu, io, rising):
    c = Case([40], [600], 4, 1, 64, 16, io)
    grow = torch.linspace(0.01, 4, 640, device="cuda")
    j = torch.arange(640, device="cuda")
    page = c.table_t[0].long()[j // 16]
    c.k[page, 0, j % 16] = (c.k[page, 0, j % 16].float() * (grow if rising else grow.flip(0))[:, None]).to(DT[io])
    banner("gdn_attn_prefill rising", io, rising)
    c.run_and_check("prefill")


@pytest.mark.parametrize("io", IO)
def test_a_step_equals_a_prompt_of_one_token(gpu, io):
    c = Case([1] * 4, [0, 50, 333, 4000], 8, 2, 128, 16, io)
    a, b = c.run("step"), c.run("prefill")
    c.check("step", a)
    c.check("prefill", b)


@pytest.mark.parametrize("op", ["prefill", "step"])
def test_lengths_outside_their_bounds_stay_in_the_buffers(gpu, op):
    c = Case([1] * 4, [40] * 4, 4, 2, 64, 16, "bf16")
    ref = c.run(op)
    c.kv_t.copy_(torch.tensor([41, -7, 1 << 30, 41]))
    c.table_t[3, 1] = -9  # a page outside the cache
    banner("lengths outside", op)
    out = Guard((c.T, c.H, c.D), DT["bf16"])
    c.run(op, out.t)
    torch.cuda.synchronize()
    assert out.intact() and torch.equal(out.t[0], ref[0]) and not out.t[1].any()
    assert torch.equal(out.t[2], ref[2])  # taken as max_kv


def test_sequence_bounds_outside_the_rows(gpu):
    c = Case([5, 6, 7], [9, 9, 9], 4, 2, 64, 16, "bf16", tail=4)
    out = Guard((c.T, c.H, c.D), DT["bf16"])
    q_out = Guard((c.T, c.H * c.D), DT["bf16"])
    for cu in ([0, 5, 11, 1 << 30], [-4, 5, 3, 18], [7, 5, 3, -2]):
        banner("cu_seqlens", cu)
        c.cu_t.copy_(torch.tensor(cu))
        c.run("prefill", out.t)
        s = c.shape(k_stride=c.qw.stride(0), v_stride=c.qw.stride(0))
        attn.gdn_attn_append(s, c.cu_t, c.kv_t, c.table_t, None, c.q, c.q, c.q, None, None, None, q_out.t, c.k, c.v)
        torch.cuda.synchronize()
        assert out.intact() and q_out.intact() and c.pages.intact()


# ------------------------------------------------------------------------ copy
@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("KV,D,page,n", [(1, 64, 16, 1), (2, 256, 64, 3), (3, 96, 16, 40), (8, 128, 16, 200)])
def test_copy_pages(gpu, io, KV, D, page, n):
    rng = np.random.default_rng([13, n])
    N = 2 * n + 5
    pages = Guard((N, 2, KV, page, D), DT[io], torch.from_numpy(rng.normal(size=(N, 2, KV, page, D))).to("cuda").to(DT[io]))
    order = rng.permutation(N)
    pairs = np.stack([order[:n], order[n:2 * n]], 1)
    if n > 2:
        pairs[1, 0] = pairs[0, 0]  # one page to two places
    extra = np.array([[-1, order[-1]], [order[-1], N], [order[-2], order[-2]], [1 << 30, order[-3]]])
    want = pages.t.clone()
    for a, b in pairs:
        want[b] = pages.t[a]
    pt = torch.from_numpy(np.concatenate([extra, pairs]).astype(np.int32)).cuda()
    s = attn.make_attn_shape(KV, KV, D, page_size=page, n_pages=N, page_stride=pages.t.stride(0), io=io)
    banner("gdn_attn_copy_pages", io, KV, D, page, n)
    attn.gdn_attn_copy_pages(s, pt, len(extra) + n, pages.t[:, 0], pages.t[:, 1])
    torch.cuda.synchronize()
    assert pages.intact() and torch.equal(want.view(torch.uint8), pages.t.view(torch.uint8))
    attn.gdn_attn_copy_pages(s, pt, 0, pages.t[:, 0], pages.t[:, 1])
    dense = [pages.t[:, i].contiguous() for i in (0, 1)]
    want = [x.clone() for x in dense]
    attn.gdn_attn_copy_pages(attn.make_attn_shape(KV, KV, D, page_size=page, n_pages=N, io=io), pt[4:5], 1, *dense)
    for x, y in zip(want, dense):
        x[pairs[0, 1]] = x[pairs[0, 0]]
        assert torch.equal(x, y)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("io", IO)
def test_a_prompt_in_chunks_and_steps_equals_one_prompt(gpu, io):
    """The whole way: the rows of a prompt in one call, against chunks and single tokens, through
    append and attention, on caches with pages in another order."""
    rng = np.random.default_rng(21)
    H, KV, D, page, T = 8, 2, 128, 16, 150
    up = lambda a, dt=DT[io]: torch.from_numpy(np.asarray(a, np.float32)).cuda().to(dt)  # noqa: E731
    proj = up(rng.normal(size=(T, (H + 2 * KV) * D)) * 1.5)
    w = up(rng.normal(1, 0.2, D)), up(rng.normal(1, 0.2, D))
    freq, scale = attn.gdn_attn_rope_freqs(64, 1e4, "parts", 4.0, 100.0)
    freq = freq.cuda()
    P = 12
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def go(cuts):
        table = i32(rng.permutation(P)[:10].tolist())[None]
        pages = torch.full((P, 2, KV, page, D), float("nan"), dtype=DT[io], device="cuda")
        outs = []
        for a, b in zip(cuts, cuts[1:]):
            n = b - a
            x = proj[a:b]
            s = attn.make_attn_shape(H, KV, D, 1, n, n, b, P, 10, page, io, rope_dim=64, rope_scale=scale, page_stride=pages.stride(0),
                                     q_stride=x.stride(0), k_stride=x.stride(0), v_stride=x.stride(0))
            q, k, v = x[:, :H * D], x[:, H * D:(H + KV) * D], x[:, (H + KV) * D:]
            q_out, out = (torch.empty(n, H * D, dtype=DT[io], device="cuda") for _ in range(2))
            kc, vc = pages[:, 0], pages[:, 1]
            attn.gdn_attn_append(s, i32([0, n]), i32([b]), table, None, q, k, v, freq, *w, q_out, kc, vc)
            s.q_stride = 0
            step = n == 1
            size = attn.gdn_attn_step_workspace_bytes if step else attn.gdn_attn_prefill_workspace_bytes
            ws = torch.empty(max(256, size(s)), dtype=torch.uint8, device="cuda")
            if step:
                attn.gdn_attn_step(s, i32([b]), table, q_out, kc, vc, None, out, ws)
            else:
                attn.gdn_attn_prefill(s, i32([0, n]), i32([b]), table, q_out, kc, vc, None, out, ws)
            outs.append((q_out, out))
        j = torch.arange(T, device="cuda")
        at = table[0].long()[j // page]
        return torch.cat([q for q, _ in outs]), torch.cat([o for _, o in outs]), kc[at, :, j % page], vc[at, :, j % page]

    q0, whole, k0, v0 = go([0, T])
    q1, parts, k1, v1 = go([0, 1, 2, 40, 41, 100, 149, 150])
    assert torch.equal(q0, q1) and torch.equal(k0, k1) and torch.equal(v0, v1)
    step, least = WEIGHTS["prefill"][io]
    ref, err = orc.attention([0, T], [T], np.arange(10)[None], f64(q0).reshape(T, H, D),
                             *(f64(torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 160 - T))).reshape(10, page, KV, D).transpose(0, 2, 1, 3)
                               for x in (k0, v0)), page, float(np.float32(D ** -0.5)), weight_step=step, weight_least=least)
    tol = orc.rounded(ref, err, io)
    check("whole", whole, ref, tol)
    check("parts", parts, ref, tol)
