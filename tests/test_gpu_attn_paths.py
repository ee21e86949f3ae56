"""The attention kernels in the ways a program uses them: few rows over long caches,
captured and replayed, two calls at once, on other streams, over caches that pass 32-bit
offsets, forked and compacted; and that results repeat bit for bit.  Tolerances are those
of test_gpu_attn.py."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_pre_amd import attn
from oracle import attn_oracle as orc

from .gpu_util import banner
from .test_gpu_attn import IO, WEIGHTS, Case
from .test_gpu_ssm import DT, Guard, check, f64

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# --------------------------------------------------- few rows over long caches
LONG = [
    # new, past, H, KV, D, page, window
    ([1], [5000], 8, 2, 64, 16, 0), ([130, 1, 0, 40], [3000, 9000, 50, 1], 6, 2, 128, 16, 0), ([256, 5, 130], [2000, 3001, 900], 16, 2, 256, 64, 0),
    ([64], [1000], 32, 8, 128, 16, 0), ([17, 33], [4000, 4100], 128, 1, 64, 16, 0), ([20, 300], [6000, 3000], 4, 4, 96, 32, 1500),
    ([3, 3, 3], [2500, 0, 700], 10, 1, 192, 16, 0), ([1] * 40, list(range(900, 4900, 100)), 2, 1, 64, 16, 0), ([90], [7000], 2, 2, 128, 16, 4097),
]


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("new,past,H,KV,D,page,window", LONG, ids=[f"{max(c[1])}-H{c[2]}D{c[4]}w{c[6]}" for c in LONG])
def test_chunks_that_go_on_from_long_caches(gpu, io, new, past, H, KV, D, page, window):
    banner("gdn_attn_prefill long caches", io, new, past, H, KV, D, page, window)
    c = Case(new, past, H, KV, D, page, io, tail=2, window=window, stale=float("nan"))
    assert attn.gdn_attn_prefill_workspace_bytes(c.shape()) > 0  # their keys are dealt to more blocks than there are of rows
    a = c.run_and_check("prefill")
    assert torch.equal(a[:c.used], c.run("prefill")[:c.used])


# rows that may be cut (a workspace is asked for) and are not, or are only by the lengths on the device;
# more blocks of rows than are resident at once
MIXED = [
    ([115, 1, 5, 393, 1, 64], [3780, 0, 0, 37, 0, 2], 20, 2, 192, 64, 0, 3900), ([700], [3000], 24, 4, 256, 64, 0, 3700),
    ([3, 50], [0, 10], 6, 2, 128, 16, 0, 30000), ([90, 0, 4], [200, 0, 100], 8, 2, 64, 16, 0, 20000), ([650], [900], 32, 8, 256, 16, 700, 1550),
]


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("new,past,H,KV,D,page,window,max_kv", MIXED, ids=[f"{c[0]}-D{c[4]}" for c in MIXED])
def test_batches_of_mixed_lengths(gpu, io, new, past, H, KV, D, page, window, max_kv):
    banner("gdn_attn_prefill mixed", io, new, past, H, KV, D, page, window, max_kv)
    c = Case(new, past, H, KV, D, page, io, tail=1, window=window, stale=float("nan"))
    pages = -(-max_kv // page)
    more = dict(max_kv=max_kv, table_pages=pages)
    c.table_t = torch.cat([c.table_t, torch.full((c.n, max(0, pages - c.table_t.shape[1])), 1 << 30, dtype=torch.int32, device="cuda")], 1)
    a = c.run("prefill", **more)
    c.check("prefill", a)
    for _ in range(2):
        assert torch.equal(a[:c.used], c.run("prefill", **more)[:c.used])


@pytest.mark.parametrize("io", IO)
def test_long_caches_with_a_value_that_is_not_finite(gpu, io):
    c = Case([70], [4000], 4, 2, 64, 16, io, gate=False)
    y0 = c.run("prefill")
    for at in (4020, 1000):  # a key in the rows' own part, and one that all see
        page, row = int(c.table[0, at // 16]), at % 16
        was = c.v[page, 0, row, 9].clone()
        c.v[page, 0, row, 9] = float("inf")
        banner("gdn_attn_prefill long caches, infinity", io, at)
        y = c.run("prefill")
        c.v[page, 0, row, 9] = was
        first = max(0, at - 4000)
        assert not torch.isfinite(y[first:, :2, 9]).any() and torch.equal(y[:first], y0[:first]) and torch.equal(y[:, 2:], y0[:, 2:])
        assert torch.equal(y[:, :, :9], y0[:, :, :9]) and torch.equal(y[:, :, 10:], y0[:, :, 10:])


# ------------------------------------------------- many query heads to a key head
@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("kv,H,KV,D,window", [([3000, 1, 65, 0, 500], 100, 1, 256, 0), ([700, 40], 66, 2, 128, 0), ([1500], 128, 1, 192, 0),
                                              ([5000, 17], 24, 1, 64, 600), ([900, 901], 160, 2, 96, 33), ([300] * 150, 17, 1, 64, 0)])
def test_step_of_large_groups(gpu, io, kv, H, KV, D, window):
    banner("gdn_attn_step large groups", io, kv[:5], H, KV, D, window)
    Case([1] * len(kv), [n - 1 for n in kv], H, KV, D, 16, io, window=window, stale=float("nan")).run_and_check("step")


# --------------------------------------------------------------- many sequences
@pytest.mark.parametrize("op", ["prefill", "step"])
def test_many_sequences(gpu, op):
    n, H, D = 40000, 2, 64
    rng = np.random.default_rng(31)
    kv = np.maximum(1, (rng.integers(0, 50, n) - 5))
    pages = torch.from_numpy(rng.normal(size=(64, 2, 1, 16, D))).cuda().bfloat16()
    table = rng.integers(0, 64, (n, 3))
    q = torch.from_numpy(rng.normal(size=(n, H, D))).cuda().bfloat16()
    s = attn.make_attn_shape(H, 1, D, n, n, 1, 48, 64, 3, 16, "bf16", page_stride=pages.stride(0))
    size = attn.gdn_attn_step_workspace_bytes if op == "step" else attn.gdn_attn_prefill_workspace_bytes
    ws = torch.empty(max(256, size(s)), dtype=torch.uint8, device="cuda")
    out = Guard((n, H, D), torch.bfloat16)
    args = (i32(kv), i32(table), q, pages[:, 0], pages[:, 1], None, out.t, ws)
    banner("many sequences", op)
    attn.gdn_attn_step(s, *args) if op == "step" else attn.gdn_attn_prefill(s, torch.arange(n + 1, dtype=torch.int32, device="cuda"), *args)
    torch.cuda.synchronize()
    assert out.intact()
    some = np.unique(np.concatenate([[0, 1, 255, 256, n - 1], rng.integers(0, n, 400)]))
    step, least = WEIGHTS[op]["bf16"]
    ref, err = orc.attention(np.arange(len(some) + 1), kv[some], table[some], f64(q)[some], f64(pages[:, 0]), f64(pages[:, 1]), 16,
                             float(np.float32(D ** -0.5)), weight_step=step, weight_least=least)
    check("out", out.t[torch.from_numpy(some).cuda()], ref, orc.rounded(ref, err, "bf16"))


# ------------------------------------------------------- offsets past 32 bits
def test_offsets_past_32_bits(gpu):
    """Two layers' pages in one buffer of 2^32 and more values; the sequences' pages lie at its end."""
    KV, D, page, H = 2, 128, 64, 8
    size = 2 * KV * page * D
    N = (1 << 32) // (2 * size) + 40  # pages of two layers
    pages = torch.empty(N, 2, 2, KV, page, D, dtype=torch.bfloat16, device="cuda")
    assert pages.numel() > 1 << 32
    rng = np.random.default_rng(41)
    last = np.arange(N - 30, N)
    pages[N - 30:] = torch.from_numpy(rng.normal(size=(30, 2, 2, KV, page, D)).astype(np.float32)).cuda().bfloat16()
    kc, vc = pages[:, 1, 0], pages[:, 1, 1]
    order = rng.permutation(last)
    table = order[:20].reshape(2, 10)
    kv = np.array([600, 333])
    lib = dict(max_kv=640, n_pages=N, table_pages=10, page_size=page, io="bf16", page_stride=pages.stride(0))
    f = lambda t: f64(t[N - 30:])  # noqa: E731
    # append: the last 5 and 3 tokens
    proj = torch.from_numpy(rng.normal(size=(8, (H + 2 * KV) * D)).astype(np.float32)).cuda().bfloat16()
    q, k, v = proj[:, :H * D], proj[:, H * D:(H + KV) * D], proj[:, (H + KV) * D:]
    s = attn.make_attn_shape(H, KV, D, 2, 8, 5, q_stride=proj.stride(0), k_stride=proj.stride(0), v_stride=proj.stride(0), **lib)
    q_out = torch.empty(8, H * D, dtype=torch.bfloat16, device="cuda")
    banner("offsets past 32 bits")
    attn.gdn_attn_append(s, i32([0, 5, 8]), i32(kv), i32(table), None, q, k, v, None, None, None, q_out, kc, vc)
    seq, p = orc.positions(np.array([0, 5, 8]), kv)
    at = torch.from_numpy(table[seq, p // page]).cuda()
    assert torch.equal(vc[at, :, torch.from_numpy(p % page).cuda()].reshape(8, -1), v) and torch.equal(q_out, q)
    assert torch.equal(kc[at, :, torch.from_numpy(p % page).cuda()].reshape(8, -1), k)
    # attention
    for op in ("prefill", "step"):
        n = 8 if op == "prefill" else 2
        s = attn.make_attn_shape(H, KV, D, 2, n, 5 if n == 8 else 1, **lib)
        ask = attn.gdn_attn_step_workspace_bytes if op == "step" else attn.gdn_attn_prefill_workspace_bytes
        ws = torch.empty(max(256, ask(s)), dtype=torch.uint8, device="cuda")
        out = torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda")
        qq = q_out if n == 8 else q_out[[4, 7]]
        args = (i32(kv), i32(table), qq, kc, vc, None, out, ws)
        cu = np.array([0, 5, 8]) if n == 8 else np.arange(3)
        attn.gdn_attn_step(s, *args) if op == "step" else attn.gdn_attn_prefill(s, i32(cu), *args)
        step, least = WEIGHTS[op]["bf16"]
        ref, err = orc.attention(cu, kv, table - (N - 30), f64(qq).reshape(n, H, D), f(kc), f(vc), page, float(np.float32(D ** -0.5)),
                                 weight_step=step, weight_least=least)
        check(op, out, ref, orc.rounded(ref, err, "bf16"))
    # copy: from the end to the beginning, and back to a free page of the end
    free = order[20:]
    s = attn.make_attn_shape(KV, KV, D, **lib)
    attn.gdn_attn_copy_pages(s, i32([[table[0, 0], 3], [table[1, 1], int(free[0])]]), 2, kc, vc)
    for a, b in ((table[0, 0], 3), (table[1, 1], free[0])):
        assert torch.equal(kc[a], kc[b]) and torch.equal(vc[a], vc[b])


# ---------------------------------------------------- repeats, graphs, streams
@pytest.mark.parametrize("op", ["prefill", "step"])
def test_results_repeat_bit_for_bit(gpu, op):
    for new, past, D in (([200, 3], [100, 4000], 128), ([30, 1], [9000, 60], 256)):
        c = Case([1] * 2 if op == "step" else new, past, 8, 2, D, 16, "bf16")
        first = c.run(op)
        for _ in range(5):
            assert torch.equal(first, c.run(op))


@pytest.mark.parametrize("io", IO)
def test_captured_calls_follow_what_changes_on_the_device(gpu, io):
    """One graph of a decode step (append, attention, copy of a page) replayed as the sequences grow,
    with eager work and synchronisations between; each replay against the eager calls on the same inputs."""
    H, KV, D, page, n, TP, N = 8, 2, 64, 16, 3, 80, 300
    rng = np.random.default_rng(51)
    up = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda().to(DT[io])  # noqa: E731
    pages = up(rng.normal(size=(N, 2, KV, page, D)))
    twin = pages.clone()
    table = i32(rng.permutation(N - 10)[:n * TP].reshape(n, TP))
    kv, pairs, cu = i32([1] * n), i32([[0, N - 1]]), i32(list(range(n + 1)))
    proj = up(rng.normal(size=(n, (H + 2 * KV) * D)))
    gate, w = up(rng.normal(size=(n, H * D))), up(rng.normal(1, 0.2, D))
    freq = attn.gdn_attn_rope_freqs(32)[0].cuda()
    st = proj.stride(0)
    s = attn.make_attn_shape(H, KV, D, n, n, 1, TP * page, N, TP, page, io, rope_dim=32, q_stride=st, k_stride=st, v_stride=st,
                             page_stride=pages.stride(0), gate_stride=gate.stride(0))
    d = attn.make_attn_shape(H, KV, D, n, n, 1, TP * page, N, TP, page, io, page_stride=pages.stride(0))

    def buffers():
        return [torch.empty(n, H * D, dtype=DT[io], device="cuda") for _ in range(3)], \
            [torch.empty(max(256, size(d)), dtype=torch.uint8, device="cuda")
             for size in (attn.gdn_attn_step_workspace_bytes, attn.gdn_attn_prefill_workspace_bytes)]

    def go(cache, outs, ws):
        k, v = cache[:, 0], cache[:, 1]
        attn.gdn_attn_append(s, cu, kv, table, None, proj[:, :H * D], proj[:, H * D:(H + KV) * D], proj[:, (H + KV) * D:], freq, w, w,
                             outs[0], k, v)
        attn.gdn_attn_step(d, kv, table, outs[0], k, v, gate, outs[1], ws[0])
        attn.gdn_attn_prefill(d, cu, kv, table, outs[0], k, v, gate, outs[2], ws[1])
        attn.gdn_attn_copy_pages(d, pairs, 1, k, v)

    mine, ws = buffers()
    eager, ews = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(pages, mine, ws)
    torch.cuda.current_stream().wait_stream(side)
    pages.copy_(twin)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(pages, mine, ws)
    for i, lengths in enumerate(([1, 1, 1], [2, 17, 900], [64, 0, 1280], [65, 1, 3], [1000, 1100, 1200], [1, 1, 1])):
        kv.copy_(i32(lengths))
        proj.copy_(up(rng.normal(size=proj.shape)))
        gate.copy_(up(rng.normal(size=gate.shape)))
        pairs.copy_(i32([[i, N - 1 - i]]))
        banner("replay", io, i, lengths)
        graph.replay()
        go(twin, eager, ews)
        torch.cuda.synchronize()
        for a, b in zip(mine, eager):
            assert torch.equal(a, b), (i, lengths)
        assert torch.equal(pages, twin)


@pytest.mark.parametrize("op", ["prefill", "step"])
def test_two_calls_at_once(gpu, op):
    """Two layers' calls on two streams with workspaces of their own, each behind work on its stream."""
    many = [1] * 30
    cases = [Case(many if op == "step" else [60, 5], [3000] * 30 if op == "step" else [3000, 4000], 8, 2, D, 16, "bf16", seed=D) for D in (128, 256)]
    want = [c.run(op) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                q = c.qw.clone()
                c.qw.copy_(torch.zeros_like(q))
                c.qw.copy_(q)  # (the call has to come behind this)
                got.append(c.run(op))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_another_stream_given_as_an_argument(gpu):
    c = Case([1] * 3, [50, 700, 2000], 8, 2, 128, 16, "f16")
    want = c.run("step")
    s = c.shape()
    ws = torch.empty(attn.gdn_attn_step_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    out = torch.zeros(3, 8, 128, dtype=torch.float16, device="cuda")
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        torch.cuda.synchronize()
        attn.gdn_attn_step(s, c.kv_t, c.table_t, c.q, c.k, c.v, c.gate, out, ws, stream=stream)
        st.synchronize()
        assert torch.equal(out, want)
        out.zero_()


# ------------------------------------------------------------------ tensors
def test_tensors_on_the_wrong_device_or_of_the_wrong_kind(gpu):
    c = Case([1], [40], 4, 2, 64, 16, "bf16")
    s = c.shape()
    ws = torch.empty(attn.gdn_attn_step_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    out = torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    good = dict(kv_len=c.kv_t, page_table=c.table_t, q=c.q, k_cache=c.k, v_cache=c.v, gate=c.gate, out=out, workspace=ws)
    for name in good:
        with pytest.raises(ValueError, match="host memory"):
            attn.gdn_attn_step(s, **{**good, name: torch.empty_strided(good[name].shape, good[name].stride(), dtype=good[name].dtype)})
    for name, x in (("out", out.half()), ("q", c.q[:, :-64]), ("k_cache", c.k[1:]), ("page_table", c.table_t.long())):
        with pytest.raises(ValueError, match=name):
            attn.gdn_attn_step(s, **{**good, name: x})
    with pytest.raises(Exception, match="gdn_attn_step"):
        attn.gdn_attn_step(s, **{**good, "workspace": ws[:-256]})


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("io", IO)
def test_a_fork_and_a_compaction(gpu, io):
    """A prompt is appended and attended; its last page is copied for a second sequence that shares the
    others; both go on by steps of their own; then all pages move to other places."""
    rng = np.random.default_rng(61)
    H, KV, D, page, N, TP, T = 4, 2, 96, 16, 40, 12, 70
    up = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda().to(DT[io])  # noqa: E731
    pages = torch.full((N, 2, KV, page, D), float("nan"), dtype=DT[io], device="cuda")
    k, v = pages[:, 0], pages[:, 1]
    freq = attn.gdn_attn_rope_freqs(96, 1e4, "base", 2.0)[0].cuda()
    keys, values = [], []  # of both sequences, as the cache rounds them
    table = rng.permutation(N - 20)[:TP]
    tables = np.stack([table, table])

    def put(x, seqs, kv):
        n, t = len(seqs), x.shape[0] // len(seqs)
        s = attn.make_attn_shape(H, KV, D, n, n * t, t, TP * page, N, TP, page, io, rope_dim=96, page_stride=pages.stride(0),
                                 q_stride=x.stride(0), k_stride=x.stride(0), v_stride=x.stride(0))
        q_out, out = (torch.empty(n * t, H * D, dtype=DT[io], device="cuda") for _ in range(2))
        cu, kv_t, tab = i32([t * i for i in range(n + 1)]), i32([kv] * n), i32(tables[seqs])
        attn.gdn_attn_append(s, cu, kv_t, tab, None, x[:, :H * D], x[:, H * D:(H + KV) * D], x[:, (H + KV) * D:], freq, None, None, q_out, k, v)
        s.q_stride = 0
        size = attn.gdn_attn_prefill_workspace_bytes if t > 1 else attn.gdn_attn_step_workspace_bytes
        ws = torch.empty(max(256, size(s)), dtype=torch.uint8, device="cuda")
        if t > 1:
            attn.gdn_attn_prefill(s, cu, kv_t, tab, q_out, k, v, None, out, ws)
        else:
            attn.gdn_attn_step(s, kv_t, tab, q_out, k, v, None, out, ws)
        step, least = WEIGHTS["prefill" if t > 1 else "step"][io]
        # (stale rows hold NaN: the oracle reads those below kv alone)
        clean = [torch.nan_to_num(f) for f in (k, v)]
        ref, err = orc.attention([t * i for i in range(n + 1)], [kv] * n, tables[seqs], f64(q_out).reshape(n * t, H, D), *(f64(f) for f in clean),
                                 page, float(np.float32(D ** -0.5)), weight_step=step, weight_least=least)
        check("out", out, ref, orc.rounded(ref, err, io))
        return out

    draw = lambda n: up(rng.normal(size=(n, (H + 2 * KV) * D)))  # noqa: E731
    put(draw(T), [0], T)
    s = attn.make_attn_shape(KV, KV, D, page_size=page, n_pages=N, io=io, page_stride=pages.stride(0))
    tables[1, T // page:] = np.arange(N - 20, N - 20 + TP - T // page)  # the page in use, and those to come
    attn.gdn_attn_copy_pages(s, i32([[table[T // page], tables[1, T // page]]]), 1, k, v)
    shared = pages[torch.from_numpy(table[:T // page].copy()).cuda()].clone()
    for i in range(1, 30):
        put(draw(2), [0, 1], T + i)
    assert torch.equal(shared, pages[torch.from_numpy(table[:T // page].copy()).cuda()])
    x = draw(2)
    held = -(-(T + 30) // page)
    before = put(x, [0, 1], T + 30)
    free = np.array([p for p in range(N) if p not in tables[:, :held]])
    move = np.unique(tables[1, :held])
    pairs = np.stack([move, free[:len(move)]], 1)
    attn.gdn_attn_copy_pages(s, i32(pairs), len(pairs), k, v)
    where = dict(pairs.tolist())
    tables[1, :held] = [where[p] for p in tables[1, :held]]
    assert torch.equal(before, put(x, [0, 1], T + 30))
