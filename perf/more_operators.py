"""Benchmark cases of the attention operators that stand beside Gated DeltaNet
layers: norm and rotary positions with the write to the paged key-value cache,
attention of whole prompts and of single tokens over that cache, and the copy of
its pages.

`own = False`: `run` computes the plain form with elementary torch operations in
32 bits.  `own = True`: `run` makes the calls of
`gated_deltanet_linear_pre_amd.attn` (include/gdn_attn.h).

Symbols: H query heads and KV key-value heads of D values (KV divides H), pages of
`page` token rows; sequence n has `past[n]` tokens in the cache and brings `new[n]`
more, packed one sequence after the other, so its query t stands at position
past[n] + t and sees the keys up to that one (the last `window` of them, if not 0).
The cache is one tensor [pages][K and V][KV][page][D], a sequence's pages are given
by its row of the page table.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- cases
def _append(name, new, past, H=16, KV=2, D=256, page=64, io="bf16", rope=64, pairs=False, norm=True, scaled=False):
    return {"name": name, "op": "append", "new": new, "past": past, "H": H, "KV": KV, "D": D, "page": page, "io": io,
            "rope": rope, "pairs": pairs, "norm": norm, "scaled": scaled}


def _attn(op, name, new, past, H=16, KV=2, D=256, page=64, io="bf16", window=0, gate=True):
    return {"name": name, "op": op, "new": new, "past": past, "H": H, "KV": KV, "D": D, "page": page, "io": io,
            "window": window, "gate": gate}


def _copy(name, n, KV=2, D=256, page=64, io="bf16"):
    return {"name": name, "op": "copy", "n": n, "KV": KV, "D": D, "page": page, "io": io}


RAGGED = "1,17,16383,300,511,8190,2047,37,4095,1000,129,64,12001,640,33,5000"


def listed():
    return [
        # a decode step's token of one sequence, a quarter of the head rotated: latency
        _append("append_one", "1", "700"),
        # one ordinary prompt: pairs of neighbours rotated over the whole head, no norm
        _append("append_prompt", "2048", "0", H=32, KV=8, D=128, page=16, io="f16", rope=128, pairs=True, norm=False),
        # a long packed batch, positions scaled for long contexts, a sequence that goes on from its cache
        _append("append_packed", "16384,8192,2048,511", "0,0,0,30000", scaled=True),
        # a decode step of one sequence with a short cache: latency
        _attn("step", "step_one", "1", "700"),
        # one sequence with a long cache of odd length
        _attn("step", "step_long", "1", "99990", H=32, KV=8, D=128, page=16, io="f16", gate=False),
        # a served batch of 64 sequences of very different lengths
        _attn("step", "step_ragged", ",".join(["1"] * 64), ",".join([RAGGED] * 4)),
        # a short prompt of a small layer in 32 bits
        _attn("prefill", "prefill_short", "37", "0", H=6, KV=2, D=64, page=16, io="f32", gate=False),
        # one ordinary prompt
        _attn("prefill", "prefill_prompt", "2048", "0", H=32, KV=8, D=128, page=16, io="f16", gate=False),
        # one long prompt of a layer with wide heads
        _attn("prefill", "prefill_long", "8192", "0"),
        # a batch of prompts' chunks that go on from long caches, one of a few tokens: few rows, many keys
        _attn("prefill", "prefill_chunk", "256,5,130", "32768,20001,9000"),
        # a sequence is forked: its last page, in use, is copied
        _copy("copy_fork", 1),
        # a cache is compacted: many pages move to free ones
        _copy("copy_compact", 4000, KV=8, D=128, page=16, io="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(v):
    return ",".join(map(str, v))


def draw(rng):
    op = rng.choice(["append", "step", "step", "prefill", "prefill", "copy"])
    io = rng.choice(["f16", "bf16", "bf16", "f32"])
    KV = rng.choice([1, 2, 2, 4, 8])
    D = rng.choice([64, 128, 128, 256, 256]) if rng.random() < 0.8 else rng.choice([96, 192])
    case = {"op": op, "KV": KV, "D": D, "page": rng.choice([16, 16, 32, 64, 64, 128, 256]), "io": io}
    if op == "copy":
        return {**case, "n": max(1, min(_log(rng, 1, 4000), 130_000_000 // (case["page"] * KV * D * (4 if io == "f32" else 2))))}
    case["H"] = KV * rng.randint(1, min(16, 32 // KV))
    if op == "append":
        n = rng.randint(1, 8)
        new = [_log(rng, 1, 8000 // n) for _ in range(n)]
        past = [_log(rng, 1, 20000) - 1 for _ in new]
        case["rope"] = rng.choice([D, D, D // 2 // 16 * 16, D // 4 // 16 * 16])
        return {**case, "new": _text(new), "past": _text(past), "pairs": rng.random() < 0.4, "norm": rng.random() < 0.6,
                "scaled": rng.random() < 0.4}
    case["window"] = _log(rng, 16, 4096) if rng.random() < 0.25 else 0
    case["gate"] = rng.random() < 0.5
    small = 4 if io == "f32" else 1
    if op == "step":
        n = _log(rng, 1, 64)
        most = max(64, min(65000, 250_000_000 // (n * KV * D)) // small)
        return {**case, "new": _text([1] * n), "past": _text([_log(rng, 1, most) - 1 for _ in range(n)])}
    n = rng.randint(1, 6)
    new = [_log(rng, 1, 3000 // n // small) for _ in range(n)]
    most = max(1, min(16000, 250_000_000 // (n * max(new) * case["H"])) // small)
    return {**case, "new": _text(new), "past": _text([rng.choice([0, _log(rng, 1, most)]) for _ in new])}


def _ints(text):
    return [int(n) for n in text.split(",")]


# ------------------------------------------------------------------ inputs
def _frequencies(rope, scaled):
    """Angles a position of each rotated pair; scaled: those of slow pairs divided by 8, of the ones between by less
    (positions then reach 8 times as far), with a factor on the rotated values."""
    f = 1e6 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)
    if not scaled:
        return f.float(), 1.0
    turns = 32768 * f / (2 * math.pi)  # over the length trained on
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (f * (keep + (1 - keep) / 8)).float(), 0.1 * math.log(8) + 1


def prepare(case, seed):
    """What a layer has in hand: its projection's rows, the cache with its page table, buffers for the results."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    io = DT[case["io"]]
    KV, D, page = case["KV"], case["D"], case["page"]

    def normal(*size, std=1.0, mean=0.0):
        return (torch.randn(*size, generator=g, device=DEV) * std + mean).to(io)

    s = dict(case)
    if case["op"] == "copy":
        n = case["n"]
        s["pages"] = normal(2 * n + 3, 2, KV, page, D)
        s["list"] = torch.randperm(2 * n + 3, generator=g, device=DEV)[:2 * n].view(n, 2).to(torch.int32)
        return s
    H, new, past = case["H"], _ints(case["new"]), _ints(case["past"])
    n_seq, T = len(new), sum(new)
    kv = [a + b for a, b in zip(new, past)]
    s["n_seq"], s["T"], s["max_new"], s["max_kv"] = n_seq, T, max(new), max(kv)
    s["cu"] = torch.tensor([sum(new[:i]) for i in range(n_seq + 1)], dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    # pages in any order; entries behind a sequence's last page hold no page
    held = [-(-n // page) for n in kv]
    free = torch.randperm(sum(held) + 5, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.full((n_seq, max(held)), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(max(held), device=DEV)[None, :]
    count = torch.tensor(held, device=DEV)
    first = torch.cumsum(count, 0) - count
    s["table"] = torch.where(at < count[:, None], free[(first[:, None] + at).clamp(max=sum(held) - 1)], s["table"]).contiguous()
    s["pages"] = normal(sum(held) + 5, 2, KV, page, D)
    if case["op"] == "append":
        # one packed projection q | k | v of a layer: the rows are read in place
        s["proj"] = normal(T, (H + 2 * KV) * D, std=1.5)
        s["q"], s["k"], s["v"] = s["proj"][:, :H * D], s["proj"][:, H * D:(H + KV) * D], s["proj"][:, (H + KV) * D:]
        s["q_norm"] = normal(D, std=0.2, mean=1.0) if case["norm"] else None
        s["k_norm"] = normal(D, std=0.2, mean=1.0) if case["norm"] else None
        freq, s["rope_scale"] = _frequencies(case["rope"], case["scaled"])
        s["inv_freq"] = freq.to(DEV)
        s["q_out"] = torch.empty(T, H * D, dtype=io, device=DEV)
        return s
    s["q"] = normal(T, H * D, std=1.5)
    s["gate_in"] = normal(T, H * D) if case["gate"] else None
    s["out"] = torch.empty(T, H * D, dtype=io, device=DEV)
    return s


# -------------------------------------------------------------- plain forms
def _positions(s):
    """Each token's sequence and its position."""
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(s["n_seq"], device=DEV), cu[1:] - cu[:-1], output_size=s["T"])
    return seq, torch.arange(s["T"], device=DEV) - cu[1:][seq] + s["kv_len"][seq]


def _plain_rotated(s, x, weight, pos):
    """Norm and rotation of rows [T][heads][D] in 32 bits, the angles in 64."""
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    r = s["rope"]
    angle = pos[:, None].double() * s["inv_freq"].double()
    cos, sin = ((f(angle) * s["rope_scale"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if s["pairs"] else (x[..., :r // 2], x[..., r // 2:r])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if s["pairs"] else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_append(s):
    H, KV, D, T = s["H"], s["KV"], s["D"], s["T"]
    seq, pos = _positions(s)
    q = _plain_rotated(s, s["q"].reshape(T, H, D), s["q_norm"], pos)
    k = _plain_rotated(s, s["k"].reshape(T, KV, D), s["k_norm"], pos)
    s["q_out"].copy_(q.view(T, H * D))
    page, row = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    s["pages"][page, 0, :, row] = k.to(s["pages"].dtype)
    s["pages"][page, 1, :, row] = s["v"].reshape(T, KV, D)
    return {"q": s["q_out"], "pages": s["pages"]}


def _plain_attention(s):
    """All sequences at once, padded to the longest."""
    H, KV, D, n, T, L = s["H"], s["KV"], s["D"], s["n_seq"], s["T"], s["max_kv"]
    cu, kv_len = s["cu"].long(), s["kv_len"].long()
    key = torch.arange(L, device=DEV)
    page = s["table"].long()[:, key // s["page"]].clamp(min=0)
    k, v = (s["pages"][page, i, :, key % s["page"]].float().transpose(1, 2) for i in (0, 1))  # [n][KV][L][D]
    M = s["max_new"]
    row = torch.arange(M, device=DEV)
    new = cu[1:] - cu[:-1]
    q = s["q"].view(T, KV, H // KV, D)[(cu[:-1, None] + row).clamp(max=T - 1)].float()
    q = q.permute(0, 2, 1, 3, 4).reshape(n, KV, M * (H // KV), D)
    x = (q @ k.transpose(-1, -2).contiguous()) * D ** -0.5
    pos = (kv_len - new)[:, None] + row  # [n][M]
    seen = (key <= pos[..., None]) & (key < kv_len[:, None, None])
    if s["window"]:
        seen &= key > pos[..., None] - s["window"]
    seen = seen.repeat_interleave(H // KV, 1)[:, None]
    x = x.masked_fill(~seen, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x @ v.contiguous()) / x.sum(-1, keepdim=True)
    o = o.view(n, KV, M, H // KV, D).transpose(1, 2).reshape(n, M, H * D)
    o = o[row < new[:, None]]
    if s["gate_in"] is not None:
        o = o * torch.sigmoid(s["gate_in"].float())
    return {"out": o.to(s["out"].dtype)}


def _plain(s):
    if s["op"] == "copy":
        source, to = s["list"].long().unbind(1)
        s["pages"][to] = s["pages"][source]
        return {"pages": s["pages"]}
    return _plain_append(s) if s["op"] == "append" else _plain_attention(s)


# ----------------------------------------------------------- the framework's
def _own(s):
    from gated_deltanet_linear_pre_amd import attn

    pages = s["pages"]
    if "shape" not in s:  # sizes and workspace: made once, and kept, as a program keeps them
        kw = dict(page_size=s["page"], n_pages=pages.shape[0], page_stride=pages.stride(0), io=s["io"])
        if s["op"] != "copy":
            kw |= dict(n_seq=s["n_seq"], total_T=s["T"], max_T=s["max_new"], max_kv=s["max_kv"], table_pages=s["table"].shape[1])
        if s["op"] == "append":
            kw |= dict(rope_dim=s["rope"], interleaved=s["pairs"], rope_scale=s["rope_scale"], eps=EPS,
                       q_stride=s["q"].stride(0), k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))
        elif s["op"] != "copy":
            kw |= dict(window=s["window"])
        s["shape"] = attn.make_attn_shape(s.get("H", s["KV"]), s["KV"], s["D"], **kw)
        if s["op"] in ("step", "prefill"):
            size = attn.gdn_attn_step_workspace_bytes if s["op"] == "step" else attn.gdn_attn_prefill_workspace_bytes
            s["workspace"] = torch.empty(max(256, size(s["shape"])), dtype=torch.uint8, device=DEV)
        s["k_cache"], s["v_cache"] = pages[:, 0], pages[:, 1]
    k, v = s["k_cache"], s["v_cache"]
    if s["op"] == "copy":
        attn.gdn_attn_copy_pages(s["shape"], s["list"], s["n"], k, v)
        return {"pages": pages}
    if s["op"] == "append":
        attn.gdn_attn_append(s["shape"], s["cu"], s["kv_len"], s["table"], None, s["q"], s["k"], s["v"], s["inv_freq"],
                             s["q_norm"], s["k_norm"], s["q_out"], k, v)
        return {"q": s["q_out"], "pages": pages}
    if s["op"] == "step":
        attn.gdn_attn_step(s["shape"], s["kv_len"], s["table"], s["q"], k, v, s["gate_in"], s["out"], s["workspace"])
    else:
        attn.gdn_attn_prefill(s["shape"], s["cu"], s["kv_len"], s["table"], s["q"], k, v, s["gate_in"], s["out"], s["workspace"])
    return {"out": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def work(case):
    io = 4 if case["io"] == "f32" else 2
    KV, D = case["KV"], case["D"]
    if case["op"] == "copy":
        n = case["n"] * 2 * KV * case["page"] * D
        return {"bytes": 2 * n * io + 8 * case["n"], "flops": 0}
    H, new, past = case["H"], _ints(case["new"]), _ints(case["past"])
    T, W = sum(new), case.get("window") or 1 << 60
    if case["op"] == "append":
        turned = 3 * case["rope"] + (5 * D if case["norm"] else 0)
        return {"bytes": 2 * T * (H + 2 * KV) * D * io, "flops": T * (H + KV) * turned}
    pairs = keys = 0
    for t, p in zip(new, past):
        full = max(0, min(t, W - p))  # queries that the window cuts nothing from
        pairs += full * p + full * (full + 1) // 2 + (t - full) * W
        keys += min(t + p, t + W - 1)
    rows = T * H * D
    return {"bytes": keys * KV * D * 2 * io + rows * (2 + bool(case["gate"])) * io, "flops": 4 * D * H * pairs}


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """One sequence and one head after the other, in 64 bits."""
    s = prepare(case, seed)
    KV, D, page = case["KV"], case["D"], case["page"]
    if case["op"] == "copy":
        pages = s["pages"].double()
        was = pages.clone()
        for a, b in s["list"].tolist():
            pages[b] = was[a]
        return {"pages": pages}
    H, new, past = case["H"], _ints(case["new"]), _ints(case["past"])
    begin, res = 0, []
    if case["op"] == "append":
        pages, r = s["pages"].double(), case["rope"]
        even = torch.arange(r // 2, device=DEV) * 2 if case["pairs"] else torch.arange(r // 2, device=DEV)
        odd = even + 1 if case["pairs"] else even + r // 2
        for n, (t, p) in enumerate(zip(new, past)):
            pos = torch.arange(p, p + t, device=DEV)
            turn = pos[:, None].double() * s["inv_freq"].double()

            def turned(x, weight):
                x = x[begin:begin + t].double().reshape(t, -1, D)
                if case["norm"]:
                    x = x * ((x ** 2).sum(2, keepdim=True) / D + EPS) ** -0.5 * weight.double()
                y = x.clone()
                c, z = torch.cos(turn)[:, None] * s["rope_scale"], torch.sin(turn)[:, None] * s["rope_scale"]
                y[..., even] = x[..., even] * c - x[..., odd] * z
                y[..., odd] = x[..., even] * z + x[..., odd] * c
                return y

            res.append(turned(s["q"], s["q_norm"]).reshape(t, H * D))
            where = s["table"][n].long()[pos // page]
            pages[where, 0, :, pos % page] = turned(s["k"], s["k_norm"])
            pages[where, 1, :, pos % page] = s["v"][begin:begin + t].double().reshape(t, KV, D)
            begin += t
        return {"q": torch.cat(res), "pages": pages}
    out = torch.empty(sum(new), H, D, dtype=torch.float64, device=DEV)
    for n, (t, p) in enumerate(zip(new, past)):
        where = s["table"][n, :-(-(t + p) // page)].long()
        at, key = torch.arange(p, p + t, device=DEV)[:, None], torch.arange(t + p, device=DEV)[None, :]
        hidden = key > at
        if case["window"]:
            hidden = hidden | (at - key >= case["window"])
        for h in range(KV):
            k, v = (s["pages"][where, i, h].reshape(-1, D)[:t + p].double() for i in (0, 1))
            for j in range(h * (H // KV), (h + 1) * (H // KV)):
                x = s["q"][begin:begin + t, j * D:(j + 1) * D].double() @ k.t().contiguous() / math.sqrt(D)
                x[hidden] = -math.inf
                w = torch.exp(x - x.max(1, keepdim=True)[0])
                out[begin:begin + t, j] = (w / w.sum(1, keepdim=True)) @ v
        begin += t
    out = out.reshape(-1, H * D)
    return {"out": out / (1 + torch.exp(-s["gate_in"].double())) if case["gate"] else out}
