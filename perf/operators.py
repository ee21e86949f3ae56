"""Benchmark cases of the state space operators: the short causal convolution,
the selective scan, the single-token step and the gated group norm.

`own = False`: `run` computes the plain form with elementary torch operations in
32 bits.  `own = True`: `run` makes the calls of
`gated_deltanet_linear_pre_amd.ssm` (include/gdn_ssm.h).

Symbols: H heads of P channels each, G groups of H/G heads that share their B
and C vectors of N values, K conv taps, C = H*P + 2*G*N channels x | B | C of a
token row, sequences packed one after the other (`lens`).
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
CHUNK = 64  # tokens of a chunk of the plain scan


# ------------------------------------------------------------------- cases
def _conv(name, lens, H=64, P=64, G=1, N=128, K=4, io="bf16"):
    return {"name": name, "op": "conv", "lens": lens, "H": H, "P": P, "G": G, "N": N, "K": K, "io": io}


def _scan(name, lens, H=64, P=64, G=1, N=128, io="bf16", out="bf16"):
    return {"name": name, "op": "scan", "lens": lens, "H": H, "P": P, "G": G, "N": N, "io": io, "out": out}


def _step(name, n, H=64, P=64, G=1, N=128, K=4, io="bf16", out="bf16"):
    return {"name": name, "op": "step", "n": n, "H": H, "P": P, "G": G, "N": N, "K": K, "io": io, "out": out}


def _norm(name, rows, channels, groups, x="bf16", io="bf16", centre=False, last=False, bias=False):
    return {"name": name, "op": "norm", "rows": rows, "channels": channels, "groups": groups, "x": x, "io": io,
            "centre": centre, "last": last, "bias": bias}


def listed():
    return [
        # a short prompt of a small layer: latency
        _conv("conv_short", "37", H=6, N=64, io="f32"),
        # one ordinary prompt
        _conv("conv_prompt", "2048", io="f16"),
        # a long packed batch with a ragged last sequence
        _conv("conv_packed", "16384,8192,2048,511", G=8),
        # a short prompt of a small layer in 32 bits, 3 heads a group
        _scan("scan_short", "37", H=6, G=2, N=64, io="f32", out="f32"),
        # one ordinary prompt, B and C shared by all heads
        _scan("scan_prompt", "2048", io="f16", out="f16"),
        # a served batch of ragged prompts, a single token and an empty one among them
        _scan("scan_ragged", "1,300,37,0,1024,513,130", H=32, P=128, G=2, N=256, out="f32"),
        # the long packed batch, 8 heads a group
        _scan("scan_packed", "16384,8192,2048,511", G=8),
        # a decode step of one sequence: latency
        _step("step_one", 1),
        # a decode step of a served batch: the state's traffic
        _step("step_batch", 64, G=8, io="f16", out="f16"),
        # one decode token's norm: latency
        _norm("norm_one", 1, 4096, 1),
        # after a prompt's scan, gate first, one group for 8 heads
        _norm("norm_prompt", 2048, 4096, 8, x="f32", io="f16"),
        # after the long packed batch: one centred group a head, gate last
        _norm("norm_packed", 27135, 4096, 64, centre=True, last=True, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "step", "norm"])
    io = rng.choice(["f16", "bf16", "bf16", "f32"])
    if op == "norm":
        size = 8 * _log(rng, 4, 512)
        groups = rng.randint(1, max(1, 8192 // size))
        rows = min(_log(rng, 1, 27000), 110_000_000 // (size * groups))
        centre = rng.random() < 0.4
        return {"op": op, "rows": rows, "channels": size * groups, "groups": groups, "x": rng.choice(["f32", io]), "io": io,
                "centre": centre, "last": rng.random() < 0.5, "bias": centre and rng.random() < 0.7}
    G = rng.choice([1, 1, 2, 4, 8])
    H = G * rng.randint(1, 64 // G)
    P = rng.choice([32, 64, 64, 64, 128] if op != "scan" else [32, 64, 64, 64])
    N = rng.choice([64, 128, 128, 128] if op != "step" else [64, 128, 128, 256])
    case = {"op": op, "H": H, "P": P, "G": G, "N": N, "io": io}
    if op != "scan":
        case["K"] = rng.choice([2, 3, 4, 4, 4])
    if op == "step":
        return {**case, "n": _log(rng, 1, 64 if N <= 128 and P <= 64 else 16), "out": rng.choice([io, "f32"])}
    if rng.random() < 0.5:
        lens = [_log(rng, 1, 12000)]
    else:
        lens = [_log(rng, 1, 3000) for _ in range(rng.randint(2, 8))]
    if io == "f32" or op == "conv":
        lens = [max(1, n // 2) for n in lens]
    case["lens"] = ",".join(map(str, lens))
    if op == "scan":
        case["out"] = rng.choice([io, "f32"])
    return case


def _lens(case):
    return [int(n) for n in case["lens"].split(",")] if "lens" in case else [1] * case["n"]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    """Inputs as an ordinary layer meets them, and the buffers that its results go to."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    io = DT[case["io"]]

    def normal(*size, std=1.0, mean=0.0, dtype=io):
        return (torch.randn(*size, generator=g, device=DEV) * std + mean).to(dtype)

    def uniform(*size, lo, hi):
        return torch.rand(*size, generator=g, device=DEV) * (hi - lo) + lo

    s = dict(case)
    if case["op"] == "norm":
        rows, ch = case["rows"], case["channels"]
        s["x_in"] = normal(rows, ch, std=0.5, mean=0.1, dtype=DT[case["x"]])
        s["z"] = normal(rows, ch)
        s["weight"] = normal(ch, std=0.1, mean=1.0)
        s["bias_in"] = normal(ch, std=0.1) if case["bias"] else None
        s["y"] = torch.empty(rows, ch, dtype=io, device=DEV)
        return s
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    lens = _lens(case)
    C, T, n_seq = H * P + 2 * G * N, sum(lens), len(lens)
    s["T"], s["n_seq"], s["max_T"] = T, n_seq, max(lens)
    s["cu"] = torch.tensor([sum(lens[:i]) for i in range(n_seq + 1)], dtype=torch.int32, device=DEV)
    if case["op"] in ("conv", "step"):
        # one packed projection z | xbc | dt of a layer: the rows are read in place
        K = case["K"]
        s["proj"] = normal(T, -(-(C + H) // 8) * 8)
        s["xbc"], s["dt"] = s["proj"][:, :C], s["proj"][:, C:C + H]
        s["conv_w"], s["conv_b"] = normal(C, K, std=0.4), normal(C, std=0.2)
        s["hist"] = normal(n_seq, K - 1, C)
        s["hist_out"] = torch.empty_like(s["hist"])
    if case["op"] == "conv":
        s["out_buf"] = torch.empty(T, C, dtype=io, device=DEV)
        return s
    if case["op"] == "scan":
        x = torch.randn(T, C, generator=g, device=DEV)
        s["xbc"], s["dt"] = (x * torch.sigmoid(x)).to(io), normal(T, H)
    s["A_log"] = torch.log(uniform(H, lo=1.0, hi=16.0))
    dt0 = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))  # softplus(dt_bias) = dt0
    s["D"] = normal(H, std=0.2, mean=1.0, dtype=torch.float32)
    s["state"] = normal(n_seq, H, P, N, std=0.1, dtype=torch.float32)
    s["state_out"] = torch.empty_like(s["state"])
    s["y"] = torch.empty(T, H * P, dtype=DT[case["out"]], device=DEV)
    return s


# -------------------------------------------------------------- plain forms
def _silu(x):
    return x * torch.sigmoid(x)


def _plain_norm(s):
    rows, ch, groups = s["rows"], s["channels"], s["groups"]
    gate = _silu(s["z"].float())
    v = s["x_in"].float() * (1.0 if s["last"] else gate)
    v = v.view(rows, groups, ch // groups)
    v = v - v.mean(-1, keepdim=True) if s["centre"] else v
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)
    y = v.view(rows, ch) * s["weight"].float()
    y = y + s["bias_in"].float() if s["bias_in"] is not None else y
    y = y * gate if s["last"] else y
    return {"y": y.to(s["y"].dtype)}


def _plain_conv(s, xbc):
    """SiLU(conv) in 32 bits and the new history: rows are taken from [histories; tokens] by their index."""
    K, n_seq, T = s["K"], s["n_seq"], s["T"]
    cu = s["cu"].long()
    ext = torch.cat([s["hist"].reshape(n_seq * (K - 1), -1), xbc])
    seq = torch.repeat_interleave(torch.arange(n_seq, device=DEV), cu[1:] - cu[:-1], output_size=T)
    pos = torch.arange(T, device=DEV) - cu[seq]  # place in its sequence
    tap = torch.arange(K, device=DEV)
    at = pos[:, None] + tap[None, :]  # row of [history; tokens of the sequence]
    rows = torch.where(at < K - 1, seq[:, None] * (K - 1) + at, n_seq * (K - 1) + cu[seq][:, None] + at - (K - 1))
    x = ext[rows].float()
    pre = (x * s["conv_w"].float().t()[None]).sum(1) + s["conv_b"].float()
    at = (cu[1:] - cu[:-1])[:, None] + torch.arange(K - 1, device=DEV)[None, :]
    n = torch.arange(n_seq, device=DEV)[:, None]
    rows = torch.where(at < K - 1, n * (K - 1) + at, n_seq * (K - 1) + cu[:-1][:, None] + at - (K - 1))
    return _silu(pre), ext[rows]


def _plain_dt(s):
    dt = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
    return dt, -torch.exp(s["A_log"]) * dt


def _plain_scan(s):
    """Chunks of CHUNK tokens, all at once; sums of log decays in 64 bits."""
    H, P, G, N, T, n_seq, Q = s["H"], s["P"], s["G"], s["N"], s["T"], s["n_seq"], CHUNK
    cu = s["cu"].long()
    length = cu[1:] - cu[:-1]
    chunks = (length + Q - 1) // Q  # of each sequence
    nc = (T + Q - 1) // Q + n_seq  # room for the chunks of all sequences
    first = torch.cumsum(chunks, 0) - chunks
    seq = torch.repeat_interleave(torch.arange(n_seq, device=DEV), length, output_size=T)
    pos = torch.arange(T, device=DEV) - cu[seq]
    slot = (first[seq] + pos // Q) * Q + pos % Q  # where a token stands in the padded chunks
    chunk = torch.arange(nc, device=DEV)
    cseq = (torch.searchsorted(first + chunks, chunk, right=True)).clamp(max=n_seq - 1)  # a chunk's sequence

    def padded(v):
        w = torch.zeros(nc * Q, *v.shape[1:], dtype=v.dtype, device=DEV)
        w[slot] = v
        return w.view(nc, Q, *v.shape[1:])

    dt, lam = _plain_dt(s)
    xbc = padded(s["xbc"].float())
    x = xbc[..., :H * P].reshape(nc, Q, H, P).transpose(1, 2).contiguous()
    B = xbc[..., H * P:H * P + G * N].reshape(nc, Q, G, N).transpose(1, 2).contiguous()
    Cm = xbc[..., H * P + G * N:].reshape(nc, Q, G, N).transpose(1, 2).contiguous()
    dt, lam = padded(dt).transpose(1, 2).contiguous(), padded(lam.double()).transpose(1, 2)
    L = torch.cumsum(lam, -1)  # [nc][H][Q]
    xdt = x * dt[..., None]

    # within a chunk
    low = torch.tril(torch.ones(Q, Q, dtype=torch.bool, device=DEV))
    decay = (L[..., :, None] - L[..., None, :]).float().masked_fill(~low, -math.inf).exp()
    CB = Cm @ B.transpose(-1, -2).contiguous()  # [nc][G][Q][Q]
    M = (decay.view(nc, G, H // G, Q, Q) * CB[:, :, None]).view(nc, H, Q, Q)
    y = M @ xdt

    # each chunk's own state, then the state that each chunk starts from
    tail = (L[..., -1:] - L).float().exp()
    own_S = (xdt * tail[..., None]).transpose(-1, -2).reshape(nc, G, H // G * P, Q) @ B  # [nc][G][H/G*P][N]
    own_S = own_S.reshape(nc, H, P * N).transpose(0, 1).contiguous()
    total = torch.cumsum(L[..., -1], 0).t()  # [H][nc], summed over all chunks before and this one
    before = total - L[..., -1].t()
    same = (cseq[:, None] == cseq[None, :]) & (chunk[:, None] > chunk[None, :])
    W = (before[:, :, None] - total[:, None, :]).float().masked_fill(~same, -math.inf).exp()
    S = W @ own_S  # [H][nc][P*N]
    start = (before - before.gather(1, first.clamp(max=nc - 1)[cseq][None].expand(H, nc))).float().exp()
    S = S + start[:, :, None] * s["state"].transpose(0, 1).reshape(H, n_seq, P * N)[:, cseq]
    Sg = S.view(G, H // G, nc, P, N).permute(2, 0, 4, 1, 3).reshape(nc, G, N, H // G * P).contiguous()
    inter = (Cm @ Sg).view(nc, G, Q, H // G, P).transpose(2, 3).reshape(nc, H, Q, P)
    y = y + L.float().exp()[..., None] * inter + s["D"][None, :, None, None] * x
    y = y.transpose(1, 2).reshape(nc * Q, H * P)[slot].to(s["y"].dtype)

    # after a sequence's last chunk
    end = (first + chunks - 1).clamp(min=0)
    after = L[..., -1].t().float().exp()[:, end, None] * S[:, end] + own_S[:, end]
    after = after.view(H, n_seq, P, N).transpose(0, 1)
    return {"y": y, "state": torch.where((chunks > 0)[:, None, None, None], after, s["state"])}


def _plain_step(s):
    H, P, G, N, n = s["H"], s["P"], s["G"], s["N"], s["n_seq"]
    c, hist = _plain_conv(s, s["xbc"])
    x = c[:, :H * P].view(n, H, P)
    B = c[:, H * P:H * P + G * N].view(n, G, N).repeat_interleave(H // G, 1)
    Cm = c[:, H * P + G * N:].view(n, G, N).repeat_interleave(H // G, 1)
    dt, lam = _plain_dt(s)
    S = torch.exp(lam)[..., None, None] * s["state"] + (dt[..., None] * x)[..., None] * B[:, :, None, :]
    y = (S * Cm[:, :, None, :]).sum(-1) + s["D"][None, :, None] * x
    return {"y": y.reshape(n, H * P).to(s["y"].dtype), "state": S, "hist": hist}


def _plain(s):
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "conv":
        out, hist = _plain_conv(s, s["xbc"])
        return {"out": out.to(s["out_buf"].dtype), "hist": hist}
    return _plain_scan(s) if s["op"] == "scan" else _plain_step(s)


# ----------------------------------------------------------- the framework's
def _own(s):
    from gated_deltanet_linear_pre_amd import ssm

    if "shape" not in s:  # sizes and workspace: made once, and kept, as a program keeps them
        if s["op"] == "norm":
            s["shape"] = ssm.make_norm_shape(s["rows"], s["channels"], s["groups"], x=s["x"], io=s["io"], eps=1e-5,
                                             centre=s["centre"], gate_last=s["last"])
        else:
            strided = s["op"] != "scan"
            s["shape"] = ssm.make_ssm_shape(s["H"], s["P"], s["G"], s["N"], s["n_seq"], s["T"], s["max_T"], io=s["io"],
                                            out=s.get("out", s["io"]), conv_width=s.get("K", 4),
                                            xbc_stride=s["xbc"].stride(0) if strided else 0,
                                            dt_stride=s["dt"].stride(0) if strided else 0)
        if s["op"] == "scan":
            s["workspace"] = torch.empty(max(256, ssm.gdn_ssm_scan_workspace_bytes(s["shape"])), dtype=torch.uint8, device=DEV)
    if s["op"] == "norm":
        ssm.gdn_group_norm(s["shape"], s["x_in"], s["z"], s["weight"], s["bias_in"], s["y"])
        return {"y": s["y"]}
    if s["op"] == "conv":
        ssm.gdn_ssm_conv(s["shape"], s["cu"], s["xbc"], s["conv_w"], s["conv_b"], s["hist"], s["hist_out"], s["out_buf"])
        return {"out": s["out_buf"], "hist": s["hist_out"]}
    if s["op"] == "scan":
        ssm.gdn_ssm_scan(s["shape"], s["cu"], s["xbc"], s["dt"], s["A_log"], s["dt_bias"], s["D"], s["state"], s["state_out"],
                         s["y"], s["workspace"])
        return {"y": s["y"], "state": s["state_out"]}
    ssm.gdn_ssm_step(s["shape"], s["xbc"], s["conv_w"], s["conv_b"], s["dt"], s["A_log"], s["dt_bias"], s["D"], s["hist"],
                     s["hist_out"], s["state"], s["state_out"], s["y"])
    return {"y": s["y"], "state": s["state_out"], "hist": s["hist_out"]}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def work(case):
    b = {"f32": 4, "f16": 2, "bf16": 2}
    io = b[case["io"]]
    if case["op"] == "norm":
        n = case["rows"] * case["channels"]
        return {"bytes": n * (b[case["x"]] + 2 * io) + case["channels"] * io, "flops": 12 * n}
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    lens = _lens(case)
    C, T, n_seq = H * P + 2 * G * N, sum(lens), len(lens)
    conv_bytes, conv_flops, K = 0, 0, case.get("K", 0)
    if K:
        conv_bytes = T * C * io + 2 * n_seq * (K - 1) * C * io + C * (K + 1) * io
        conv_flops = T * C * (2 * K + 5)
    if case["op"] == "conv":
        return {"bytes": conv_bytes + T * C * io, "flops": conv_flops}
    rest = T * H * io + T * H * P * b[case["out"]] + 2 * n_seq * H * P * N * 4 + 3 * H * 4
    return {"bytes": rest + (conv_bytes or T * C * io), "flops": conv_flops + T * H * P * (5 * N + 4)}


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """One token after the other, one row after the other, in 64 bits."""
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if case["op"] == "norm":
        size = case["channels"] // case["groups"]
        sig = d["z"] / (1 + torch.exp(-d["z"]))
        v = (d["x_in"] if case["last"] else d["x_in"] * sig).unflatten(1, (case["groups"], size))
        m = v.sum(2, keepdim=True) / size if case["centre"] else torch.zeros_like(v[..., :1])
        var = ((v - m) ** 2).sum(2, keepdim=True) / size
        y = ((v - m) * (var + 1e-5) ** -0.5).flatten(1) * d["weight"]
        if case["bias"]:
            y = y + d["bias_in"]
        return {"y": y * sig if case["last"] else y}
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    lens = _lens(case)
    begins = [sum(lens[:i]) for i in range(len(lens))]
    if case["op"] != "scan":
        K = case["K"]
        out, hist = torch.empty_like(d["xbc"]), []
        for n, (b, T) in enumerate(zip(begins, lens)):
            X = torch.cat([d["hist"][n], d["xbc"][b:b + T]])
            v = sum(X[k:k + T] * d["conv_w"][:, k] for k in range(K)) + d["conv_b"]
            out[b:b + T] = v / (1 + torch.exp(-v))
            hist.append(X[T:])
        hist = torch.stack(hist)
        if case["op"] == "conv":
            return {"out": out, "hist": hist}
        xbc = out
    else:
        xbc = d["xbc"]
    u = d["dt"] + d["dt_bias"]
    dt = torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs()))
    a = torch.exp(-torch.exp(d["A_log"]) * dt)
    S, y = d["state"].clone(), torch.empty(sum(lens), H, P, dtype=torch.float64, device=DEV)
    order = sorted(range(len(lens)), key=lambda n: -lens[n])  # the longest first: those that still run are the first ones
    S = S[order]
    heads = torch.arange(H, device=DEV) // (H // G)
    at0 = torch.tensor([begins[n] for n in order], device=DEV)
    for t in range(max(lens)):
        live = sum(lens[n] > t for n in order)
        at = at0[:live] + t
        row = xbc[at]
        x = row[:, :H * P].reshape(live, H, P)
        B = row[:, H * P:H * P + G * N].reshape(live, G, N)[:, heads]
        Cv = row[:, H * P + G * N:].reshape(live, G, N)[:, heads]
        S[:live].mul_(a[at][:, :, None, None]).add_((dt[at][:, :, None] * x)[..., None] * B[:, :, None, :])
        y[at] = (S[:live] @ Cv[..., None])[..., 0] + d["D"][:, None] * x
    state = torch.empty_like(S)
    state[order] = S
    res = {"y": y.reshape(-1, H * P), "state": state}
    return res if case["op"] == "scan" else {**res, "hist": hist}
