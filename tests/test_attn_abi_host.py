"""Host-side checks of include/gdn_attn.h: exports, struct layouts, every refusal,
workspaces and the table of rotary frequencies.  No GPU: each call fails validation or
has no rows, so nothing is enqueued and the fake addresses are never touched."""
import ctypes
import itertools
import json
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from gated_deltanet_linear_pre_amd import attn
from gated_deltanet_linear_pre_amd import binding as B

P = 0x10000  # 64 KiB-aligned fake device address, never dereferenced
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(os.path.dirname(B.HEADER), "gdn_attn.h")


def shape(**kw):
    d = dict(heads=8, kv_heads=2, head_dim=128, n_seq=3, total_T=100, max_T=60, max_kv=4000, n_pages=500, table_pages=250,
             page_size=16, io="bf16", rope_dim=64)
    d.update(kw)
    return attn.make_attn_shape(**d)


def step_shape(**kw):
    return shape(**{**dict(total_T=3, max_T=1), **kw})


def append(s, **over):
    a = dict(cu=P, kv=P, table=P, pos=P, q=P, k=P, v=P, freq=P, qn=P, kn=P, q_out=P, kc=P, vc=P)
    a.update(over)
    return attn.gdn_attn_append(s, *a.values(), stream=0, check=False)


def prefill(s, ws_bytes=1 << 40, **over):
    a = dict(cu=P, kv=P, table=P, q=P, kc=P, vc=P, gate=P, out=P, ws=P)
    a.update(over)
    return attn.gdn_attn_prefill(s, *a.values(), workspace_bytes=ws_bytes, stream=0, check=False)


def step(s, ws_bytes=1 << 40, **over):
    a = dict(kv=P, table=P, q=P, kc=P, vc=P, gate=P, out=P, ws=P)
    a.update(over)
    return attn.gdn_attn_step(s, *a.values(), workspace_bytes=ws_bytes, stream=0, check=False)


def copy(s, n=4, **over):
    a = dict(pairs=P, n=n, kc=P, vc=P)
    a.update(over)
    return attn.gdn_attn_copy_pages(s, *a.values(), stream=0, check=False)


def test_exports_and_struct_layouts():
    names = set(re.findall(r"^(?:int|size_t) (gdn_\w+)\(", open(HEADER).read(), re.M))
    assert names == {"gdn_attn_append", "gdn_attn_prefill", "gdn_attn_prefill_workspace_bytes", "gdn_attn_step",
                     "gdn_attn_step_workspace_bytes", "gdn_attn_copy_pages", "gdn_attn_rope_freqs"}
    for n in names:
        assert hasattr(attn.lib(), n), n
    assert ctypes.sizeof(attn.gdn_attn_shape) == 8 * 4 + 11 * 8 + 4 * 4 and attn.gdn_attn_shape.scale.offset == 120
    assert ctypes.sizeof(attn.gdn_rope) == 2 * 4 + 5 * 8


@pytest.mark.parametrize("over,code", [
    (dict(heads=0), -2), (dict(kv_heads=0), -2), (dict(heads=7), -2), (dict(heads=4098), -2), (dict(heads=258), -2),
    (dict(head_dim=0), -2), (dict(head_dim=32), -2), (dict(head_dim=80), -2), (dict(head_dim=512), -2),
    (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=2048), -2), (dict(page_size=-16), -2),
    (dict(n_seq=0), -2), (dict(n_seq=65537), -2), (dict(io=3), -5), (dict(io=-1), -5), (dict(n_pages=0), -2),
    (dict(n_pages=1 << 31), -2), (dict(table_pages=0), -2), (dict(table_pages=(1 << 30) + 1), -2), (dict(max_kv=-1), -2),
    (dict(max_kv=4001), -2), (dict(max_kv=(1 << 30) + 1, table_pages=1 << 30), -2), (dict(page_stride=2 * 16 * 128 - 8), -2),
    (dict(page_stride=-1), -2), (dict(page_stride=1 << 41), -2), (dict(page_stride=1 << 40, n_pages=1 << 17), -2),
    (dict(page_stride=2 * 16 * 128 + 4), -3), (dict(q_stride=8 * 128 - 8), -2), (dict(gate_stride=8 * 128 - 8), -2),
    (dict(k_stride=2 * 128 - 8), -2), (dict(v_stride=2 * 128 - 8), -2), (dict(q_stride=8 * 128 + 4), -3),
    (dict(gate_stride=8 * 128 + 4), -3), (dict(k_stride=2 * 128 + 4), -3), (dict(v_stride=2 * 128 + 4), -3),
    (dict(io="f32", q_stride=8 * 128 + 2), -3), (dict(rope_dim=-16), -2), (dict(rope_dim=8), -2), (dict(rope_dim=144), -2),
    (dict(window=-1), -2), (dict(scale=0.0), -2), (dict(scale=-1.0), -2), (dict(scale=float("nan")), -2),
    (dict(scale=float("inf")), -2), (dict(rope_scale=-1.0), -2), (dict(rope_scale=float("inf")), -2), (dict(eps=-1.0), -2),
    (dict(eps=float("nan")), -2),
])
def test_bad_shapes_are_refused_by_every_entry_point(over, code):
    assert append(shape(**over)) == code and prefill(shape(**over)) == code and copy(shape(**over)) == code
    assert step(step_shape(**over)) == code
    assert attn.gdn_attn_prefill_workspace_bytes(shape(**over)) == 0
    assert attn.gdn_attn_step_workspace_bytes(step_shape(**over)) == 0


@pytest.mark.parametrize("over", [dict(total_T=-1), dict(max_T=101), dict(max_T=-1), dict(total_T=(1 << 26) + 1, max_T=1)])
def test_bad_lengths_are_refused(over):
    assert append(shape(**over)) == -2 and prefill(shape(**over)) == -2


def test_flags_and_reserved():
    for field, value in (("flags", 2), ("flags", -1), ("reserved", 1)):
        s = shape()
        setattr(s, field, value)
        assert append(s) == -2 and prefill(s) == -2 and copy(s) == -2


def test_step_takes_one_token_per_sequence():
    assert step(step_shape(total_T=4)) == -2 and step(step_shape(total_T=4, max_T=2)) == -2
    assert step(step_shape(total_T=0, max_T=0)) == -2 and step(step_shape(max_T=0)) == -2


def test_null_shape():
    L = attn.lib()
    assert L.gdn_attn_append(None, *([P] * 13), None) == -1
    assert L.gdn_attn_prefill(None, *([P] * 9), 1 << 30, None) == -1 and L.gdn_attn_step(None, *([P] * 8), 1 << 30, None) == -1
    assert L.gdn_attn_copy_pages(None, P, 1, P, P, None) == -1
    assert L.gdn_attn_prefill_workspace_bytes(None) == 0 and L.gdn_attn_step_workspace_bytes(None) == 0


@pytest.mark.parametrize("call,s,needed,aligned", [
    (append, shape(), ["cu", "kv", "table", "q", "k", "v", "freq", "q_out", "kc", "vc"],
     dict(cu=2, kv=2, table=2, pos=2, q=8, k=8, v=8, freq=2, qn=8, kn=8, q_out=8, kc=8, vc=8)),
    (prefill, shape(), ["cu", "kv", "table", "q", "kc", "vc", "out"],
     dict(cu=2, kv=2, table=2, q=8, kc=8, vc=8, gate=8, out=8, ws=128)),
    (step, step_shape(), ["kv", "table", "q", "kc", "vc", "out", "ws"], dict(kv=2, table=2, q=8, kc=8, vc=8, gate=8, out=8, ws=128)),
    (copy, shape(), ["pairs", "kc", "vc"], dict(pairs=2, kc=8, vc=8)),
], ids=["append", "prefill", "step", "copy"])
def test_null_and_unaligned_pointers_are_refused(call, s, needed, aligned):
    for name in needed:
        assert call(s, **{name: None}) == -1, name
    for name, off in aligned.items():
        assert call(s, **{name: P + off}) == -3, name


def test_calls_without_rows():
    none = shape(total_T=0, max_T=0)
    assert append(none, q=None, k=None, v=None, q_out=None) == 0 and prefill(none, q=None, out=None) == 0
    assert append(shape(max_T=0)) == 0 and prefill(shape(max_T=0)) == 0
    assert copy(shape(), n=0) == 0 and copy(shape(), n=0, pairs=None) == 0
    assert copy(shape(), n=-1) == -2 and copy(shape(), n=(1 << 24) + 1) == -2


@pytest.mark.parametrize("call,size,s", [
    (step, attn.gdn_attn_step_workspace_bytes, step_shape()), (step, attn.gdn_attn_step_workspace_bytes, step_shape(max_kv=1)),
    (prefill, attn.gdn_attn_prefill_workspace_bytes, shape()),
], ids=["step", "short", "prefill"])
def test_workspaces_are_checked(call, size, s):
    need = size(s)
    assert need > 0 and need % 256 == 0
    assert call(s, ws_bytes=need - 1) == -4 and call(s, ws=None) == -1 and call(s, ws_bytes=0) == -4


QUERY = """
import json, sys
from gated_deltanet_linear_pre_amd import attn
out = []
for H, KV, D, page, n, T, kv, window, io in json.load(sys.stdin):
    kw = dict(max_kv=kv, n_pages=1 << 20, table_pages=max(1, -(-kv // page)), page_size=page, window=window, io=io)
    out.append((attn.gdn_attn_prefill_workspace_bytes(attn.make_attn_shape(H, KV, D, n, T, T, **kw)),
                attn.gdn_attn_step_workspace_bytes(attn.make_attn_shape(H, KV, D, n, n, 1, **kw))))
print(json.dumps(out))
"""


def test_workspaces_of_the_largest_and_smallest_sizes():
    # in a process of its own: a division by zero there would end this one
    cases = [(*c[:5], T, *c[5:]) for c in itertools.product(
        (1, 4096), (1,), (64, 256), (16, 1024), (1, 65536), (0, 1, 1 << 30), (0, 1, 1 << 62), ("f32", "bf16"))
        for T in (0, 1, 1 << 26)]
    cases = [(H, H // 128 if H > 128 else KV, *c) for H, KV, *c in cases]
    r = subprocess.run([sys.executable, "-c", QUERY], input=json.dumps(cases), capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, f"the query ended its process: {r.returncode}\n{r.stderr[-500:]}"
    for (H, KV, D, page, n, T, kv, window, io), (a, b) in zip(cases, json.loads(r.stdout)):
        # at most 512 parts of 128 rows (16 to 128 in a step), twice, and a record for each
        assert 0 <= a <= 512 * (2 * 128 * (4 * D + 8) + 64) and 256 <= b <= 256 * (2 * (128 if H > 16 * KV else 16) * (4 * D + 8) + 64), (H, KV, D, page, n, T, kv, window, io)
        if T >= 1 << 20:
            assert a == 0  # many rows: nothing is cut


# ------------------------------------------------------------ rotary frequencies
def frequencies(kind, r, base, factor, trained, slow, fast):
    if kind == "base":
        base *= factor ** (r / (r - 2))
    f = base ** (-2.0 * np.arange(r // 2) / r)
    if kind == "linear":
        f = f / factor
    if kind == "parts":
        keep = np.clip((trained * f / (2 * math.pi) - slow) / (fast - slow), 0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f, 0.1 * math.log(factor) + 1 if kind == "parts" else 1.0


@pytest.mark.parametrize("kind", list(attn.ROPE_KIND))
@pytest.mark.parametrize("r,base,factor", [(16, 1e4, 1.0), (64, 1e4, 4.0), (96, 1e7, 2.5), (256, 5e5, 40.0)])
def test_rope_freqs(kind, r, base, factor):
    got, scale = attn.gdn_attn_rope_freqs(r, base, kind, factor, 4096.0, 1.0, 32.0)
    want, s = frequencies(kind, r, base, factor, 4096.0, 1.0, 32.0)
    assert got.dtype == torch.float32 and got.shape == (r // 2,)
    # one rounding to fp32; the 64-bit powers and quotients of both sides are off by some 2^-50
    assert (np.abs(got.double().numpy() - want) <= want * (2.0 ** -24 + 2.0 ** -48)).all() and abs(scale - s) <= s * 2.0 ** -23
    assert got[0] == 1.0 or kind == "linear"


def test_rope_freqs_at_their_ends():
    plain, _ = attn.gdn_attn_rope_freqs(64, 1e4)
    base, _ = attn.gdn_attn_rope_freqs(64, 1e4, "base", 8.0)
    parts, _ = attn.gdn_attn_rope_freqs(64, 1e4, "parts", 8.0, 1000.0, 1.0, 32.0)
    assert abs(base[-1] * 8 / plain[-1] - 1) < 2.0 ** -20 and base[0] == plain[0]  # the slowest by factor, the fastest as it is
    turns = 1000.0 * plain.double() / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], plain[turns >= 32]) and (turns >= 32).any()
    assert torch.allclose(parts[turns <= 1] * 8, plain[turns <= 1], rtol=2.0 ** -22, atol=0) and (turns <= 1).any()


@pytest.mark.parametrize("kw", [
    dict(rope_dim=0), dict(rope_dim=8), dict(rope_dim=24), dict(rope_dim=272), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(kind=4), dict(kind=-1), dict(kind="linear", factor=0.5), dict(kind="base", factor=float("nan")),
    dict(kind="parts", factor=2.0, trained=0.0), dict(kind="parts", factor=2.0, trained=10.0, slow=-1.0),
    dict(kind="parts", factor=2.0, trained=10.0, slow=4.0, fast=4.0), dict(kind="parts", factor=2.0, trained=10.0, fast=float("inf")),
    dict(kind="parts", factor=2.0, trained=10.0, slow=float("nan")),
])
def test_rope_freqs_refusals(kw):
    with pytest.raises(B.GdnError):
        attn.gdn_attn_rope_freqs(**{**dict(rope_dim=64), **kw})


def test_rope_freqs_null():
    r, out, s = attn.gdn_rope(0, 16, 1e4, 1, 1, 1, 32), torch.zeros(8), ctypes.c_float()
    f = attn.lib().gdn_attn_rope_freqs
    assert f(None, out.data_ptr(), ctypes.byref(s)) == -1 and f(ctypes.byref(r), None, ctypes.byref(s)) == -1
    assert f(ctypes.byref(r), out.data_ptr(), None) == -1 and f(ctypes.byref(r), out.data_ptr(), ctypes.byref(s)) == 0
