"""Host-side checks of include/gdn_ssm.h: exports, struct layouts, and every
refusal.  No GPU: each call fails validation, so nothing is enqueued and the
fake addresses are never touched."""
import ctypes
import os
import re

import pytest
import torch

from gated_deltanet_linear_pre_amd import binding as B
from gated_deltanet_linear_pre_amd import ssm

P = 0x10000  # 64 KiB-aligned fake device address, never dereferenced
HEADER = os.path.join(os.path.dirname(B.HEADER), "gdn_ssm.h")


def shape(**kw):
    d = dict(heads=8, head_dim=64, groups=2, state_dim=128, n_seq=2, total_T=100, max_T=60, io="bf16")
    d.update(kw)
    return ssm.make_ssm_shape(**d)


def step_shape(**kw):
    return shape(**{**dict(n_seq=3, total_T=3, max_T=1), **kw})


def conv(s, **over):
    a = dict(cu=P, xbc=P, w=P, b=P, hist=P, hist_out=P, out=P)
    a.update(over)
    return ssm.gdn_ssm_conv(s, *a.values(), stream=0, check=False)


def scan(s, ws_bytes=1 << 40, **over):
    a = dict(cu=P, xbc=P, dt=P, A_log=P, dt_bias=P, D=P, state=P, state_out=P, y=P, ws=P)
    a.update(over)
    return ssm.gdn_ssm_scan(s, *a.values(), workspace_bytes=ws_bytes, stream=0, check=False)


def step(s, **over):
    a = dict(xbc=P, w=P, b=P, dt=P, A_log=P, dt_bias=P, D=P, hist=P, hist_out=P, state=P, state_out=P, y=P)
    a.update(over)
    return ssm.gdn_ssm_step(s, *a.values(), stream=0, check=False)


def norm(s, **over):
    a = dict(x=P, z=P, w=P, b=P, y=P)
    a.update(over)
    return ssm.gdn_group_norm(s, *a.values(), stream=0, check=False)


def test_exports_and_struct_layouts():
    names = set(re.findall(r"^(?:int|size_t) (gdn_\w+)\(", open(HEADER).read(), re.M))
    assert names == {"gdn_ssm_conv", "gdn_ssm_scan", "gdn_ssm_scan_workspace_bytes", "gdn_ssm_step", "gdn_group_norm"}
    for n in names:
        assert hasattr(ssm.lib(), n), n
    assert ctypes.sizeof(ssm.gdn_ssm_shape) == 8 * 4 + 4 * 8 + 2 * 4 and ssm.gdn_ssm_shape.dt_min.offset == 64
    assert ctypes.sizeof(ssm.gdn_norm_shape) == 8 + 4 * 4 + 2 * 8 + 4 + 4


@pytest.mark.parametrize("over,code", [
    (dict(heads=0), -2), (dict(heads=4098, groups=2), -2), (dict(groups=0), -2), (dict(groups=3), -2),
    (dict(head_dim=0), -2), (dict(head_dim=24), -2), (dict(head_dim=272), -2), (dict(state_dim=16), -2),
    (dict(state_dim=96), -2), (dict(state_dim=512), -2), (dict(conv_width=1), -2), (dict(conv_width=5), -2),
    (dict(n_seq=0), -2), (dict(n_seq=(1 << 20) + 1), -2), (dict(io=3), -5), (dict(io="f16", out="bf16"), -5),
    (dict(io="f32", out="f16"), -5), (dict(dt_min=-1.0), -2), (dict(dt_min=float("nan")), -2),
    (dict(dt_min=1.0, dt_max=0.5), -2), (dict(dt_max=float("nan")), -2), (dict(dt_stride=7), -2),
    (dict(xbc_stride=8 * 64 + 2 * 2 * 128 - 8), -2),
])
def test_bad_shapes_are_refused_by_every_entry_point(over, code):
    assert conv(shape(**over)) == code and scan(shape(**over)) == code
    assert step(step_shape(**{k: v for k, v in over.items() if k != "n_seq"})) == code or "n_seq" in over
    assert ssm.gdn_ssm_scan_workspace_bytes(shape(**over)) == 0


@pytest.mark.parametrize("over", [dict(total_T=-1), dict(max_T=101), dict(total_T=(1 << 27) + 1, max_T=1)])
def test_bad_lengths_are_refused(over):
    assert conv(shape(**over)) == -2 and scan(shape(**over)) == -2


def test_step_takes_one_token_per_sequence():
    assert step(step_shape(total_T=4)) == -2 and step(step_shape(max_T=2)) == -2
    assert step(step_shape(total_T=0, max_T=0)) == -2


@pytest.mark.parametrize("io,stride", [("bf16", 8 * 64 + 512 + 4), ("f32", 8 * 64 + 512 + 2)])
def test_unaligned_rows_are_refused(io, stride):
    assert conv(shape(io=io, xbc_stride=stride)) == -3
    assert step(step_shape(io=io, xbc_stride=stride)) == -3


def test_null_shape():
    assert ssm.lib().gdn_ssm_conv(None, *([P] * 7), None) == -1
    assert ssm.lib().gdn_group_norm(None, *([P] * 5), None) == -1
    assert ssm.lib().gdn_ssm_scan_workspace_bytes(None) == 0


@pytest.mark.parametrize("call,s,needed,aligned", [
    (conv, shape(), ["cu", "xbc", "w", "out"], dict(cu=2, xbc=8, w=8, b=8, hist=8, hist_out=8, out=8)),
    (scan, shape(), ["cu", "xbc", "dt", "A_log", "dt_bias", "y"],
     dict(cu=2, xbc=8, dt=1, A_log=2, dt_bias=2, D=2, state=8, state_out=8, y=8, ws=128)),
    (step, step_shape(), ["xbc", "w", "dt", "A_log", "dt_bias", "y"],
     dict(xbc=8, w=8, b=8, dt=1, A_log=2, dt_bias=2, D=2, hist=8, hist_out=8, state=8, state_out=8, y=8)),
    (norm, ssm.make_norm_shape(5, 64, 2), ["x", "y"], dict(x=8, z=8, w=8, b=8, y=8)),
], ids=["conv", "scan", "step", "norm"])
def test_null_and_unaligned_pointers_are_refused(call, s, needed, aligned):
    for name in needed:
        assert call(s, **{name: None}) == -1, name
    for name, off in aligned.items():
        assert call(s, **{name: P + off}) == -3, name


def test_scan_workspace_is_checked():
    s = shape(heads=64, groups=8, total_T=16384, max_T=16384, n_seq=1)
    need = ssm.gdn_ssm_scan_workspace_bytes(s)
    if need:
        assert scan(s, ws_bytes=need - 1) == -4 and scan(s, ws=None) == -1


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -2), (dict(rows=(1 << 27) + 1), -2), (dict(channels=60), -2), (dict(channels=8, groups=2), -2),
    (dict(groups=0), -2), (dict(groups=3), -2), (dict(channels=16392, groups=1), -2), (dict(channels=65544, groups=8), -2),
    (dict(x="f16"), -5), (dict(io=9), -5), (dict(eps=-1.0), -2), (dict(eps=float("inf")), -2),
    (dict(x_stride=56), -2), (dict(z_stride=56), -2), (dict(z_stride=68), -3), (dict(x_stride=66), -3),
])
def test_bad_norm_shapes_are_refused(over, code):
    assert norm(ssm.make_norm_shape(**{**dict(rows=5, channels=64, groups=2), **over})) == code


def test_norm_flags_and_no_rows():
    s = ssm.make_norm_shape(5, 64, 2)
    s.flags = 4
    assert norm(s) == -2
    assert norm(ssm.make_norm_shape(0, 64, 2), x=None, y=None) == 0


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        ssm.gdn_group_norm(ssm.make_norm_shape(1, 8, 1, x="f32", io="f32"), torch.zeros(8), None, None, None, torch.zeros(8), stream=0)
