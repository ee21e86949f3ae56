"""What the binding of include/gdn_ssm.h refuses: tensors that are not what the
shape says.  No GPU: one host tensor a call, refused for its layout before its
place is looked at; the other addresses are never used."""
import pytest
import torch

from gated_deltanet_linear_pre_amd import ssm

P = 0x10000
H, HD, G, N, K, T, n = 8, 64, 2, 128, 4, 100, 3
C = H * HD + 2 * G * N
BF, F32 = torch.bfloat16, torch.float32

# argument: (type, elements)
DENSE = {
    "gdn_ssm_conv": dict(cu_seqlens=(torch.int32, n + 1), xbc=None, conv_w=(BF, C * K), conv_b=(BF, C), hist=(BF, n * (K - 1) * C),
                         hist_out=(BF, n * (K - 1) * C), out=(BF, T * C)),
    "gdn_ssm_scan": dict(cu_seqlens=(torch.int32, n + 1), xbc=(BF, T * C), dt=None, A_log=(F32, H), dt_bias=(F32, H), D=(F32, H),
                         state=(F32, n * H * HD * N), state_out=(F32, n * H * HD * N), y=(F32, T * H * HD)),
    "gdn_ssm_step": dict(xbc=None, conv_w=(BF, C * K), conv_b=(BF, C), dt=None, A_log=(F32, H), dt_bias=(F32, H), D=(F32, H),
                         hist=(BF, n * (K - 1) * C), hist_out=(BF, n * (K - 1) * C), state=(F32, n * H * HD * N),
                         state_out=(F32, n * H * HD * N), y=(F32, n * H * HD)),
    "gdn_group_norm": dict(x=None, z=None, weight=(BF, 512), bias=(BF, 512), y=(BF, 10 * 512)),
}
ROWS = {
    "gdn_ssm_conv": dict(xbc=(BF, T, C, C + 16)),
    "gdn_ssm_scan": dict(dt=(BF, T, H, C + 16)),
    "gdn_ssm_step": dict(xbc=(BF, n, C, C + 16), dt=(BF, n, H, C + 16)),
    "gdn_group_norm": dict(x=(F32, 10, 512, 528), z=(BF, 10, 512, 544)),
}


def shape(name):
    if name == "gdn_group_norm":
        return ssm.make_norm_shape(10, 512, 4, x="f32", io="bf16", x_stride=528, z_stride=544)
    t, m = (n, 1) if name == "gdn_ssm_step" else (T, T)
    return ssm.make_ssm_shape(H, HD, G, N, n, t, m, io="bf16", out="f32", xbc_stride=C + 16, dt_stride=C + 16)


def call(name, **over):
    args = {**{k: P for k in DENSE[name]}, **over}
    return getattr(ssm, name)(shape(name), **args, stream=0)


IN_HOST = "host memory"  # what is left to refuse of a host tensor whose layout is right


@pytest.mark.parametrize("name,arg", [(f, a) for f, d in DENSE.items() for a, v in d.items() if v])
def test_dense_tensors(name, arg):
    dtype, size = DENSE[name][arg]
    with pytest.raises(ValueError, match=IN_HOST):
        call(name, **{arg: torch.zeros(size, dtype=dtype)})
    with pytest.raises(ValueError, match=IN_HOST):
        call(name, **{arg: torch.zeros(size + 3, dtype=dtype)})
    with pytest.raises(ValueError, match=f"{arg} has {size - 1} elements of {size}"):
        call(name, **{arg: torch.zeros(size - 1, dtype=dtype)})
    with pytest.raises(ValueError, match=f"{arg} has gaps"):
        call(name, **{arg: torch.zeros(size, 2, dtype=dtype)[:, 0]})
    with pytest.raises(ValueError, match=f"{arg} is torch.float64"):
        call(name, **{arg: torch.zeros(size, dtype=torch.float64)})


@pytest.mark.parametrize("name,arg", [(f, a) for f, d in ROWS.items() for a in d])
def test_tensors_of_rows(name, arg):
    dtype, rows, cols, stride = ROWS[name][arg]
    wide = torch.zeros(rows, stride, dtype=dtype)
    for x in (wide, wide[:, :cols], wide[:, 5:5 + cols] if stride >= cols + 5 else wide):
        with pytest.raises(ValueError, match=IN_HOST):
            call(name, **{arg: x})
    other = torch.zeros(rows, stride + 8, dtype=dtype)
    for x in (wide[:, :cols].contiguous(), wide[:-1, :cols], wide[:, :cols - 1], other[:, :cols], wide.t(), wide[::2, :cols],
              torch.zeros(rows, 2 * stride, dtype=dtype)[:, ::2]):
        with pytest.raises(ValueError, match=f"{arg} of .* is not {rows} rows of {cols} elements, {stride} apart"):
            call(name, **{arg: x})
    with pytest.raises(ValueError, match=f"{arg} is torch.float64"):
        call(name, **{arg: wide.double()})


def test_workspace_bytes():
    ws = torch.zeros(4096, dtype=torch.uint8)
    args = [P] * 9
    for given in (4097, -1):
        with pytest.raises(ValueError, match="a workspace of 4096 bytes"):
            ssm.gdn_ssm_scan(shape("gdn_ssm_scan"), *args, ws, workspace_bytes=given, stream=0)
    with pytest.raises(ValueError, match="workspace has gaps"):
        ssm.gdn_ssm_scan(shape("gdn_ssm_scan"), *args, ws[::2], stream=0)
    with pytest.raises(ValueError, match=IN_HOST):
        ssm.gdn_ssm_scan(shape("gdn_ssm_scan"), *args, ws, stream=0)
    with pytest.raises(ssm.GdnError):  # an address says nothing of its size
        ssm.gdn_ssm_scan(ssm.make_ssm_shape(64, 64, 8, 128, 1, 16384, 16384), *args, P, stream=0)


def test_a_changed_shape_is_looked_at_again():
    s = ssm.make_norm_shape(10, 512, 4, x="bf16", io="bf16")
    x = torch.zeros(10, 512, dtype=BF)
    with pytest.raises(ValueError, match=IN_HOST):
        ssm.gdn_group_norm(s, x, None, None, None, P, stream=0)
    s.rows = 11
    with pytest.raises(ValueError, match="x of .* is not 11 rows"):
        ssm.gdn_group_norm(s, x, None, None, None, P, stream=0)
