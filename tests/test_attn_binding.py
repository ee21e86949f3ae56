"""What the binding of include/gdn_attn.h refuses: tensors that are not what the
shape says.  No GPU: one host tensor a call, refused for its layout before its
place is looked at; the other addresses are never used."""
import pytest
import torch

from gated_deltanet_linear_pre_amd import attn

P = 0x10000
H, KV, D, n, T, TP, N, PAGE = 8, 2, 64, 3, 100, 40, 20, 16
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
CACHE = 2 * KV * PAGE * D  # elements of a page of K and V

# argument: (type, elements)
ATTENTION = dict(kv_len=(I32, n), page_table=(I32, n * TP), q=None, k_cache=None, v_cache=None, gate=None, out=(BF, T * H * D), workspace=None)
DENSE = {
    "gdn_attn_append": dict(cu_seqlens=(I32, n + 1), kv_len=(I32, n), page_table=(I32, n * TP), positions=(I32, T), q=None, k=None, v=None,
                            inv_freq=(F32, 16), q_norm=(BF, D), k_norm=(BF, D), q_out=(BF, T * H * D), k_cache=None, v_cache=None),
    "gdn_attn_prefill": dict(cu_seqlens=(I32, n + 1), **ATTENTION),
    "gdn_attn_step": dict(ATTENTION, out=(BF, n * H * D)),
}
ROWS = {
    "gdn_attn_append": dict(q=(T, H * D, 1056), k=(T, KV * D, 1040), v=(T, KV * D, 1072)),
    "gdn_attn_prefill": dict(q=(T, H * D, 1056), gate=(T, H * D, 1088)),
    "gdn_attn_step": dict(q=(n, H * D, 1056), gate=(n, H * D, 1088)),
}


def shape(name):
    t, m = (n, 1) if name == "gdn_attn_step" else (T, 60)
    return attn.make_attn_shape(H, KV, D, n, t, m, 600, N, TP, PAGE, "bf16", rope_dim=32, page_stride=CACHE, q_stride=1056, k_stride=1040,
                                v_stride=1072, gate_stride=1088)


def call(name, **over):
    if name == "gdn_attn_copy_pages":
        return attn.gdn_attn_copy_pages(shape(name), **{**dict(pairs=P, n=4, k_cache=P, v_cache=P), **over}, stream=0)
    args = {**{k: P for k in DENSE[name]}, **over}
    return getattr(attn, name)(shape(name), **args, stream=0)


IN_HOST = "host memory"  # what is left to refuse of a host tensor whose layout is right


@pytest.mark.parametrize("name,arg", [(f, a) for f, d in DENSE.items() for a, v in d.items() if v])
def test_dense_tensors(name, arg):
    dtype, size = DENSE[name][arg]
    for more in (0, 3):
        with pytest.raises(ValueError, match=IN_HOST):
            call(name, **{arg: torch.zeros(size + more, dtype=dtype)})
    with pytest.raises(ValueError, match=f"{arg} has {size - 1} elements of {size}"):
        call(name, **{arg: torch.zeros(size - 1, dtype=dtype)})
    with pytest.raises(ValueError, match=f"{arg} has gaps"):
        call(name, **{arg: torch.zeros(size, 2, dtype=dtype)[:, 0]})
    with pytest.raises(ValueError, match=f"{arg} is torch.float64"):
        call(name, **{arg: torch.zeros(size, dtype=torch.float64)})


@pytest.mark.parametrize("name,arg", [(f, a) for f, d in ROWS.items() for a in d])
def test_tensors_of_rows(name, arg):
    rows, cols, stride = ROWS[name][arg]
    wide = torch.zeros(rows, stride, dtype=BF)
    heads = cols // D
    for x in (wide, wide[:, :cols], wide[:, 8:8 + cols], wide[:, :cols].unflatten(1, (heads, D)), wide.flatten()[:(rows - 1) * stride + cols],
              torch.zeros(rows + 2, stride, dtype=BF)[:, :cols]):
        with pytest.raises(ValueError, match=IN_HOST):
            call(name, **{arg: x})
    other = torch.zeros(rows, stride + 8, dtype=BF)
    for x in (other[:, :cols], wide[:-1, :cols], wide[:, :cols - 8], wide[:, :2 * cols:2], wide[:, :cols].unflatten(1, (heads, D)).transpose(1, 2),
              wide.flatten()[:(rows - 1) * stride + cols - 1], torch.zeros(stride, rows, dtype=BF).t()[:, :cols]):
        with pytest.raises(ValueError, match=f"{arg} "):
            try:
                call(name, **{arg: x})
            except ValueError as e:
                assert IN_HOST not in str(e)
                raise
    with pytest.raises(ValueError, match=f"{arg} is torch.float16"):
        call(name, **{arg: wide.half()})


@pytest.mark.parametrize("name", [*DENSE, "gdn_attn_copy_pages"])
@pytest.mark.parametrize("arg,half", [("k_cache", 0), ("v_cache", 1)])
def test_caches(name, arg, half):
    pages = torch.zeros(N, 2, KV, PAGE, D, dtype=BF)
    more = torch.zeros(N + 1, 2, KV, PAGE, D, dtype=BF)
    for x in (pages[:, half], more[:, half], pages, pages[:, half].flatten(1)):
        with pytest.raises(ValueError, match=IN_HOST):
            call(name, **{arg: x})
    layers = torch.zeros(N, 3, 2, KV, PAGE, D, dtype=BF)  # another stride
    for x in (pages[:-1, half], layers[:, 0, half], pages[:, half, :1], pages[:, half, :, :8], pages[:, half].transpose(1, 2),
              pages[:, half, ..., :32], pages[:, half].contiguous(), pages[0, half]):
        with pytest.raises(ValueError, match=arg) as e:
            call(name, **{arg: x})
        assert IN_HOST not in str(e.value)
    with pytest.raises(ValueError, match=f"{arg} is torch.float32"):
        call(name, **{arg: pages[:, half].float()})


@pytest.mark.parametrize("name", ["gdn_attn_prefill", "gdn_attn_step"])
def test_workspaces(name):
    for dtype in (torch.uint8, F32):
        with pytest.raises(ValueError, match=IN_HOST):
            call(name, workspace=torch.zeros(1000, dtype=dtype))
        with pytest.raises(ValueError, match=IN_HOST):
            call(name, workspace=torch.zeros(1000, dtype=dtype), workspace_bytes=10)
    with pytest.raises(ValueError, match="workspace of 4000 bytes, not 4001"):
        call(name, workspace=torch.zeros(1000), workspace_bytes=4001)
    with pytest.raises(ValueError, match="not -1"):
        call(name, workspace_bytes=-1)
    with pytest.raises(ValueError, match="workspace has gaps"):
        call(name, workspace=torch.zeros(1000, 2, dtype=torch.uint8)[:, 0])


def test_pairs():
    with pytest.raises(ValueError, match="pairs has 7 elements of 8"):
        call("gdn_attn_copy_pages", pairs=torch.zeros(7, dtype=I32))
    with pytest.raises(ValueError, match="pairs is torch.int64"):
        call("gdn_attn_copy_pages", pairs=torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="pairs has gaps"):
        call("gdn_attn_copy_pages", pairs=torch.zeros(2, 4, dtype=I32).t())
    with pytest.raises(ValueError, match=IN_HOST):
        call("gdn_attn_copy_pages", pairs=torch.zeros(4, 2, dtype=I32))


def test_other_shape_other_needs():
    """The needs are those of the shape of the call, whatever was called before."""
    s = shape("gdn_attn_prefill")
    for rows, ok in ((T, True), (T - 1, False), (T, True)):
        with pytest.raises(ValueError, match=IN_HOST if ok else "out has"):
            attn.gdn_attn_prefill(s, P, P, P, P, P, P, None, torch.zeros(rows, H * D, dtype=BF), P, workspace_bytes=1 << 30, stream=0)
    s.heads = 2 * H
    with pytest.raises(ValueError, match="out has"):
        attn.gdn_attn_prefill(s, P, P, P, P, P, P, None, torch.zeros(T, H * D, dtype=BF), P, workspace_bytes=1 << 30, stream=0)
