"""Prompts whose max_kv is far above their lengths, as in a captured call that is sized for its
page table, with more blocks of rows than are resident at once: their keys are dealt by the
lengths on the device, not by the bound.  Tolerances are those of test_gpu_attn.py."""
import pytest
import torch

from gated_deltanet_linear_pre_amd import attn

from .gpu_util import banner
from .test_gpu_attn import IO, Case

pytestmark = pytest.mark.gpu

MAX_KV = 30000


def bounded(c):
    """The case's sizes with max_kv far above its lengths (and pages of none in the table)."""
    pages = -(-MAX_KV // c.page)
    c.table_t = torch.cat([c.table_t, torch.full((c.n, pages - c.table_t.shape[1]), 1 << 30, dtype=torch.int32, device="cuda")], 1)
    return dict(max_kv=MAX_KV, table_pages=pages)


# new, past, H, KV, D, window: rows of nearly the same few keys (heads of D wide, two query heads to a key head: 64 tokens a
# block, 32 in fp32)
SHORT = [([520], [0], 64, 32, 256, 0), ([300, 0, 217], [0, 5, 40], 64, 32, 192, 0), ([600], [30], 128, 64, 64, 0), ([1, 520, 3], [0, 0, 9], 128, 64, 128, 0),
         ([520], [0], 64, 32, 256, 100)]


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("new,past,H,KV,D,window", SHORT, ids=[f"{c[0]}-D{c[4]}w{c[5]}" for c in SHORT])
def test_short_prompts_under_a_large_bound_are_not_dealt(gpu, io, new, past, H, KV, D, window):
    banner("gdn_attn_prefill bounds", io, new, past, H, KV, D, window)
    c = Case([n // 2 if io == "f32" else n for n in new], past, H, KV, D, 16, io, window=window, tail=2, stale=float("nan"))
    assert attn.gdn_attn_prefill_workspace_bytes(c.shape()) == 0
    want = c.run("prefill")
    c.check("prefill", want)
    more = bounded(c)
    if not window:
        assert attn.gdn_attn_prefill_workspace_bytes(c.shape(**more)) > 0
    got = c.run("prefill", **more)
    assert torch.equal(want[:c.used], got[:c.used])  # rows that are not cut: the same sums in the same order


# long caches under a larger bound: dealt, or not, whichever pays
LONG = [([700], [3000], 24, 4, 256), ([600, 90], [4000, 0], 24, 4, 256), ([300], [9000], 64, 32, 128)]


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("new,past,H,KV,D", LONG, ids=[f"{c[0]}-D{c[4]}" for c in LONG])
def test_long_prompts_under_a_larger_bound(gpu, io, new, past, H, KV, D):
    banner("gdn_attn_prefill bounds, long", io, new, past, H, KV, D)
    c = Case([n // 2 if io == "f32" else n for n in new], past, H, KV, D, 16, io, tail=2, stale=float("nan"))
    a = c.run("prefill", **bounded(c))
    c.check("prefill", a)
    assert torch.equal(a[:c.used], c.run("prefill", max_kv=MAX_KV, table_pages=c.table_t.shape[1])[:c.used])
