"""What include/gdn_attn.h says of the attention workspaces' sizes: a bound for every
shape of the same heads, head width and type, from which a program allocates once, and which sizes a
step's grows with.  No GPU: host queries only."""
import itertools

import pytest

from gated_deltanet_linear_pre_amd import attn

TOKENS = [0, 1, 5, 16, 64, 100, 255, 391, 512, 1024, 1500, 2048, 4097, 8192, 1 << 17, 1 << 26]
KV = [0, 1, 1000, 4096, 32768, 1 << 17, 1 << 30]


def shape(H, kv_heads, D, io, T, kv, n=1, window=0, max_T=None):
    return attn.make_attn_shape(H, kv_heads, D, n, T, T if max_T is None else max_T, kv, 1 << 20, max(1, -(-kv // 64)), 64, io, window=window)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_a_prompts_workspace_is_bounded(io, D):
    P, R = 512 if D <= 128 else 256, 64 if io == "f32" else 128
    bound, most = 8 * P * R * (D + 2) + 32 * P, 0
    for (H, kv_heads), T, kv, n, window in itertools.product([(1, 1), (8, 2), (16, 2), (32, 8), (24, 1), (128, 1), (4096, 64)], TOKENS, KV, (1, 7, 300),
                                                             (0, 1024)):
        need = attn.gdn_attn_prefill_workspace_bytes(shape(H, kv_heads, D, io, T, kv, n, window))
        assert 0 <= need <= bound, (H, kv_heads, T, kv, n, window)
        most = max(most, need)
    assert most > 0.9 * bound  # (and it is no idle one)


def test_a_smaller_prompt_may_need_more():
    need = [attn.gdn_attn_prefill_workspace_bytes(shape(16, 2, 256, "bf16", T, 32768)) for T in (1024, 8192)]
    assert need[0] > need[1] == 0


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,kv_heads", [(1, 1), (16, 2), (64, 1), (4096, 64)])
def test_a_steps_workspace_grows_with_its_sizes(io, D, H, kv_heads):
    size = lambda n, kv, window: attn.gdn_attn_step_workspace_bytes(shape(H, kv_heads, D, io, n, kv, n, window, 1))  # noqa: E731
    for window in (0, 1, 100, 5000):
        for n in (1, 3, 300):
            needs = [size(n, kv, window) for kv in KV]
            assert needs == sorted(needs)
        for kv in KV:
            needs = [size(n, kv, window) for n in (1, 2, 3, 64, 300, 65536)]
            assert needs == sorted(needs)
    for kv in KV:
        assert all(size(3, kv, window) <= size(3, kv, 0) for window in (1, 100, 5000))


@pytest.mark.parametrize("scale,code", [(2.0 ** 127, 0), (2.0 ** 127 * (1 + 2.0 ** -23), -2), (2.4e38, -2), (3.4e38, -2), (2.0 ** -149, 0)])
def test_scales_that_the_kernels_can_form(scale, code):
    """Scores are formed times scale log2(e), which has to be finite: refused, or (with no rows) not."""
    s = shape(8, 2, 128, "bf16", 0, 100)
    s.scale = scale
    P = 0x10000  # an address that is never used
    need = attn.gdn_attn_prefill_workspace_bytes(s)
    assert attn.gdn_attn_prefill(s, P, P, P, P, P, P, None, P, P, workspace_bytes=need, stream=0, check=False) == code
    assert attn.gdn_attn_append(s, P, P, P, None, P, P, P, None, None, None, P, P, P, stream=0, check=False) == code
