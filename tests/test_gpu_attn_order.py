"""Prompts whose blocks are taken in another order: as many as are resident at once (512 of
heads up to 128 wide), a few less and more, and those whose last rows make one more of them.
Tolerances are those of test_gpu_attn.py."""
import pytest

from .gpu_util import banner
from .test_gpu_attn import IO, Case

pytestmark = pytest.mark.gpu


# 64 key-value heads of one query head each: 128 tokens a block (64 in fp32), 64 blocks along the heads
@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("new", [[512], [1000], [1024], [1025], [1100], [500, 24], [300, 0, 1, 700]], ids=str)
def test_blocks_about_as_many_as_are_resident(gpu, io, new):
    banner("gdn_attn_prefill order", io, new)
    c = Case([n // 2 if io == "f32" else n for n in new], [0] * len(new), 64, 64, 64, 16, io, tail=1)
    c.run_and_check("prefill")
