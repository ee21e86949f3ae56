"""The attention kernels' registers: none of them spills to scratch memory, and their LDS
fits as often as their launch bounds ask.  Compiles them to assembly with the library's own
flags (hipcc cross-compiles without a GPU)."""
import os
import re
import subprocess

import pytest

from gated_deltanet_linear_pre_amd import build as B

LDS = 160 * 1024  # of a CU


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src,kernels", [("attn_append.hip", 15), ("attn_copy.hip", 1), ("attn_prefill.hip", 45), ("attn_step.hip", 45)])
def test_no_scratch(src, kernels, tmp_path):
    out = tmp_path / "a.s"
    flags = [f for f in B.CFLAGS if f != "-fPIC"]
    r = subprocess.run([B.HIPCC, *flags, "--offload-device-only", "-S", os.path.join(B.CSRC, src), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = out.read_text()
    found = re.findall(r"\.amdhsa_kernel (\S+)\s+\.amdhsa_group_segment_fixed_size (\d+)\s+\.amdhsa_private_segment_fixed_size (\d+)", asm)
    assert len(found) == kernels
    for name, lds, scratch in found:
        assert int(scratch) == 0, name
        assert int(lds) <= LDS, name
        # prompts of heads up to 128 wide: two blocks a CU
        if "prefill_kernel" in name and re.search(r"Li(64|96|128)E", name):
            assert 2 * int(lds) <= LDS, name
