"""No kernel's vector-memory instruction reads a scalar register too soon after it was
written (see tests/asm_waits.py).  The assembly is that of
tests/test_asm_hazards.py, every csrc/*.hip compiled with the library's own flags."""
import os

import pytest

from gated_deltanet_linear_pre_amd import build as B
from tests.asm_waits import short_waits
from tests.test_asm_hazards import SOURCES, _asm


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src", SOURCES, ids=[os.path.basename(s) for s in SOURCES])
def test_no_load_reads_a_scalar_register_too_soon(src, tmp_path):
    found = short_waits(_asm(src, tmp_path))
    assert not found, f"{len(found)}\n" + "\n".join(f"{f[:60]} line {n}: {ins} (s{r} after {w} of {need})" for f, n, ins, r, w, need in found[:20])


COPY = ["\ts_mov_b32 m0, s7", "\ts_nop %d", "\tglobal_load_lds_dwordx4 v18, s[8:9]", "\ts_endpgm"]


def planted(*before, nop=0):
    return "\n".join(["_Zplanted:", *before, *COPY]) % nop


@pytest.mark.parametrize("before,nop,want", [
    (["\tv_readlane_b32 s9, v13, 0", "\tv_readlane_b32 s8, v12, 0"], 0, [(8, 2)]),
    (["\tv_readlane_b32 s9, v13, 0", "\tv_readlane_b32 s8, v12, 0"], 2, [(8, 4)]),
    (["\tv_readlane_b32 s9, v13, 0", "\tv_readlane_b32 s8, v12, 0"], 3, []),
    (["\tv_readlane_b32 s9, v13, 0", "\ts_mov_b32 s8, 0"], 0, [(9, 3)]),
    (["\tv_readlane_b32 s9, v13, 0", "\ts_add_u32 s8, s8, s2", "\ts_addc_u32 s9, s9, s3"], 0, [(9, 4)]),  # as the compiler counts
    (["\tv_readlane_b32 s10, v13, 0"], 0, []),
    (["\tv_cmp_eq_u32_e64 s[8:9], v1, v2"], 0, [(8, 2)]),
    (["\tv_add_co_u32_e64 v3, s[8:9], v1, v2"], 0, [(8, 2)]),
    # on one way out of two, and round a loop
    (["\ts_cbranch_scc1 .L1", "\tv_readlane_b32 s8, v12, 0", "\ts_nop 1", ".L1:"], 0, [(8, 4)]),
    (["\tv_readlane_b32 s8, v12, 0", "\ts_cbranch_scc1 .L1", "\ts_nop 7", ".L1:"], 0, [(8, 3)]),
    (["\ts_branch .L2", ".L1:", "\tv_readlane_b32 s8, v12, 0", "\ts_branch .L3", ".L2:", "\ts_nop 7", "\ts_branch .L1", ".L3:"], 0, [(8, 3)]),
])
def test_checker_counts_wait_states(before, nop, want):
    found = short_waits(planted(*before, nop=nop))
    assert [(x[3], x[4]) for x in found] == want


def test_checker_knows_m0():
    asm = "\n".join(["_Zplanted:", COPY[0], *COPY[2:]])
    assert [(x[3], x[4], x[5]) for x in short_waits(asm)] == [("m0", 0, 1)]
