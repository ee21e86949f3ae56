"""A kernel that runs out of vector registers keeps some in scratch memory or in accumulation
registers.  What brings them back are loads like any other: scratch loads may not land on
an operand of a product in flight either, nor may loads into accumulation registers (the rule
of tests/asm_hazards.py, which looks at LDS and global loads into vector registers).  The assembly is that of
tests/test_asm_hazards.py, every csrc/*.hip compiled with the library's own flags."""
import os
import re

import pytest

from gated_deltanet_linear_pre_amd import build as B
from tests import asm_hazards
from tests.test_asm_hazards import SOURCES, _asm


def loads_over_operands(asm_text, monkeypatch):
    monkeypatch.setattr(asm_hazards, "_LOADS", asm_hazards._LOADS + ("scratch_load", "flat_load"))
    # accumulation register n as vector register 1000 + n, which no kernel has
    text = re.sub(r"\ba\[(\d+):(\d+)\]", lambda m: f"v[{1000 + int(m[1])}:{1000 + int(m[2])}]", asm_text)
    return asm_hazards.load_over_mfma_operands(re.sub(r"\ba(\d+)\b", lambda m: f"v{1000 + int(m[1])}", text))


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src", SOURCES, ids=[os.path.basename(s) for s in SOURCES])
def test_no_spill_overwrites_an_mfma_operand_in_flight(src, tmp_path, monkeypatch):
    found = loads_over_operands(_asm(src, tmp_path), monkeypatch)
    assert not found, "\n".join(f"{f[:60]} line {n}: {ins} (MFMA at line {m})" for f, n, ins, m in found)


@pytest.mark.parametrize("operands,load,found", [
    ("v[4:7], v[8:11], 0", "scratch_load_dwordx4 v[4:7], off, off offset:16", True),
    ("v[4:7], v[8:11], 0", "scratch_load_dword v9, off, s32", True),
    ("v[4:7], v[8:11], 0", "scratch_load_dword v12, off, s32", False),
    ("v[4:7], v[8:11], 0", "scratch_store_dword off, v4, s32", False),
    ("a[4:7], v[8:11], 0", "ds_read_b128 a[4:7], v20", True),
    ("v[4:7], v[8:11], 0", "ds_read_b128 a[4:7], v20", False),
])
def test_checker_flags_a_planted_spill(operands, load, found, monkeypatch):
    asm = "\n".join(["_Zplanted:", f"\tv_mfma_f32_16x16x32_f16 v[0:3], {operands}", f"\t{load}", "\tv_add_f32_e32 v30, v0, v1"])
    assert bool(loads_over_operands(asm, monkeypatch)) == found
