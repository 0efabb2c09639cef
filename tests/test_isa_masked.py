"""The build's check for vector registers that are copied between the two halves of a lane-dependent branch, where the
lanes of the second half miss the copy (no GPU)."""
import glob
import os

import pytest

from gated_delta_rule_46_amd import isa_check

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# as the compiler emitted it for a kernel that ran short of registers: v155 is read by all lanes later on
LOST = """
_Zkernel:
	s_and_saveexec_b64 s[4:5], vcc
; %bb.70:
	v_and_b32_e32 v1, 48, v0
                                        ; implicit-def: $vgpr10
; %bb.71:
	v_mov_b32_e32 v155, v102
	s_mov_b64 s[22:23], s[78:79]
	s_andn2_saveexec_b64 s[4:5], s[4:5]
	s_cbranch_execz .LBB15_76
"""

FINE = """
_Zkernel:
	s_and_saveexec_b64 s[4:5], vcc
; %bb.1:
	v_and_b32_e32 v1, 48, v0
.LBB0_2:
	v_writelane_b32 v255, s96, 22
	v_cmp_gt_u32_e32 vcc, 32, v1
	s_or_saveexec_b64 s[4:5], s[4:5]
	v_mov_b32_e32 v131, s20
.LBB0_3:
	s_or_b64 exec, exec, s[4:5]
	v_mov_b32_e32 v2, v3
"""


def test_copies_that_lanes_miss_are_found():
    assert isa_check.masked_copies(LOST) == [("_Zkernel", 8, "v_mov_b32_e32 v155, v102")]
    assert [h[2] for h in isa_check.masked_copies(LOST.replace("s_andn2_saveexec", "s_or_saveexec"))] == \
        ["v_mov_b32_e32 v155, v102"]
    assert isa_check.masked_copies(FINE) == []


def test_built_listings_have_none():
    listings = sorted(glob.glob(os.path.join(ROOT, "gated_delta_rule_46_amd", "_build", "*.s")))
    if not listings:
        pytest.skip("library not built (gated_delta_rule_46_amd/build.py emits the listings)")
    for p in listings:
        with open(p) as f:
            assert isa_check.masked_copies(f.read()) == [], p
