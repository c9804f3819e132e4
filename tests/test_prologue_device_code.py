"""The machine code of the steps before the experts keeps every value in registers: no kernel uses scratch memory, and
none declares more LDS than two blocks of a CU have (the router's float32 operands, and more than 256 experts: one).
Loops around a kernel made the compiler keep its constants in registers from pass to pass: the choice's kernels stay
below 128 (CPU only)."""
import os

import pytest

from moe_routed_expert_amd import build as hip_build
from tests.test_device_code import kernel_metadata

SOURCES = {"rms_norm.hip": 16 * 1024, "moe_route.hip": 40 * 1024, "router_logits.hip": 160 * 1024}


@pytest.mark.parametrize("source", sorted(SOURCES))
def test_no_scratch_and_bounded_lds(source, tmp_path):
    out = hip_build.device_asm(os.path.join(hip_build.CSRC, source), str(tmp_path / (source + ".s")))
    meta = kernel_metadata(out)
    assert meta, "no kernels found"
    for name, k in meta.items():
        assert k[".private_segment_fixed_size"] == 0, f"{name} uses scratch memory"
        assert k[".group_segment_fixed_size"] <= SOURCES[source], f"{name} declares {k['.group_segment_fixed_size']}"
        if source == "moe_route.hip":
            assert k[".vgpr_count"] <= 128, f"{name} takes {k['.vgpr_count']} registers"
