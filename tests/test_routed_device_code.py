"""The machine code of the steps around the routed experts keeps every value in registers: no kernel uses scratch
memory, and the kernels that move rows declare no LDS beyond their few partial sums (CPU only)."""
import os

import pytest

from moe_routed_expert_amd import build as hip_build
from tests.test_device_code import kernel_metadata

# bytes of LDS a kernel of the source may declare
SOURCES = {"moe_sort.hip": 16 * 1024, "moe_permute.hip": 4 * 8 * 4, "quantize_rows.hip": 4 * 4,
           "grouped_int8.hip": 160 * 1024}


@pytest.mark.parametrize("source", sorted(SOURCES))
def test_no_scratch_and_bounded_lds(source, tmp_path):
    out = hip_build.device_asm(os.path.join(hip_build.CSRC, source), str(tmp_path / (source + ".s")))
    meta = kernel_metadata(out)
    assert meta, "no kernels found"
    for name, k in meta.items():
        assert k[".private_segment_fixed_size"] == 0, f"{name} uses scratch memory"
        assert k[".group_segment_fixed_size"] <= SOURCES[source], f"{name} declares {k['.group_segment_fixed_size']}"
