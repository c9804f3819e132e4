"""The loads of the router's weight gradient stay inside its tensors (csrc/router_map.h), checked on the CPU.

A host-only build of the library's own header walks the steps that load without bounds the way the kernel's lanes do,
for every row length and number of tokens around a step's, and adds up which elements they reach.
"""
import os
import shutil
import subprocess

import pytest

from moe_routed_expert_amd import build as hip_build

SOURCE = r'''
#include <hip/hip_runtime.h>
#include "router_map.h"
#include <cstdio>
using namespace moe_epi;

int main() {
    int bad = 0, n = 0;
    for (int width : {2, 4})                                   // float32 and 16-bit elements of 8 bytes
        for (int64_t hidden = 1; hidden <= 20; ++hidden)
            for (int64_t tokens = 1; tokens <= 300; ++tokens) {
                const int64_t inside = steps_inside(tokens, hidden, width), steps = (tokens + kGradStep - 1) / kGradStep;
                int64_t most = -1;                             // the last element that a lane loads
                for (int64_t s = 0; s < inside; ++s)
                    for (int64_t t = s * kGradStep; t < (s + 1) * kGradStep; ++t)
                        for (int64_t h = 0; h < hidden; h += width)
                            most = t * hidden + h + width - 1 > most ? t * hidden + h + width - 1 : most;
                ++n;
                const bool early = inside + 1 < steps && hidden >= width;   // no more steps than needed go by bounds
                if (inside < 0 || inside > steps || most >= tokens * hidden || early) {
                    if (++bad < 10)
                        printf("width=%d hidden=%ld tokens=%ld: steps inside %ld of %ld, last element %ld of %ld\n", width,
                               (long)hidden, (long)tokens, (long)inside, (long)steps, (long)most, (long)(tokens * hidden));
                }
            }
    printf("walks %d failed %d\n", n, bad);
    return bad != 0;
}
'''


def test_loads_without_bounds_stay_in_the_tensor(tmp_path):
    hipcc = hip_build.HIPCC
    if not (os.path.exists(hipcc) or shutil.which(hipcc)):
        pytest.skip("hipcc not available")
    src, exe = tmp_path / "routermap.cpp", tmp_path / "routermap"
    src.write_text(SOURCE)
    cmd = [hipcc, "-x", "hip", "--cuda-host-only", "-std=c++17", "-O1", f"-I{hip_build.INCLUDE}", f"-I{hip_build.CSRC}",
           str(src), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "failed 0" in run.stdout
