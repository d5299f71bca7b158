"""Compiler resource report of the rotated append's and the 4-bit cache's kernels
(CPU, no GPU needed).  The attention's are tiled for two or three wavefronts to a
SIMD: some hold a few values in scratch memory (up to 26 accesses a unit), and a
configuration that spills more (head_dim 256 in tiles of 16 rows took 208 bytes and
eight times as long) shows here."""

import os
import re
import shutil
import subprocess

import pytest

from tests.test_kv_kernel_resources import CSRC, HIPCC, ROOT


@pytest.mark.skipif(not os.path.exists(HIPCC) or shutil.which("ld.lld") is None and
                    not os.path.exists("/opt/rocm/llvm/bin/ld.lld"),
                    reason="hipcc is not installed")
@pytest.mark.parametrize("src,kernels,most,waves", [
    ("kvrotary.hip", 6, 0, 4), ("kvq4.hip", 15, 0, 4), ("kvattend_q4_d64.hip", 16, 32, 2),
    ("kvattend_q4_d128.hip", 16, 96, 2), ("kvattend_q4_d256.hip", 12, 64, 2)])
def test_scratch_and_registers(src, kernels, most, waves):
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Xclang",
           "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-c",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, os.path.join(CSRC, src),
           "-o", os.devnull, "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]

    def figures(name):
        return [int(n) for n in re.findall(name + r"[^:]*: (\d+)", out.stderr)]
    scratch = figures("ScratchSize")
    assert len(scratch) == kernels, (src, len(scratch))
    assert max(scratch) <= most, scratch
    assert not any(figures("AGPRs"))
    assert min(figures("Occupancy")) >= waves
