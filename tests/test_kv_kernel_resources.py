"""Compiler resource report of the paged-KV kernels (CPU, no GPU needed): no
kernel may use scratch memory, and the attention kernels keep to the registers
of the wavefronts per SIMD they are tiled for."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lossless_token_verification_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC) or shutil.which("ld.lld") is None and
                    not os.path.exists("/opt/rocm/llvm/bin/ld.lld"),
                    reason="hipcc is not installed")
@pytest.mark.parametrize("src,kernels", [
    ("kvblocks.hip", 3), ("kvappend.hip", 3), ("kvattend_rows.hip", 6),
    ("kvattend_d64.hip", 12), ("kvattend_d128.hip", 12), ("kvattend_d256.hip", 8)])
def test_no_kernel_uses_scratch(src, kernels):
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Xclang",
           "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-c",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, os.path.join(CSRC, src),
           "-o", os.devnull, "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    scratch = [int(n) for n in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", out.stderr)]
    agprs = [int(n) for n in re.findall(r"AGPRs: (\d+)", out.stderr)]
    assert len(scratch) == kernels, (src, len(scratch))
    assert not any(scratch), scratch
    # accumulators moved through the other half of the register file cost a move per
    # accumulator and unit
    assert not any(agprs), agprs
