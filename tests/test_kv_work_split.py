"""The attention's work search on the CPU (no GPU): tests/hostwave builds the host
code of kv_paged_attention and the device code of attend_find for the CPU, every
thread of a workgroup in lockstep, and checks every item of a sweep of batches --
barriers and lane exchanges met by all threads, every key unit of every tile
taken once, within the launch and the workspace."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"
CSRC = os.path.join(ROOT, "lossless_token_verification_amd", "csrc")
WAVE = os.path.join(ROOT, "tests", "hostwave")


@pytest.mark.skipif(not os.path.exists(CLANG), reason="clang is not installed")
def test_every_item_is_found_by_all_threads(tmp_path):
    exe = str(tmp_path / "split")
    r = subprocess.run([CLANG, "-std=c++17", "-O2", "-w", "-I" + WAVE, "-I" + CSRC,
                        "-I" + os.path.join(ROOT, "include"), "-x", "c++",
                        os.path.join(WAVE, "kv_work_split.cpp"), os.path.join(CSRC, "kvapi.hip"),
                        "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:]
    assert r.stdout.splitlines()[-1].startswith("work split ok")
