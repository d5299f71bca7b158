"""The work search of the attention over a 4-bit cache on the CPU (no GPU), as
test_kv_work_split.py has it for the other caches."""

import os
import subprocess

import pytest

from tests.test_kv_work_split import CLANG, CSRC, ROOT, WAVE


@pytest.mark.skipif(not os.path.exists(CLANG), reason="clang is not installed")
def test_every_item_is_found_by_all_threads(tmp_path):
    exe = str(tmp_path / "split")
    r = subprocess.run([CLANG, "-std=c++17", "-O2", "-w", "-I" + WAVE, "-I" + CSRC,
                        "-I" + os.path.join(ROOT, "include"), "-x", "c++",
                        os.path.join(WAVE, "kv_work_split_q4.cpp"), os.path.join(CSRC, "kvapi.hip"),
                        os.path.join(CSRC, "kvapi_q4.hip"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:]
    assert r.stdout.splitlines()[-1].startswith("work split ok")
