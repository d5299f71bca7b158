"""Appends and read-backs of the 4-bit cache in parts, on the CPU under AddressSanitizer
and UndefinedBehaviorSanitizer (tests/hostwave/kv_q4_parts.cpp)."""

import os
import subprocess

import pytest

from tests.test_kv_work_split import CLANG, CSRC, ROOT, WAVE


@pytest.mark.skipif(not os.path.exists(CLANG), reason="clang is not installed")
def test_parts_are_whole_and_clean(tmp_path):
    exe = str(tmp_path / "parts")
    r = subprocess.run([CLANG, "-std=c++17", "-O1", "-g", "-w", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=all", "-I" + WAVE, "-I" + CSRC,
                        "-I" + os.path.join(ROOT, "include"), os.path.join(WAVE, "kv_q4_parts.cpp"),
                        "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-3000:])
    assert "runtime error" not in r.stderr
    assert r.stdout.startswith("parts ok")
