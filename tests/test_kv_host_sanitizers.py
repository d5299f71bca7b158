"""Host-side sanitizers for the paged-KV calls (CPU, no GPU): the library's
host code built with AddressSanitizer and UndefinedBehaviorSanitizer (device
code unchanged), under the refusals of test_kv_abi_cpu.py and a sweep of extreme
descriptors.  Any report aborts the child and fails the test."""

import os
import subprocess
import sys

import pytest

from tests.test_host_sanitizers import ASAN_RT, HIPCC, ROOT, _env, asan_lib  # noqa: F401

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC) or not ASAN_RT,
                                reason="hipcc or the sanitizer runtime is not installed")

SWEEP = r'''
import ctypes, itertools, sys
sys.path.insert(0, sys.argv[1])
import lossless_token_verification_amd as sv
from lossless_token_verification_amd import kv
lib = sv.library()
big = 2**31 - 1
n = planned = 0
for B, T, (heads, kvh), dim, bs, nb, width in itertools.product(
        [-1, 0, 1, 4096, big], [0, 1, 1 << 20, big],
        [(1, 1), (65536, 65536), (64, 8), (65536, 1), (7, 2)], [8, 64, 256, big], [1, 16, big],
        [0, 1, 1 << 20, big], [0, 1, big]):
    for dt, window, stride, scale in ((0, 0, 0, 1.0), (1, big, 2**40, 3e38), (2, 1, 2**62, 1e-45),
                                      (1, 5, -2**63, 0.5), (1, big, 0, 2.0)):
        d = kv.AttentionDesc(B, T, heads, kvh, dim, bs, nb, width, dt, window, big if window else 0,
                             0, stride, stride, scale, 0.0)
        planned += lib.kv_paged_attention_workspace_bytes(ctypes.byref(d)) > 0
        # no pointers: a plan that passes is refused for them, or has nothing to do
        lib.kv_paged_attention(ctypes.byref(d), *[None] * 9, 0, None)
        a = kv.AppendDesc(T, kvh, dim, bs, nb, dt, stride, stride, stride)
        lib.kv_cache_append(ctypes.byref(a), *[None] * 5, None)
        n += 1
for v in itertools.product([-2**31, -1, 0, 1, big], repeat=4):
    lib.kv_blocktable_extend(v[0], v[1], v[2], *[None] * 4, v[3], None, None, v[1], None, v[0],
                             *[None] * 7)
assert planned > 100, planned
print("sweep", n)
'''


def _run(lib, args):
    return subprocess.run([sys.executable, *args], capture_output=True, text=True, env=_env(lib),
                          cwd=ROOT, timeout=600)


def test_extreme_descriptors_are_clean(asan_lib):   # noqa: F811
    r = _run(asan_lib, ["-c", SWEEP, ROOT])
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "runtime error" not in r.stderr
    assert "sweep" in r.stdout


def test_refusals_are_clean(asan_lib):   # noqa: F811
    r = _run(asan_lib, ["-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_kv_abi_cpu.py")])
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "runtime error" not in r.stderr
