"""Host-side sanitizers for the rotated append and the 4-bit cache's calls (CPU, no
GPU): the refusals of test_kv_q4_abi_cpu.py and a sweep of extreme descriptors in the
library's sanitized host code.  Any report aborts the child and fails the test."""

import os

import pytest

from tests.test_host_sanitizers import ASAN_RT, HIPCC, ROOT, asan_lib  # noqa: F401
from tests.test_kv_host_sanitizers import _run

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
        [-1, 0, 1, 65536, big], [0, 1, 1 << 20, big],
        [(1, 1), (65536, 65536), (64, 8), (65536, 1), (7, 2)], [32, 64, 160, 256, big], [1, 16, big],
        [0, 1, 1 << 20, big], [0, 1, big]):
    for dt, window, stride, scale in ((1, 0, 0, 1.0), (2, big, 2**40, 3e38), (2, 1, 2**62, 1e-45),
                                      (1, 5, -2**63, 0.5), (2, big, 0, 2.0)):
        d = kv.AttentionDesc(B, T, heads, kvh, dim, bs, nb, width, dt, window, big if window else 0,
                             0, stride, 0, scale, 0.0)
        planned += lib.kv_paged_attention_q4_workspace_bytes(ctypes.byref(d)) > 0
        # no pointers: a plan that passes is refused for them, or has nothing to do
        lib.kv_paged_attention_q4(ctypes.byref(d), *[None] * 11, 0, None)
        for rot in (0, 2, dim, -big):
            r = kv.RotaryDesc(T, heads, kvh, dim, bs, nb, dt, rot, window & 1, width, stride, stride,
                              stride, stride, stride if rot == 2 else 0)
            lib.kv_cache_append_rotary(ctypes.byref(r), *[None] * 9, None)
            lib.kv_cache_append_q4(ctypes.byref(r), *[None] * 11, None)
        lib.kv_cache_read_q4(T, kvh, dim, bs, nb, dt, *[None] * 7, None)
        n += 1
assert planned > 100, planned
print("sweep", n)
'''


def test_extreme_descriptors_are_clean(asan_lib):   # noqa: F811
    r = _run(asan_lib, ["-c", SWEEP, ROOT])
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "runtime error" not in r.stderr
    assert "sweep" in r.stdout


def test_refusals_are_clean(asan_lib):   # noqa: F811
    r = _run(asan_lib, ["-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_kv_q4_abi_cpu.py")])
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "runtime error" not in r.stderr
