"""The MXFP4 and norm entry points' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): their
refusals (tests/test_abi_mx_host.py) and sizes whose products leave 64 bits."""

import os
import subprocess
import sys

from test_sanitized_host import ROOT, _env, sanitized  # noqa: F401

SIZES = """
from nvfp4_w4a4_mixture_amd import _lib
L, big, P = _lib.lib(), (1 << 63) - 1, 0x10000
for a in [(big, 8, 8, 256, 128), (4, big, 8, 256, 128), (4, 2, 8, 256, big), (1 << 40, 8, 8, 256, 1 << 40)]:
    assert L.mxfp4_ffn_workspace_bytes(*a) == 0, a
assert L.mxfp4_linear_workspace_bytes(big, big, big) == 0
for dt in (0, 1):
    assert L.mxfp4_quantize(P, dt, 4, 64, big, P, P, None) == 3  # a stride that is no multiple of 16 bytes
    assert L.mxfp4_dequantize(P, P, 4, 64, dt, P, big, None) == 3
    assert L.mxfp4_linear(P, P, 4, 64, P, P, 40, dt, P, big, None, 0, None) == 2
    assert L.mxfp4_linear(P, P, big, 64, P, P, 40, dt, P, 40, None, 0, None) == 2
for T, H, E, I, k in [(big, 256, 8, 128, 2), (4, big - 31, 8, 128, 2), (4, 256, 8, big - 31, 2), (4, 256, big, 128, big)]:
    assert L.mxfp4_grouped_ffn(P, P, T, H, P, P, P, P, P, E, I, k, P, P, P, P, P, P, big, None) == 2
for rows, cols in [(big, 64), (4, big - 31), (1 << 40, 1 << 40)]:
    assert L.mxfp4_quantize(P, 0, rows, cols, big, P, P, None) == 2
    assert L.mxfp4_quantize_weights(P, 1, rows, cols, P, P, P, None) == 2
    assert L.moe_norm_in(P, rows, cols, big, P, 1e-6, P, big, P, P, None) == 2
print("done")
"""


def test_refusals_under_sanitizers(sanitized):  # noqa: F811
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_mx_host.py")],
                       cwd=ROOT, env=_env(*sanitized), capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and " passed" in out, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out


def test_large_sizes_under_sanitizers(sanitized):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", SIZES], cwd=ROOT, env=_env(*sanitized), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), (r.stdout + r.stderr)[-3000:]
