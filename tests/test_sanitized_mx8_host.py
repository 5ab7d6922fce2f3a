"""The MXFP8 entry points' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): their refusals
(tests/test_abi_mx8_host.py) and sizes whose products leave 64 bits."""

import os
import subprocess
import sys

from test_sanitized_host import ROOT, _env, sanitized  # noqa: F401

SIZES = """
from nvfp4_w4a4_mixture_amd import _lib
L, big, P, Q = _lib.lib(), (1 << 63) - 1, 0x10000, 0x20000
for a in [(big, 8, 8, 256, 128), (4, big, 8, 256, 128), (4, 2, 8, 256, big), (1 << 40, 8, 8, 256, 1 << 40)]:
    assert L.mxfp8_ffn_workspace_bytes(*a) == 0, a
for T, H, E, k, I in [(big, 256, 8, 2, 128), (33, 256, 8, 2, 128), (4, big - 31, 8, 2, 128), (4, 256, big, 2, 128),
                      (4, 256, 8, big, 128), (4, 256, 8, 2, big - 31), (4, 1 << 24, 8, 2, 1 << 24)]:
    assert L.mxfp8_moe_layer_workspace_bytes(T, H, E, k, I) == 0
    assert L.mxfp8_moe_layer(P, T, H, big, P, P, E, k, 1.0, P, P, P, P, I, 0, P, P, P, P, big, None) == 2
for a in [(32, (1 << 24) - 32, 256, 256, (1 << 24) - 32), (32, 32, 256, 256, 32), (1, 32, 1, 1, (1 << 24) - 32)]:
    need = L.mxfp8_moe_layer_workspace_bytes(*a)
    T, H, E, k, I = a
    assert need % 256 == 0 and need > T * k * I
    assert L.mxfp8_moe_layer(P, T, H, H, P, P, E, k, 1.0, P, P, P, P, I, 0, P, P, P, P, need - 1, None) == 4
for dt in (0, 1):
    assert L.mxfp8_quantize(P, dt, 4, 64, big, P, P, None) == 3  # a stride that is no multiple of 16 bytes
    assert L.mxfp8_dequantize(P, P, 4, 64, dt, P, big, None) == 3
    assert L.mxfp8_linear(P, P, 4, 64, P, P, 40, None, 0, None, 0, 0, dt, Q, big, None) == 2
    assert L.mxfp8_linear(P, P, 4, 64, P, P, 40, None, 0, P, 0, big, dt, Q, 40, None) == 2
    assert L.mxfp8_linear(P, P, big, 64, P, P, 40, None, 0, None, 0, 0, dt, Q, 40, None) == 2
    assert L.mxfp8_linear(P, P, 4, big - 31, P, P, big, None, 0, None, 0, 0, dt, Q, big, None) == 2
for T, H, E, I, k in [(big, 256, 8, 128, 2), (4, big - 31, 8, 128, 2), (4, 256, 8, big - 31, 2), (4, 256, big, 128, big)]:
    assert L.mxfp8_grouped_ffn(P, P, T, H, P, P, P, P, P, E, I, k, P, P, P, P, P, P, big, None) == 2
for rows, cols in [(big, 64), (4, big - 31), (1 << 40, 1 << 40)]:
    assert L.mxfp8_quantize(P, 0, rows, cols, big, P, P, None) == 2
    assert L.moe_norm_in_mxfp8(P, rows, cols, big, P, 1e-6, P, big, P, P, None) == 2
    assert L.moe_norm_out_mxfp8(P, 1, rows, cols, big, P, big, P, None, 0, 0, 1.0, P, 1e-6, Q, big, None, 0, P, P, None) == 2
print("done")
"""


def test_refusals_under_sanitizers(sanitized):  # noqa: F811
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_mx8_host.py")],
                       cwd=ROOT, env=_env(*sanitized), capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and " passed" in out, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out


def test_large_sizes_under_sanitizers(sanitized):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", SIZES], cwd=ROOT, env=_env(*sanitized), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), (r.stdout + r.stderr)[-3000:]
