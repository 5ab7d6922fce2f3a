"""The library without the compiled binding: what is marshalled in Python works, the rest says what is missing (CPU)."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
sys.modules["nvfp4_w4a4_mixture_amd._binding"] = None  # importing it fails
import torch
from nvfp4_w4a4_mixture_amd import layer, mx_block, ops
assert ops.moe_ffn_workspace_bytes(4, 2, 8, 256, 128) > 0
x = torch.zeros((2, 64), dtype=torch.bfloat16)
for call in (lambda: ops.nvfp4_quantize_act(x, x), lambda: ops.mxfp4_quantize_weights(x[None])):
    try:
        call()
        raise SystemExit("not refused")
    except ValueError as e:
        assert "GPU" in str(e), e
for call in (lambda: ops.mxfp4_quantize(x), lambda: ops.moe_norm_in(x, x[0]), lambda: ops.mxfp4_quantize(x)):
    try:
        call()
        raise SystemExit("not refused")
    except RuntimeError as e:
        assert "binding is not built" in str(e), e
print("done")
"""


def test_ops_without_the_binding():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr[-2000:]


def test_binding_functions_are_bound_once():
    from nvfp4_w4a4_mixture_amd import _binding, ops

    assert ops._b.mxfp4_quantize is _binding.mxfp4_quantize and "moe_combine" in vars(ops._b)
    with pytest.raises(AttributeError):
        ops._b.nothing


def test_a_failed_binding_leaves_the_library(monkeypatch, tmp_path):
    """The library is linked whatever happens to the binding, and the failure is still raised."""
    from nvfp4_w4a4_mixture_amd import build

    made = []
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "none.so"))
    monkeypatch.setattr(build, "_compile", lambda src, *a: src)
    monkeypatch.setattr(build, "HIPCC", sys.executable)  # any file that exists

    def link(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def failing():
        made.append(1)
        raise RuntimeError("no compiler")

    monkeypatch.setattr(build.subprocess, "run", link)
    monkeypatch.setattr(build, "build_binding", failing)
    with pytest.raises(RuntimeError, match="no compiler"):
        build.build(out_dir=str(tmp_path / "lib"), build_dir=str(tmp_path / "b"))
    assert made and os.path.exists(tmp_path / "lib" / build.LIB_NAME)


def test_importing_ops_without_the_library_raises():
    env = dict(os.environ, MOE_NVFP4_LIB=os.path.join(ROOT, "no", "such.so"))
    r = subprocess.run([sys.executable, "-c", "import nvfp4_w4a4_mixture_amd.ops"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode != 0 and "is not built" in r.stderr
